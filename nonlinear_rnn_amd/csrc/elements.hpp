// Single float32 or bfloat16 elements of device arrays.
#pragma once

#include "scan.hpp"

namespace pararnn {

template <bool BF16>
__device__ __forceinline__ float load_gate(const void *p, int64_t i)
{
    if constexpr (BF16)
        return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    else
        return static_cast<const float *>(p)[i];
}
// float32 to bfloat16, nearest even; a NaN stays one.
__device__ __forceinline__ uint32_t bf16_bits(float x)
{
    const uint32_t b = __float_as_uint(x);
    return x != x ? (b >> 16) | 0x40u : (b + 0x7fffu + ((b >> 16) & 1u)) >> 16;
}
template <bool BF16>
__device__ __forceinline__ void store_gate(void *p, int64_t i, float x)
{
    if constexpr (BF16)
        static_cast<uint16_t *>(p)[i] = (uint16_t)bf16_bits(x);
    else
        static_cast<float *>(p)[i] = x;
}

}  // namespace pararnn
