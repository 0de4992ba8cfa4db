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

// K contiguous elements at any element address: 16-byte accesses, which
// gfx9 global memory takes at any alignment (unaligned-access-mode, on for
// every amdhsa target).
typedef uint32_t Words4 __attribute__((ext_vector_type(4)));
typedef uint32_t Words2 __attribute__((ext_vector_type(2)));
typedef Words4 __attribute__((aligned(2))) Words4Any;
typedef Words2 __attribute__((aligned(2))) Words2Any;
typedef uint32_t __attribute__((aligned(2))) Word1Any;

// K elements as loaded: 2 or 4 bytes each.
template <bool BF16, int K>
struct Raw {
    static constexpr int kWords = BF16 ? K / 2 : K;
    static_assert(kWords % 4 == 0, "16-byte accesses");
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int k) const
    {
        if constexpr (BF16)
            return __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
        else
            return __uint_as_float(w[k]);
    }
    __device__ __forceinline__ void set(const float (&v)[K])
    {
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            if constexpr (BF16)
                w[j] = bf16_bits(v[2 * j]) | bf16_bits(v[2 * j + 1]) << 16;
            else
                w[j] = __float_as_uint(v[j]);
        }
    }
};

// Elements first .. first + K - 1 of a row (its first element at `off`), the
// ones from `end` on left zero.
template <bool BF16, int K>
__device__ __forceinline__ Raw<BF16, K> load_raw(const void *p, int64_t off, int64_t first,
                                                 int64_t end)
{
    constexpr int N = Raw<BF16, K>::kWords;
    const char *a = static_cast<const char *>(p) + (off + first) * (BF16 ? 2 : 4);
    Raw<BF16, K> r;
    if (first + K <= end) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const Words4 v = *reinterpret_cast<const Words4Any *>(a + 4 * j);
            r.w[j] = v.x, r.w[j + 1] = v.y, r.w[j + 2] = v.z, r.w[j + 3] = v.w;
        }
    } else {
        float v[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] = first + k < end ? load_gate<BF16>(p, off + first + k) : 0.0f;
        r.set(v);
    }
    return r;
}
template <bool BF16, int K>
__device__ __forceinline__ void store_raw(void *p, int64_t off, int64_t first, int64_t end,
                                          const float (&v)[K])
{
    constexpr int N = Raw<BF16, K>::kWords;
    char *a = static_cast<char *>(p) + (off + first) * (BF16 ? 2 : 4);
    if (first + K <= end) {
        Raw<BF16, K> r;
        r.set(v);
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const Words4 w = {r.w[j], r.w[j + 1], r.w[j + 2], r.w[j + 3]};
            *reinterpret_cast<Words4Any *>(a + 4 * j) = w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (first + k < end) store_gate<BF16>(p, off + first + k, v[k]);
    }
}
// K = 4 or 8 bytes as a bit mask: bit k set where byte first + k is not zero.
template <int K>
__device__ __forceinline__ uint32_t load_flags(const uint8_t *p, int64_t first, int64_t end)
{
    static_assert(K == 4 || K == 8, "one access");
    uint32_t m = 0;
    if (first + K <= end) {
        uint32_t w[K / 4];
        __builtin_memcpy(w, p + first, K);
#pragma unroll
        for (int j = 0; j < K / 4; ++j) {
            // each byte to its 1 or 0, then bytes 0..3 to bits 28..31 (no two
            // products of the multiplication share a bit)
            const uint32_t one = (((w[j] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w[j]) >> 7 & 0x01010101u;
            m |= (one * 0x10204080u >> 28) << (4 * j);
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (first + k < end && p[first + k]) m |= 1u << k;
    }
    return m;
}

}  // namespace pararnn
