// One step of the gated delta rule for many requests, their states in a pool.
// Per request and head, with S [dk][dv] the slot's state,
//     S <- a S,   w = beta (v - k^T S),   S <- S + k w^T,   o = scale q^T S.
#pragma once

#include "elements.hpp"
#include "pararnn.h"

namespace pararnn {
namespace delta {

constexpr float kForget = -104.0f;  // exp of less is 0 in float32

struct StepArgs {
    const void *q, *k, *v;
    int64_t q_b, q_h, q_d, k_b, k_h, k_d, v_b, v_h, v_d, o_b, o_h, o_d, gate_b, gate_h;
    const float *beta, *decay;
    const int32_t *slots;
    float *states, *o;
    int64_t B, pool;
    int32_t Hk, Hv, key, value, blocks;
    float scale;
};

constexpr int kStepThreads = 256, kStepColumns = 64, kStepRows = kStepThreads / (kStepColumns / 4);

// Sums x over the 16 threads that hold the same columns, in a fixed order; the
// result in all of them.
__device__ __forceinline__ float4 sum_rows(float4 x, float4 (&part)[kStepThreads / kWave][kStepColumns / 4])
{
    const int wave = threadIdx.x / kWave, c = threadIdx.x % 16;
#pragma unroll
    for (int o = 16; o < kWave; o *= 2) {
        x.x += __shfl_xor(x.x, o);
        x.y += __shfl_xor(x.y, o);
        x.z += __shfl_xor(x.z, o);
        x.w += __shfl_xor(x.w, o);
    }
    if (threadIdx.x % kWave < 16) part[wave][c] = x;
    __syncthreads();
    x = part[0][c];
#pragma unroll
    for (int w = 1; w < kStepThreads / kWave; ++w) {
        x.x += part[w][c].x;
        x.y += part[w][c].y;
        x.z += part[w][c].z;
        x.w += part[w][c].w;
    }
    return x;
}

// A workgroup for a request's head and 64 columns of its state, which is read
// and written once: 16 threads side by side along a row, R rows each, 16 apart.
// Bound by HBM where there are many requests, else by latency: 256 requests of 16
// heads of 128 x 128, 537 MB: 115 us, 4.7 TB/s (86 us where the last call's states
// are still in the cache); 4 of 4 heads of 64 x 64: 4.7 us.
template <bool HALF, int R>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(StepArgs A)
{
    __shared__ float ks[R * kStepRows], qs[R * kStepRows];
    __shared__ float4 part[2][kStepThreads / kWave][kStepColumns / 4];
    const int64_t row = blockIdx.x / A.blocks, b = row / A.Hv, h = row % A.Hv, hk = h / (A.Hv / A.Hk);
    const int v0 = (int)(blockIdx.x % A.blocks) * kStepColumns + threadIdx.x % 16 * 4, d0 = threadIdx.x / 16;
    const int64_t slot = A.slots ? A.slots[b] : b;
    const bool live = slot >= 0 && slot < A.pool;
    const int left = A.value - v0;  // columns from the thread's first on
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (live) {
        float *const S = A.states + (slot * A.Hv + h) * A.key * A.value;
        float4 s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int d = d0 + r * kStepRows;
            s[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (d >= A.key) continue;
            const float *p = S + (int64_t)d * A.value + v0;
            if (left >= 4) {
                const Words4 w = *reinterpret_cast<const Words4Any *>(p);
                s[r] = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                                   __uint_as_float(w.w));
            } else {
                if (left > 0) s[r].x = p[0];
                if (left > 1) s[r].y = p[1];
                if (left > 2) s[r].z = p[2];
            }
        }
        for (int d = threadIdx.x; d < R * kStepRows; d += kStepThreads) {
            ks[d] = d < A.key ? load_gate<HALF>(A.k, b * A.k_b + hk * A.k_h + d * A.k_d) : 0.0f;
            qs[d] = d < A.key ? load_gate<HALF>(A.q, b * A.q_b + hk * A.q_h + d * A.q_d) : 0.0f;
        }
        float4 v = o;
        const int64_t v_at = b * A.v_b + h * A.v_h + v0 * A.v_d;
        if (left > 0) v.x = load_gate<HALF>(A.v, v_at);
        if (left > 1) v.y = load_gate<HALF>(A.v, v_at + A.v_d);
        if (left > 2) v.z = load_gate<HALF>(A.v, v_at + 2 * A.v_d);
        if (left > 3) v.w = load_gate<HALF>(A.v, v_at + 3 * A.v_d);
        const float beta = A.beta[b * A.gate_b + h * A.gate_h];
        const float g = A.decay ? A.decay[b * A.gate_b + h * A.gate_h] : 0.0f;
        const bool forget = g < kForget;  // keeps nothing, also of what is not finite
        const float a = expf(g);
        __syncthreads();
        float4 sum = o;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float k = ks[d0 + r * kStepRows];
            s[r].x = forget ? 0.0f : a * s[r].x;
            s[r].y = forget ? 0.0f : a * s[r].y;
            s[r].z = forget ? 0.0f : a * s[r].z;
            s[r].w = forget ? 0.0f : a * s[r].w;
            sum.x = fmaf_(k, s[r].x, sum.x);
            sum.y = fmaf_(k, s[r].y, sum.y);
            sum.z = fmaf_(k, s[r].z, sum.z);
            sum.w = fmaf_(k, s[r].w, sum.w);
        }
        sum = sum_rows(sum, part[0]);
        const float4 w = make_float4(beta * (v.x - sum.x), beta * (v.y - sum.y), beta * (v.z - sum.z),
                                     beta * (v.w - sum.w));
        sum = o;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int d = d0 + r * kStepRows;
            const float k = ks[d], q = qs[d];
            s[r].x = fmaf_(k, w.x, s[r].x);
            s[r].y = fmaf_(k, w.y, s[r].y);
            s[r].z = fmaf_(k, w.z, s[r].z);
            s[r].w = fmaf_(k, w.w, s[r].w);
            sum.x = fmaf_(q, s[r].x, sum.x);
            sum.y = fmaf_(q, s[r].y, sum.y);
            sum.z = fmaf_(q, s[r].z, sum.z);
            sum.w = fmaf_(q, s[r].w, sum.w);
            if (d >= A.key) continue;
            float *p = S + (int64_t)d * A.value + v0;
            if (left >= 4) {
                const Words4 out = {__float_as_uint(s[r].x), __float_as_uint(s[r].y), __float_as_uint(s[r].z),
                                    __float_as_uint(s[r].w)};
                *reinterpret_cast<Words4Any *>(p) = out;
            } else {
                if (left > 0) p[0] = s[r].x;
                if (left > 1) p[1] = s[r].y;
                if (left > 2) p[2] = s[r].z;
            }
        }
        o = sum_rows(sum, part[1]);
    }
    if (threadIdx.x < 16) {
        float *p = A.o + b * A.o_b + h * A.o_h + v0 * A.o_d;
        if (left > 0) p[0] = A.scale * o.x;
        if (left > 1) p[A.o_d] = A.scale * o.y;
        if (left > 2) p[2 * A.o_d] = A.scale * o.z;
        if (left > 3) p[3 * A.o_d] = A.scale * o.w;
    }
}

}  // namespace delta
}  // namespace pararnn
