// Scores of given tokens: log probability, entropy, log of the sum of
// exponentials and the most likely tokens of each row of logits, and the
// gradient for the logits.  With m the largest logit of a row and
// d_j = scale (x_j - m),
//     s = sum exp(d_j),  w = sum d_j exp(d_j),
//     lse = scale m + log s,  logprob = d_token - log s,  entropy = log s - w / s.
// A masked logit (-inf) adds nothing to either sum.  Sums and statistics are
// float32.
//
// Alternatives are ordered by the logits themselves, not by the rounded log
// probabilities: a key of 64 bits, the logit's order in the upper half and
// the token's distance from the end in the lower one, makes every order
// strict, so equal logits go lowest token first whatever the work split.
#pragma once

#include "elements.hpp"

namespace pararnn {

struct ScoreArgs {
    const void *x;
    const int64_t *tokens;
    float *logprob, *entropy, *lse;
    int64_t *top_index;
    float *top_logprob;
    int64_t N, V, stride;
    int32_t top;
    float scale;
    // backward
    const float *lse_in, *entropy_in, *g_logprob, *g_entropy, *g_lse;
    void *dx;
    int64_t dstride;
};

// Keys grow with the logit (-0 and +0 alike) and, among equals, fall with
// the token; 0 is below every key.
__device__ __forceinline__ uint64_t top_key(float x, uint32_t token)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return ((uint64_t)o << 32) | (0xffffffffu - token);
}
__device__ __forceinline__ float key_value(uint64_t k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint32_t key_token(uint64_t k) { return 0xffffffffu - (uint32_t)k; }
// A masked or NaN logit is no alternative.
__device__ __forceinline__ bool may_be_top(float x) { return x > -__builtin_inff(); }

constexpr int kScoreThreads = 256;
constexpr int kScoreWaves = kScoreThreads / kWave;

__device__ __forceinline__ float wave_max(float v)
{
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float wave_sum(float v)
{
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// One workgroup per row: a pass for the maximum, one for the sums, and one
// for each alternative.
template <bool BF16>
__global__ void __launch_bounds__(kScoreThreads) score_row_kernel(ScoreArgs A)
{
    __shared__ float part[3][kScoreWaves];
    __shared__ uint64_t best[kScoreWaves];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    for (int64_t n = blockIdx.x; n < A.N; n += gridDim.x) {
        const int64_t row = n * A.stride;
        float m = -__builtin_inff();
        for (int64_t j = threadIdx.x; j < A.V; j += kScoreThreads)
            m = fmaxf(m, load_gate<BF16>(A.x, row + j));
        m = wave_max(m);
        __syncthreads();
        if (lane == 0) part[0][wave] = m;
        __syncthreads();
        for (int w = 0; w < kScoreWaves; ++w) m = fmaxf(m, part[0][w]);
        const float base = m > -__builtin_inff() ? m : 0.0f;
        float s = 0.0f, ws = 0.0f;
        for (int64_t j = threadIdx.x; j < A.V; j += kScoreThreads) {
            const float d = A.scale * (load_gate<BF16>(A.x, row + j) - base);
            const float e = ex2(kLog2e * d);
            s += e;
            if (e > 0.0f) ws = fmaf_(e, d, ws);
        }
        s = wave_sum(s);
        ws = wave_sum(ws);
        if (lane == 0) part[1][wave] = s, part[2][wave] = ws;
        __syncthreads();
        s = ws = 0.0f;
        for (int w = 0; w < kScoreWaves; ++w) s += part[1][w], ws += part[2][w];
        const bool empty = s == 0.0f;
        const float ls = empty ? -__builtin_inff() : logf(s);
        if (threadIdx.x == 0) {
            const int64_t t = A.tokens[n];
            float lp = 0.0f;
            if (t >= A.V)
                lp = __builtin_nanf("");
            else if (t >= 0)
                lp = empty ? ls : A.scale * (load_gate<BF16>(A.x, row + t) - base) - ls;
            A.logprob[n] = lp;
            if (A.lse) A.lse[n] = fmaf_(A.scale, base, ls);
            if (A.entropy) A.entropy[n] = empty ? 0.0f : ls - ws / s;
        }
        uint64_t last = ~0ull;
        for (int k = 0; k < A.top; ++k) {
            uint64_t key = 0;
            if (last)
                for (int64_t j = threadIdx.x; j < A.V; j += kScoreThreads) {
                    const float x = load_gate<BF16>(A.x, row + j);
                    const uint64_t c = may_be_top(x) ? top_key(x, (uint32_t)j) : 0;
                    if (c < last && c > key) key = c;
                }
            for (int o = 32; o > 0; o >>= 1) {
                const uint64_t c = __shfl_xor(key, o);
                if (c > key) key = c;
            }
            __syncthreads();
            if (lane == 0) best[wave] = key;
            __syncthreads();
            for (int w = 0; w < kScoreWaves; ++w)
                if (best[w] > key) key = best[w];
            last = key;
            if (threadIdx.x == 0) {
                A.top_index[n * A.top + k] = key ? (int64_t)key_token(key) : -1;
                A.top_logprob[n * A.top + k] =
                    key ? A.scale * (key_value(key) - base) - ls : -__builtin_inff();
            }
        }
    }
}

// The gradient, a workgroup per row.
template <bool BF16>
__global__ void __launch_bounds__(kScoreThreads) score_adjoint_kernel(ScoreArgs A)
{
    for (int64_t n = blockIdx.x; n < A.N; n += gridDim.x) {
        const int64_t row = n * A.stride, out = n * A.dstride;
        const float lse = A.lse_in[n], H = A.entropy_in ? A.entropy_in[n] : 0.0f;
        const int64_t t = A.tokens[n];
        const float glp = A.g_logprob && t >= 0 ? A.g_logprob[n] : 0.0f;
        const float gh = A.g_entropy ? A.g_entropy[n] : 0.0f;
        const float c0 = (A.g_lse ? A.g_lse[n] : 0.0f) - glp;
        const bool empty = lse == -__builtin_inff();
        for (int64_t j = threadIdx.x; j < A.V; j += kScoreThreads) {
            const float lp = fmaf_(A.scale, load_gate<BF16>(A.x, row + j), -lse);
            const float p = empty ? 0.0f : ex2(kLog2e * lp);
            float g = p == 0.0f ? 0.0f : p * fmaf_(-gh, lp + H, c0);
            if (j == t && !empty) g += glp;
            store_gate<BF16>(A.dx, out + j, A.scale * g);
        }
    }
}

}  // namespace pararnn
