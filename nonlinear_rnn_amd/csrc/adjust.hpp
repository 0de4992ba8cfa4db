// What is done to logits before a token is sampled from them.  Per row and
// token j, with c_j how often the row's history holds it behind its prompt:
//     x <- x / repetition where x > 0, x repetition elsewhere   (j in the history)
//     x <- x - frequency c_j - presence                         (c_j > 0)
//     x <- x + bias_j                                           (j in the row's list)
//     x <- -inf                                                 (j not allowed)
// in float32, rounded once.
#pragma once

#include "score.hpp"

namespace pararnn {
namespace adjust {

constexpr int kThreads = 256;
constexpr int kTokens = 8192;  // of a row, a workgroup
constexpr int kAtOnce = 8;     // tokens of the history that a thread has under way

struct Args {
    const void *x;
    void *out;
    int64_t N, V, stride, out_stride;
    int32_t parts;
    const int64_t *tokens;
    int64_t token_stride, length;
    const int32_t *lengths, *prompt;
    const float *repetition, *presence, *frequency;
    const int64_t *bias_index;
    const float *bias_value;
    int64_t biases;
    const uint32_t *allowed;
    int64_t allowed_stride, allowed_count;
    const int32_t *allowed_rows;
};

constexpr uint32_t kSeen = 0x80000000u;  // in the prompt; the lower bits count it behind

// A workgroup for a part of a row.  It goes through the row's whole history and
// counts in LDS what falls into its part (integers: in any order); of a token's
// entries in the bias list the last is kept.  Its phases wait for one another: the
// counts are cleared, then the history is read, and only behind it the logits, which
// nothing has under way.  512 rows of 100003 bfloat16, histories of 6000: 95 us, 2.5
// TB/s, half of it with vector instructions, waves waiting for 53% of their time (one
// token at a time 107 us instead of 87; parts of 16384 by 512 threads 89).  16 rows of
// 65536 float32, 144 workgroups: 12.5 us, waiting for 65%.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) adjust_kernel(Args A)
{
    using Row = RowView<BF16>;
    constexpr int K = Row::K, kVectors = kTokens / K;
    __shared__ uint4 counts4[kTokens / 4];
    uint32_t *const counts = reinterpret_cast<uint32_t *>(counts4);
    extern __shared__ uint4 entries4[];  // 1 + a token's last place in the list; only where there is one
    uint32_t *const entries = reinterpret_cast<uint32_t *>(entries4);
    const int64_t n = blockIdx.x / A.parts;
    const Row row(A.x, n * A.stride, A.V);
    const int64_t first = (blockIdx.x - n * A.parts) * kVectors, base = row.element(first);
    int64_t length = 0, prompt = 0;
    if (A.tokens) {
        length = A.lengths ? min((int64_t)max(A.lengths[n], 0), A.length) : A.length;
        prompt = A.prompt ? A.prompt[n] : 0;
    }
    const bool counted = length > 0, listed = A.biases > 0;
    for (int i = threadIdx.x; i < kTokens / 4; i += kThreads) {
        if (counted) counts4[i] = make_uint4(0, 0, 0, 0);
        if (listed) entries4[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    // the part's tokens: `skip` places of its first vector belong to the row before
    const int skip = base < 0 ? (int)-base : 0;
    const uint64_t tokens = (uint64_t)max((int64_t)0, min(A.V - base, (int64_t)kTokens) - skip);
    const auto place = [&](int64_t j) {  // in the part, or -1
        const uint64_t at = (uint64_t)j - (uint64_t)(base + skip);
        return at < tokens ? (int)at + skip : -1;
    };
    for (int64_t i0 = threadIdx.x; i0 < length; i0 += kAtOnce * kThreads) {
        int64_t token[kAtOnce];
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s)
            token[s] = A.tokens[n * A.token_stride + min(i0 + s * kThreads, length - 1)];
#pragma unroll
        for (int s = 0; s < kAtOnce; ++s) {
            const int64_t i = i0 + s * kThreads;
            const int at = place(token[s]);
            if (at < 0 || i >= length) continue;
            if (i >= prompt)
                atomicAdd(&counts[at], 1u);
            else
                atomicOr(&counts[at], kSeen);
        }
    }
    for (int64_t i = threadIdx.x; i < A.biases; i += kThreads) {
        const int at = place(A.bias_index[n * A.biases + i]);
        if (at >= 0) atomicMax(&entries[at], (uint32_t)i + 1);
    }
    __syncthreads();
    const float rep = A.repetition ? A.repetition[n] : 1.0f;
    const float presence = A.presence ? A.presence[n] : 0.0f, frequency = A.frequency ? A.frequency[n] : 0.0f;
    const uint32_t *allowed = nullptr;
    if (A.allowed) {
        const int64_t r = A.allowed_rows ? A.allowed_rows[n] : n;
        if (r >= 0 && r < A.allowed_count) allowed = A.allowed + r * A.allowed_stride;
    }
    for (int v = threadIdx.x; v < kVectors && first + v < row.vectors; v += kThreads) {
        float x[K];
        row.load(first + v, x);
        const int64_t e = row.element(first + v);
        uint32_t bits = ~0u;
        if (allowed) {
            const int64_t lo = e < 0 ? 0 : e, hi = min(e + K, A.V) - 1;
            const uint64_t two = (uint64_t)allowed[hi >> 5] << 32 | allowed[lo >> 5];
            const uint32_t from = (lo >> 5) == (hi >> 5) ? allowed[lo >> 5] >> (lo & 31) : (uint32_t)(two >> (lo & 31));
            bits = from << (lo - e);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const uint32_t count = counted ? counts[v * K + k] : 0;
            if (count) {
                x[k] = x[k] > 0.0f ? x[k] / rep : x[k] * rep;
                if (count & ~kSeen) x[k] -= fmaf_(frequency, (float)(count & ~kSeen), presence);
            }
            const uint32_t entry = listed ? entries[v * K + k] : 0;
            if (entry) x[k] += A.bias_value[n * A.biases + entry - 1];
            if (!(bits >> k & 1)) x[k] = -__builtin_inff();
        }
        if (e >= 0) {
            store_raw<BF16, K>(A.out, n * A.out_stride, e, A.V, x);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (e + k >= 0 && e + k < A.V) store_gate<BF16>(A.out, n * A.out_stride + e + k, x[k]);
        }
    }
}

}  // namespace adjust
}  // namespace pararnn
