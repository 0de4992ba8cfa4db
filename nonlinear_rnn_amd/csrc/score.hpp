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
#include "pararnn.h"

namespace pararnn {

struct ScoreArgs {
    const void *x;
    const int64_t *tokens;
    float *logprob, *entropy, *lse;
    int64_t *top_index;
    float *top_logprob;
    int64_t N, V, stride;
    int32_t top;
    int32_t parts;       // workgroups a row
    float4 *part_stats;  // [N][parts] m, s, w
    uint64_t *part_keys; // [N][parts][top]
    float scale;
    // backward
    const float *lse_in, *entropy_in, *g_logprob, *g_entropy, *g_lse;
    void *dx;
    int64_t dstride;
};

// Unsigned integers in the order of the floats, -0 and +0 alike.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// Keys grow with the logit and, among equals, fall with
// the token; 0 is below every key.
__device__ __forceinline__ uint64_t top_key(float x, uint32_t token)
{
    return ((uint64_t)ordered(x) << 32) | (0xffffffffu - token);
}
__device__ __forceinline__ float key_value(uint64_t k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint32_t key_token(uint64_t k) { return 0xffffffffu - (uint32_t)k; }
// A masked or NaN logit is no alternative.
__device__ __forceinline__ bool may_be_top(float x) { return x > -__builtin_inff(); }

constexpr int kScoreWaves = 4;
constexpr int kScoreThreads = kScoreWaves * kWave;
constexpr int kScoreParts = 32;  // most parts of a row
// Vectors a lane loads before it uses the first.
constexpr int kScoreUnroll = 4;
// The same where it reads again, from wherever the row has gone meanwhile.
constexpr int kScoreAgain = 8;

// Running statistics of part of a row: the largest logit so far and the two
// sums, in base 2: with c = scale log2(e), s = sum 2^(c (x - m)),
// w = sum c (x - m) 2^(c (x - m)).  An empty part has the lowest finite m and
// s = 0, so that joining it changes nothing.
struct Stats {
    float m, s, w;
};
__device__ __forceinline__ Stats no_stats() { return {-__FLT_MAX__, 0.0f, 0.0f}; }
// To another reference m: s and w by 2^(c (m_old - m)); the difference is kept
// finite, since 0 sums must stay 0.
__device__ __forceinline__ void rebase(Stats &a, float m, float c)
{
    const float d = fmaxf(c * (a.m - m), -1e30f);
    const float f = ex2(d);
    a.w = f * fmaf_(a.s, d, a.w);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ Stats join(Stats a, Stats b, float c)
{
    const float m = fmaxf(a.m, b.m);
    rebase(a, m, c);
    rebase(b, m, c);
    return {m, a.s + b.s, a.w + b.w};
}
__device__ __forceinline__ Stats wave_join(Stats a, float c)
{
    float m = a.m;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    rebase(a, m, c);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        a.s += __shfl_xor(a.s, o);
        a.w += __shfl_xor(a.w, o);
    }
    return a;
}
// The two vectors of a lane with the largest logits, and the largest logit of
// all its other ones (the first one's is the statistics' m).
struct BestVectors {
    float second, rest;
    int first_at, second_at;  // -1: none
};
template <int K, bool TOP>
__device__ __forceinline__ void add_stats(Stats &a, BestVectors &v, const float (&x)[K], int at,
                                          float c)
{
    float m = x[0];
#pragma unroll
    for (int k = 1; k < K; ++k) m = fmaxf(m, x[k]);
    if constexpr (TOP) {
        const bool over_first = m > a.m, over_second = m > v.second;
        v.rest = fmaxf(v.rest, fminf(v.second, m));
        v.second_at = over_first ? v.first_at : over_second ? at : v.second_at;
        v.second = over_first ? a.m : over_second ? m : v.second;
        v.first_at = over_first ? at : v.first_at;
    }
    m = fmaxf(a.m, m);
    rebase(a, m, c);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const float d = c * (x[k] - m);
        const float e = ex2(d);  // NaN stays NaN in the sum
        a.s += e;
        a.w = fmaf_(fmaxf(d, -300.0f), e, a.w);  // -inf times 0 would be NaN
    }
}

// A row as 16-byte vectors on their own alignment: vector i holds the
// elements K i - shift .. + K - 1, the first and the last vector possibly in
// part.  What lies outside the row reads as -inf and is not touched.
template <bool BF16>
struct RowView {
    static constexpr int K = BF16 ? 8 : 4;
    const char *row;
    int shift;
    int64_t V, vectors;
    __device__ __forceinline__ RowView(const void *x, int64_t first, int64_t v)
    {
        row = static_cast<const char *>(x) + first * (BF16 ? 2 : 4);
        shift = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / (BF16 ? 2 : 4);
        V = v;
        vectors = V > 0 ? (V + shift + K - 1) / K : 0;
    }
    __device__ __forceinline__ int64_t element(int64_t i) const { return i * K - shift; }
    __device__ __forceinline__ uint4 load_raw(int64_t i) const
    {
        const int64_t j = element(i);
        if (j >= 0 && j + K <= V) return *reinterpret_cast<const uint4 *>(row + j * (BF16 ? 2 : 4));
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (BF16) {
                w[q] = 0xff80u | 0xff800000u;  // -inf twice
                const int64_t e = j + 2 * q;
                if (e >= 0 && e < V)
                    w[q] = (w[q] & 0xffff0000u) | reinterpret_cast<const uint16_t *>(row)[e];
                if (e + 1 >= 0 && e + 1 < V)
                    w[q] = (w[q] & 0xffffu) | (uint32_t)reinterpret_cast<const uint16_t *>(row)[e + 1] << 16;
            } else {
                w[q] = j + q >= 0 && j + q < V ? reinterpret_cast<const uint32_t *>(row)[j + q]
                                               : 0xff800000u;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ void values(const uint4 &v, float (&x)[K])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (BF16) {
                x[2 * q] = __uint_as_float(w[q] << 16);
                x[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
            } else {
                x[q] = __uint_as_float(w[q]);
            }
        }
    }
    __device__ __forceinline__ void load(int64_t i, float (&x)[K]) const { values(load_raw(i), x); }
};

// The best tokens seen by a wave: lane i holds the i-th best key, 0 where
// there is none.
__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane)
{
    return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32) |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, lane);
}
struct TopList {
    uint64_t key, floor;  // floor: what a key has to exceed
    int last;             // the list's last lane
    __device__ __forceinline__ void start(int top, uint64_t f)
    {
        key = 0;
        floor = f;
        last = top - 1;
    }
    // cand: the same in every lane, above the floor
    __device__ __forceinline__ void insert(uint64_t cand)
    {
        const uint32_t hi = dppu<0x138>(~0u, (uint32_t)(key >> 32));  // the lane above
        const uint32_t lo = dppu<0x138>(~0u, (uint32_t)key);
        const uint64_t up = ((uint64_t)hi << 32) | lo;
        if (key < cand) key = up < cand ? up : cand;
        const uint64_t k = lane_key(key, last);
        floor = k > floor ? k : floor;
    }
    // one key a lane, in any order
    __device__ __forceinline__ void offer(uint64_t k)
    {
        uint64_t mask = __ballot(k > floor);
        while (mask) {
            const int l = __ffsll((unsigned long long)mask) - 1;
            insert(lane_key(k, l));
            mask &= mask - 1;
            mask &= __ballot(k > floor);
        }
    }
};
// Every key that is not above this is of a masked token.
constexpr uint64_t kMaskedFloor = 0x007fffffffffffffull;  // ordered(-inf) in the upper half

// How many of n <= PARARNN_TOP_MAX falling keys are above `key`.
__device__ __forceinline__ int keys_above(const uint64_t *list, int n, uint64_t key)
{
    static_assert(PARARNN_TOP_MAX < 128, "the first step");
    int above = 0;
#pragma unroll
    for (int step = 64; step > 0; step >>= 1)
        if (above + step <= n && list[above + step - 1] > key) above += step;
    return above;
}
// Joins `count` lists of `top` falling keys in LDS two by two, between `a` and
// `b`: a key's place is its own index and the number of keys above it in the
// other list (keys 0, behind all others, may meet there: they are equal).
// Returns the buffer with the joined list.
__device__ __forceinline__ uint64_t *join_lists(uint64_t *a, uint64_t *b, int count, int top,
                                                int threads)
{
    for (; count > 1; count = (count + 1) >> 1) {
        __syncthreads();
        for (int t = threadIdx.x; t < count * top; t += threads) {
            const int list = t / top, other = list ^ 1;
            const uint64_t key = a[t];
            int place = t - list * top;
            if (other < count) place += keys_above(a + other * top, top, key);
            if (place < top) b[(list >> 1) * top + place] = key;
        }
        uint64_t *const joined = b;
        b = a;
        a = joined;
    }
    __syncthreads();
    return a;
}

// The results of row n from its statistics.
struct RowScores {
    float base, ls;
    bool empty;
    __device__ __forceinline__ explicit RowScores(const Stats &a)
        : base(a.s == 0.0f ? 0.0f : a.m), ls(a.s == 0.0f ? -__builtin_inff() : logf(a.s)),
          empty(a.s == 0.0f)
    {
    }
};
template <bool BF16>
__device__ __forceinline__ void write_scores(const ScoreArgs &A, int64_t n, const Stats &a)
{
    const RowScores r(a);
    const int64_t t = A.tokens[n];
    float lp = 0.0f;
    if (t >= A.V)
        lp = __builtin_nanf("");
    else if (t >= 0)
        lp = r.empty ? r.ls
                     : fmaf_(A.scale, load_gate<BF16>(A.x, n * A.stride + t) - r.base, -r.ls);
    A.logprob[n] = lp;
    if (A.lse) A.lse[n] = fmaf_(A.scale, r.base, r.ls);
    if (A.entropy) A.entropy[n] = r.empty ? 0.0f : r.ls - 0.6931471805599453f * (a.w / a.s);
}
__device__ __forceinline__ void write_top(const ScoreArgs &A, int64_t n, const RowScores &r, int place,
                                          uint64_t key)
{
    A.top_index[n * A.top + place] = key ? (int64_t)key_token(key) : -1;
    A.top_logprob[n * A.top + place] =
        key ? fmaf_(A.scale, key_value(key) - r.base, -r.ls) : -__builtin_inff();
}

// One workgroup of WAVES waves per row, or per part of a row (PARTS).
// Statistics: every lane keeps its own running maximum and sums over its
// vectors; one pass over the row, joined across lanes and waves at the end.
// Alternatives (TOP): a lane's maximum is the best of its own elements, so the
// top-th best of the lanes' maxima is a lower bound of the top-th best logit.
// Of its vectors a lane remembers the two with the largest logits, and the
// largest logit of the others: only the vectors that reach the bound are read
// again, and a lane goes through all its vectors again only if the others
// reach it.  What reaches it is offered to the wave's list, and the waves'
// lists are joined at the end.
// Bound by HBM: 4096 rows of 50003 bfloat16 with 8 alternatives 89 us (4.6
// TB/s; without alternatives 76, with 64 of rows of random numbers 123, where
// the second reading of vectors shows).  Where rows are few, by latency: 16 rows
// of 65536 float32 with 20 alternatives 16.8 us a call, two launches of 10.2 and
// 5.5 us on the device.
template <bool BF16, int WAVES, bool PARTS, bool TOP>
__global__ void __launch_bounds__(WAVES * kWave) score_kernel(ScoreArgs A)
{
    using Row = RowView<BF16>;
    constexpr int K = Row::K, U = kScoreUnroll, kThreads = WAVES * kWave;
    __shared__ Stats part[WAVES];
    __shared__ float maxima[TOP ? kThreads : 1];
    __shared__ uint64_t lists[2][TOP ? WAVES * PARARNN_TOP_MAX : 1];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int64_t n = PARTS ? blockIdx.x / A.parts : blockIdx.x;
    const int64_t p = PARTS ? blockIdx.x - n * A.parts : 0;
    const float c = A.scale * kLog2e;
    const Row row(A.x, n * A.stride, A.V);
    const int64_t per = PARTS ? (row.vectors + A.parts - 1) / A.parts : row.vectors;
    const int64_t v0 = p * per, v1 = min(row.vectors, v0 + per);

    Stats a = no_stats();
    BestVectors best = {a.m, a.m, -1, -1};
    int64_t i = v0 + threadIdx.x;
    for (; i + (U - 1) * kThreads < v1; i += U * kThreads) {
        float x[U][K];
#pragma unroll
        for (int q = 0; q < U; ++q) row.load(i + q * kThreads, x[q]);
#pragma unroll
        for (int q = 0; q < U; ++q) add_stats<K, TOP>(a, best, x[q], (int)i + q * kThreads, c);
    }
    for (; i < v1; i += kThreads) {
        float x[K];
        row.load(i, x);
        add_stats<K, TOP>(a, best, x, (int)i, c);
    }
    const Stats joined = wave_join(a, c);
    if (lane == 0) part[wave] = joined;
    if constexpr (TOP) maxima[threadIdx.x] = a.m;
    __syncthreads();
    [[maybe_unused]] TopList list;
    if constexpr (TOP) {
        // the top-th best maximum, rounded down to 16 bits of its order
        uint32_t o[WAVES], bound = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) o[w] = ordered(maxima[w * kWave + lane]);
        for (int bit = 31; bit >= 16; --bit) {
            const uint32_t trial = bound | 1u << bit;
            int count = 0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) count += __popcll(__ballot(o[w] >= trial));
            if (count >= A.top) bound = trial;
        }
        const uint64_t low = bound ? ((uint64_t)bound << 32) - 1 : 0;
        list.start(A.top, low > kMaskedFloor ? low : kMaskedFloor);
        const auto offer = [&](const uint4 &raw, int64_t vector) {
            float x[K], m = -__builtin_inff();
            Row::values(raw, x);
#pragma unroll
            for (int k = 0; k < K; ++k) m = fmaxf(m, x[k]);
            if (!__ballot(ordered(m) >= (uint32_t)(list.floor >> 32))) return;
            const int64_t e = row.element(vector);
#pragma unroll
            for (int k = 0; k < K; ++k)
                list.offer(may_be_top(x[k]) ? top_key(x[k], (uint32_t)(e + k)) : 0);
        };
        const uint4 none = make_uint4(~0u, ~0u, ~0u, ~0u);  // NaN: no alternative
        uint4 raw[2] = {none, none};
        if (best.first_at >= 0 && ordered(a.m) >= bound) raw[0] = row.load_raw(best.first_at);
        if (best.second_at >= 0 && ordered(best.second) >= bound) raw[1] = row.load_raw(best.second_at);
        offer(raw[0], best.first_at);
        offer(raw[1], best.second_at);
        const bool again = ordered(best.rest) >= bound;
        if (__ballot(again))
            for (int64_t j = v0 + threadIdx.x; __ballot(j < v1); j += kScoreAgain * kThreads) {
                uint4 more[kScoreAgain];
#pragma unroll
                for (int q = 0; q < kScoreAgain; ++q) {
                    const int64_t jq = j + q * kThreads;
                    more[q] = none;
                    if (again && jq < v1 && jq != best.first_at && jq != best.second_at)
                        more[q] = row.load_raw(jq);
                }
#pragma unroll
                for (int q = 0; q < kScoreAgain; ++q) offer(more[q], j + q * kThreads);
            }
    }
    // the workgroup's statistics, in every thread
    a = part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) a = join(a, part[w], c);
    if constexpr (PARTS) {
        if (threadIdx.x == 0) A.part_stats[blockIdx.x] = make_float4(a.m, a.s, a.w, 0.0f);
    } else {
        if (threadIdx.x == 0) write_scores<BF16>(A, n, a);
    }
    if constexpr (!TOP) return;
    [[maybe_unused]] const RowScores scores(a);
    [[maybe_unused]] const auto put = [&](int place, uint64_t key) {
        if constexpr (PARTS)
            A.part_keys[(int64_t)blockIdx.x * A.top + place] = key;
        else
            write_top(A, n, scores, place, key);
    };
    if constexpr (TOP && WAVES == 1) {
        if (lane < A.top) put(lane, list.key);
    } else if constexpr (TOP) {
        if (lane < A.top) lists[0][wave * A.top + lane] = list.key;
        const uint64_t *joined = join_lists(lists[0], lists[1], WAVES, A.top, kThreads);
        if (threadIdx.x < A.top) put(threadIdx.x, joined[threadIdx.x]);
    }
}

// A workgroup per row joins its parts: one wave the statistics, all of them the
// lists, two by two in LDS (a search through every list for each place took
// longer than reading the row).  Bound by latency.
constexpr int kJoinThreads = 256;
template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) score_join_kernel(ScoreArgs A)
{
    __shared__ uint64_t lists[2][kScoreParts * PARARNN_TOP_MAX];
    const int64_t n = blockIdx.x, first = n * A.parts;
    const int lane = threadIdx.x % kWave;
    for (int t = threadIdx.x; t < A.parts * A.top; t += kJoinThreads)
        lists[0][t] = A.part_keys[first * A.top + t];
    Stats a = no_stats();
    if (lane < A.parts) {
        const float4 v = A.part_stats[first + lane];
        a = {v.x, v.y, v.z};
    }
    a = wave_join(a, A.scale * kLog2e);
    if (threadIdx.x == 0) write_scores<BF16>(A, n, a);
    if (!A.top) return;
    const uint64_t *joined = join_lists(lists[0], lists[1], A.parts, A.top, kJoinThreads);
    if (threadIdx.x < A.top) write_top(A, n, RowScores(a), threadIdx.x, joined[threadIdx.x]);
}

// The gradient: U vectors a lane, a workgroup per kThreads * U vectors of a row,
// all loads issued before the first is used.  Reads a logit and writes one,
// rounded once when it is stored.  Bound by HBM: 8192 rows of 32000 bfloat16
// 202 us (5.2 TB/s), 1000 of 100003 float32, each row on its own alignment, 148
// us (5.4 TB/s).
template <bool BF16>
__global__ void __launch_bounds__(kScoreThreads) score_adjoint_kernel(ScoreArgs A)
{
    using Row = RowView<BF16>;
    constexpr int K = Row::K, U = kScoreUnroll;
    const int64_t n = blockIdx.x / A.parts;
    const Row row(A.x, n * A.stride, A.V);
    const int64_t i = (blockIdx.x - n * A.parts) * (U * kScoreThreads) + threadIdx.x;
    float x[U][K];
#pragma unroll
    for (int q = 0; q < U; ++q)
        if (i + q * kScoreThreads < row.vectors) row.load(i + q * kScoreThreads, x[q]);
    const float lse = A.lse_in[n], H = A.entropy_in ? A.entropy_in[n] : 0.0f;
    const int64_t t = A.tokens[n];
    const float glp = A.g_logprob && t >= 0 ? A.g_logprob[n] : 0.0f;
    const float gh = A.g_entropy ? A.g_entropy[n] : 0.0f;
    const float c0 = (A.g_lse ? A.g_lse[n] : 0.0f) - glp;
    const bool empty = lse == -__builtin_inff();
#pragma unroll
    for (int q = 0; q < U; ++q) {
        if (i + q * kScoreThreads >= row.vectors) break;
        const int64_t e = row.element(i + q * kScoreThreads);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float lp = fmaf_(A.scale, x[q][k], -lse);
            const float p = empty ? 0.0f : ex2(kLog2e * lp);
            // p lp -> 0 as p -> 0
            float g = p == 0.0f ? 0.0f : p * fmaf_(-gh, lp + H, c0);
            if (e + k == t && !empty) g += glp;
            x[q][k] = A.scale * g;
        }
        if (e >= 0) {
            store_raw<BF16, K>(A.dx, n * A.dstride, e, A.V, x[q]);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (e + k >= 0 && e + k < A.V) store_gate<BF16>(A.dx, n * A.dstride + e + k, x[q][k]);
        }
    }
}

}  // namespace pararnn
