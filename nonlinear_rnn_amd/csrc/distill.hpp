// Distillation from a teacher's most likely tokens: per row, with p_e the
// teacher's probabilities of the listed tokens j_e, r = 1 - sum p_e what they
// leave, and q = softmax(scale x) the student's probabilities,
//     loss = sum_e p_e (log p_e - log q_{j_e}) + r (log r - log q_rest),
// q_rest the sum of q over the tokens that are not listed (without `tail` the
// second term is left out).  The gradient for the student's logits is
//     scale (q_j (P + r) - p_j)                 for listed tokens, P = sum p_e,
//     scale q_j (P + r - r / q_rest)            for the others.
// q_rest is summed over the tokens themselves: as 1 - sum q_{j_e} it would be
// lost where the student agrees with the teacher.  q_j / q_rest is one
// exponential, a share of r however small the two are.  Where lse or log q_rest
// are too large to hold the sums that they come from, the gradient sums again.
// Sums are float32 relative to a running maximum; those of the short list float64.
#pragma once

#include "score.hpp"

namespace pararnn {
namespace distill {

constexpr int kWaves = 4, kThreads = kWaves * kWave;
constexpr int kParts = 32;              // most parts of a row
constexpr int kSection = 16384;         // vectors whose listed elements are marked at once
constexpr int kMost = PARARNN_DISTILL_MAX, kEach = (kMost + kThreads - 1) / kThreads;
constexpr int kSectionAgain = 2048;     // the same in the gradient
constexpr float kRest = 1e-6f;          // a smaller r is what rounding left of the list
// A log q_rest below leaves its tokens' shares to their own largest logit and sum:
// as a float32 it holds them within 2^-24 of its size, 4e-6 here, and where a mask of
// -1e9 made it, not at all.
constexpr float kFar = -64.0f;
// The same for q and an lse beyond: 6e-5 here, and a row that a finite mask left
// nothing of loses its log V.
constexpr float kLarge = 1024.0f;

struct Args {
    const void *x;
    const int64_t *index;
    const float *logprob;
    int64_t N, V, stride;
    int32_t count, parts, tail;
    float scale;
    float *loss, *lse, *log_rest;
    float2 *part_stats;  // [N][parts]
    // backward
    const float *lse_in, *log_rest_in, *g_loss;
    void *dx;
    int64_t dstride;
};

// The largest element and the sum of 2^(c (x - m)); an empty part has the
// lowest finite m and s = 0.
struct Sum {
    float m, s;
};
__device__ __forceinline__ Sum no_sum() { return {-__FLT_MAX__, 0.0f}; }
__device__ __forceinline__ void rebase(Sum &a, float m, float c)
{
    a.s *= ex2(fmaxf(c * (a.m - m), -1e30f));  // finite: 0 stays 0
    a.m = m;
}
__device__ __forceinline__ Sum join(Sum a, Sum b, float c)
{
    const float m = fmaxf(a.m, b.m);
    rebase(a, m, c);
    rebase(b, m, c);
    return {m, a.s + b.s};
}
// Of all threads of the workgroup, in every thread, joined in a fixed order.
__device__ __forceinline__ Sum join_all(Sum a, float c, Sum (&part)[kWaves])
{
    float m = a.m;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    rebase(a, m, c);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) a.s += __shfl_xor(a.s, o);
    __syncthreads();
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = a;
    __syncthreads();
    a = part[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) a = join(a, part[w], c);
    return a;
}
__device__ __forceinline__ double add_all(double x, double (&part)[kWaves])
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    __syncthreads();
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) x += part[w];
    return x;
}

struct Shared {
    Sum sums[kWaves];
    double adds[kWaves];
    int64_t list[kMost];
};
// The row's list to LDS; an unused entry is -1.
__device__ __forceinline__ void load_list(const Args &A, int64_t n, Shared &sh)
{
    for (int e = threadIdx.x; e < A.count; e += kThreads) {
        const int64_t j = A.index[n * A.count + e];
        sh.list[e] = j < 0 ? -1 : j;
    }
}
// Whether no entry before e names the same token.
__device__ __forceinline__ bool leads(const Shared &sh, int e)
{
    for (int i = 0; i < e; ++i)
        if (sh.list[i] == sh.list[e]) return false;
    return true;
}
// A thread's sum over the listed tokens.
template <bool BF16>
__device__ __forceinline__ Sum listed_of(const Args &A, int64_t n, const Shared &sh)
{
    const float c = A.scale * kLog2e;
    Sum all = no_sum();
    for (int e = threadIdx.x; e < A.count; e += kThreads) {
        const int64_t j = sh.list[e];
        if (j < 0 || j >= A.V || !leads(sh, e)) continue;
        const float x = load_gate<BF16>(A.x, n * A.stride + j);
        Sum one = {fmaxf(x, -__FLT_MAX__), x == -__builtin_inff() ? 0.0f : 1.0f};
        if (!(x < __builtin_inff())) one.s = __builtin_nanf("");  // as in the other tokens' sum
        all = join(all, one, c);
    }
    return all;
}
// The row's results from the sum over the tokens that are not listed.
template <bool BF16>
__device__ __forceinline__ void finish(const Args &A, int64_t n, Sum rest, Shared &sh)
{
    const float c = A.scale * kLog2e;
    bool past = false, any = false;
    for (int e = threadIdx.x; e < A.count; e += kThreads) {
        any |= sh.list[e] >= 0;
        past |= sh.list[e] >= A.V;
    }
    const Sum all = join(join_all(listed_of<BF16>(A, n, sh), c, sh.sums), rest, c);
    const bool empty = all.s == 0.0f;
    const float ls = logf(all.s);
    const float lse = empty ? -__builtin_inff() : fmaf_(A.scale, all.m, ls);
    const float log_rest = rest.s == 0.0f ? -__builtin_inff() : fmaf_(A.scale, rest.m - all.m, logf(rest.s) - ls);
    double P = 0.0, loss = 0.0;
    for (int e = threadIdx.x; e < A.count; e += kThreads) {
        const int64_t j = sh.list[e];
        if (j < 0 || j >= A.V) continue;
        const float lp = A.logprob[n * A.count + e], p = expf(lp);
        const float x = load_gate<BF16>(A.x, n * A.stride + j);
        const float lq = empty || x == -__builtin_inff() ? -__builtin_inff() : fmaf_(A.scale, x - all.m, -ls);
        P += p;
        if (p != 0.0f) loss += (double)p * ((double)lp - lq);
    }
    P = add_all(P, sh.adds);
    loss = add_all(loss, sh.adds);
    if (A.tail) {
        const float r = (float)(1.0 - P);
        if (!(r < kRest)) loss += (double)r * ((double)logf(r) - log_rest);
    }
    past = __syncthreads_or(past);
    any = __syncthreads_or(any);
    if (threadIdx.x == 0) {
        A.loss[n] = past ? __builtin_nanf("") : any ? (float)loss : 0.0f;
        A.lse[n] = lse;
        A.log_rest[n] = log_rest;
    }
}

// Marks the listed tokens of vectors s0 .. s1 - 1 of the row, a byte for each vector.
template <bool BF16, int SECTION>
__device__ __forceinline__ void mark_listed(const Args &A, const RowView<BF16> &row, int64_t s0, int64_t s1,
                                            const Shared &sh, uint32_t (&marks)[SECTION / 4])
{
    constexpr int K = RowView<BF16>::K;
    __syncthreads();
    for (int i = threadIdx.x; i < (int)((s1 - s0 + 3) / 4); i += kThreads) marks[i] = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < A.count; e += kThreads) {
        const int64_t j = sh.list[e] + row.shift, at = j / K - s0;
        if (sh.list[e] >= 0 && sh.list[e] < A.V && at >= 0 && at < s1 - s0)
            atomicOr(&marks[at / 4], 1u << (8 * (at % 4) + j % K));
    }
    __syncthreads();
}
// Adds a vector's tokens but the marked ones.
template <int K>
__device__ __forceinline__ void add_unmarked(Sum &a, float (&x)[K], uint32_t mark, float c)
{
    float m = a.m;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (mark >> k & 1) x[k] = -__builtin_inff();
        m = fmaxf(m, x[k]);
    }
    rebase(a, m, c);
#pragma unroll
    for (int k = 0; k < K; ++k) a.s += ex2(c * (x[k] - m));
}

// A workgroup per row, or per part of a row (PARTS) where there are few.  The
// listed tokens are left out of the sum and join it at the end.  Bound by HBM: 4096
// rows of 50003 bfloat16 90 us a call, 4.6 TB/s, float32 153 us, 5.3 TB/s.
template <bool BF16, bool PARTS>
__global__ void __launch_bounds__(kThreads) distill_kernel(Args A)
{
    using Row = RowView<BF16>;
    constexpr int K = Row::K, U = kScoreUnroll;
    __shared__ Shared sh;
    __shared__ uint32_t marks[kSection / 4];
    const int64_t n = PARTS ? blockIdx.x / A.parts : blockIdx.x;
    const int64_t p = PARTS ? blockIdx.x - n * A.parts : 0;
    const float c = A.scale * kLog2e;
    const Row row(A.x, n * A.stride, A.V);
    const int64_t per = PARTS ? (row.vectors + A.parts - 1) / A.parts : row.vectors;
    const int64_t v0 = p * per, v1 = min(row.vectors, v0 + per);
    load_list(A, n, sh);

    Sum a = no_sum();
    for (int64_t s0 = v0; s0 < v1; s0 += kSection) {
        const int64_t s1 = min(v1, s0 + kSection);
        mark_listed<BF16, kSection>(A, row, s0, s1, sh, marks);
        const auto mark = [&](int64_t i) { return marks[(i - s0) / 4] >> (8 * ((i - s0) % 4)) & 0xffu; };
        int64_t i = s0 + threadIdx.x;
        for (; i + (U - 1) * kThreads < s1; i += U * kThreads) {
            float x[U][K];
#pragma unroll
            for (int q = 0; q < U; ++q) row.load(i + q * kThreads, x[q]);
#pragma unroll
            for (int q = 0; q < U; ++q) add_unmarked(a, x[q], mark(i + q * kThreads), c);
        }
        for (; i < s1; i += kThreads) {
            float x[K];
            row.load(i, x);
            add_unmarked(a, x, mark(i), c);
        }
    }
    a = join_all(a, c, sh.sums);
    if constexpr (PARTS) {
        if (threadIdx.x == 0) A.part_stats[blockIdx.x] = make_float2(a.m, a.s);
    } else {
        finish<BF16>(A, n, a, sh);
    }
}
template <bool BF16>
__global__ void __launch_bounds__(kThreads) distill_join_kernel(Args A)
{
    __shared__ Shared sh;
    const int64_t n = blockIdx.x;
    load_list(A, n, sh);
    Sum a = no_sum();
    if ((int)threadIdx.x < A.parts) {
        const float2 v = A.part_stats[n * A.parts + threadIdx.x];
        a = {v.x, v.y};
    }
    finish<BF16>(A, n, join_all(a, A.scale * kLog2e, sh.sums), sh);
}

// A token's gradient where it is not listed: g times exp(d) weight, base 2.  The
// row's vector `at`, from its tokens' d.
template <bool BF16>
__device__ __forceinline__ void write_vector(const Args &A, int64_t n, const RowView<BF16> &row, int64_t at,
                                             float (&d)[RowView<BF16>::K], float g, float weight, bool none)
{
    constexpr int K = RowView<BF16>::K;
    const int64_t e = row.element(at);
#pragma unroll
    for (int k = 0; k < K; ++k) d[k] = none ? 0.0f : g * (ex2(d[k]) * weight);
    if (e >= 0) {
        store_raw<BF16, K>(A.dx, n * A.dstride, e, A.V, d);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (e + k >= 0 && e + k < A.V) store_gate<BF16>(A.dx, n * A.dstride + e + k, d[k]);
    }
}
// That of the listed token at entry e, from its q.
template <bool BF16>
__device__ __forceinline__ void write_listed(const Args &A, int64_t n, const Shared &sh, int e, float g, float q,
                                             float listed)
{
    const int64_t j = sh.list[e];
    if (!leads(sh, e)) return;
    float p = 0.0f;
#pragma unroll 8  // (by itself the compiler takes 82 registers, which leaves 5 of 8 waves)
    for (int d = e; d < A.count; ++d)
        if (sh.list[d] == j) p += expf(A.logprob[n * A.count + d]);
    store_gate<BF16>(A.dx, n * A.dstride + j, g * fmaf_(q, listed, -p));
}
// A whole row, from sums of its own.
template <bool BF16>
__device__ __forceinline__ void write_row(const Args &A, int64_t n, const RowView<BF16> &row, Shared &sh,
                                          uint32_t (&marks)[kSectionAgain / 4], float (&logit)[kMost], float g,
                                          float r, float listed)
{
    constexpr int K = RowView<BF16>::K;
    const float c = A.scale * kLog2e;
    for (int e = threadIdx.x; e < A.count; e += kThreads)
        logit[e] = sh.list[e] >= 0 && sh.list[e] < A.V ? load_gate<BF16>(A.x, n * A.stride + sh.list[e]) : 0.0f;
    Sum rest = no_sum();
    for (int64_t s0 = 0; s0 < row.vectors; s0 += kSectionAgain) {
        const int64_t s1 = min(row.vectors, s0 + kSectionAgain);
        mark_listed<BF16, kSectionAgain>(A, row, s0, s1, sh, marks);
        for (int64_t at = s0 + threadIdx.x; at < s1; at += kThreads) {
            float x[K];
            row.load(at, x);
            add_unmarked(rest, x, marks[(at - s0) / 4] >> (8 * ((at - s0) % 4)) & 0xffu, c);
        }
    }
    rest = join_all(rest, c, sh.sums);
    const Sum all = join(join_all(listed_of<BF16>(A, n, sh), c, sh.sums), rest, c);
    const float q_rest = ex2(c * (rest.m - all.m)) / all.s;  // of a token at rest.m
    const float weight = rest.s == 0.0f ? 0.0f : fmaf_(q_rest, listed, -r / rest.s);
    for (int64_t at = threadIdx.x; at < row.vectors; at += kThreads) {
        float d[K];
        row.load(at, d);
#pragma unroll
        for (int k = 0; k < K; ++k) d[k] = c * (d[k] - rest.m);
        write_vector<BF16>(A, n, row, at, d, g, weight, false);
    }
    __builtin_amdgcn_s_waitcnt(0);  // the stores above have arrived
    __syncthreads();
    for (int e = threadIdx.x; e < A.count; e += kThreads)
        if (sh.list[e] >= 0 && sh.list[e] < A.V)
            write_listed<BF16>(A, n, sh, e, g, ex2(c * (logit[e] - all.m)) / all.s, listed);
}

// The gradient, U vectors a lane as in the scores' gradient: every token as
// one that is not listed; then, behind a wait for these stores, the list's
// tokens once more.  Their logits are read before anything is written, for the
// gradient may take the logits' place.  A rare row, where the student leaves less
// than e^kFar to the other tokens or lse is beyond kLarge, is summed again by its first
// workgroup, which writes all of it (nobody may write a row that is still to be summed).
// Bound by HBM and vector instructions: 8192 rows of 32000 bfloat16 232 us a call,
// 4.5 TB/s, float32 416 us, 5.0 TB/s; all of them rare ones 960 us.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) distill_adjoint_kernel(Args A)
{
    using Row = RowView<BF16>;
    constexpr int K = Row::K, U = kScoreUnroll;
    __shared__ Shared sh;
    __shared__ uint32_t marks[kSectionAgain / 4];
    __shared__ float logit[kMost];
    const int64_t n = blockIdx.x / A.parts;
    const Row row(A.x, n * A.stride, A.V);
    const int64_t first = (blockIdx.x - n * A.parts) * (U * kThreads), i = first + threadIdx.x;
    uint4 raw[U];  // (as loaded: with twice the registers fewer waves fit)
#pragma unroll
    for (int q = 0; q < U; ++q)
        if (i + q * kThreads < row.vectors) raw[q] = row.load_raw(i + q * kThreads);
    load_list(A, n, sh);
    __syncthreads();
    // the part's entries
    const int64_t e0 = row.element(first), e1 = row.element(first + U * kThreads);
    float mine[kEach];
    double P = 0.0;
    bool any = false;
#pragma unroll
    for (int s = 0; s < kEach; ++s) {
        const int e = s * kThreads + threadIdx.x;
        mine[s] = 0.0f;
        if (e >= A.count || sh.list[e] < 0) continue;
        const int64_t j = sh.list[e];
        any = true;
        P += j < A.V ? expf(A.logprob[n * A.count + e]) : __builtin_nanf("");  // and with it the whole row, as the loss
        if (j >= e0 && j < e1 && j < A.V) mine[s] = load_gate<BF16>(A.x, n * A.stride + j);
    }
    P = add_all(P, sh.adds);
    any = __syncthreads_or(any);
    const float lse = A.lse_in[n], log_rest = A.log_rest_in[n], g = A.scale * A.g_loss[n];
    const bool none = !any || (lse == -__builtin_inff() && P == P);
    float r = A.tail ? (float)(1.0 - P) : 0.0f;
    if (r < kRest) r = 0.0f;
    const float listed = (float)P + r;
    if (!none && P == P && ((r > 0.0f && log_rest < kFar) || fabsf(lse) > kLarge)) {
        if (first == 0) write_row<BF16>(A, n, row, sh, marks, logit, g, r, listed);
        return;
    }
    // r shares of q_rest, or without an r q itself
    const float from = r == 0.0f ? lse : lse + log_rest;
    const float weight = r == 0.0f ? listed : fmaf_(expf(log_rest), listed, -r);
#pragma unroll
    for (int q = 0; q < U; ++q) {
        if (i + q * kThreads >= row.vectors) break;
        float x[K];
        Row::values(raw[q], x);
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = kLog2e * fmaf_(A.scale, x[k], -from);
        write_vector<BF16>(A, n, row, i + q * kThreads, x, g, weight, none);
    }
    __builtin_amdgcn_s_waitcnt(0);  // the stores above have arrived
    __syncthreads();
    if (none) return;
#pragma unroll
    for (int s = 0; s < kEach; ++s) {
        const int e = s * kThreads + threadIdx.x;
        if (e >= A.count) break;
        const int64_t j = sh.list[e];
        if (j < 0 || j >= A.V || j < e0 || j >= e1) continue;
        write_listed<BF16>(A, n, sh, e, g, ex2(kLog2e * fmaf_(A.scale, mine[s], -lse)), listed);
    }
}

}  // namespace distill
}  // namespace pararnn
