// Gated delta rule: a recurrence whose state is a matrix per head, S [dk][dv],
// which stores values under keys.  Per step, with key k, value v, query q, a
// rate b = beta and a decay a = exp(log_decay),
//     S <- a S,   w = b (v - k^T S),   S <- S + k w^T,   o = scale q^T S.
//
// A chunk of C steps at once.  With G_i the sum of the chunk's log decays up
// to step i, D_ij = exp(G_i - G_j) for j <= i, and S the state before the
// chunk, what the steps write, the rows w_i of W, solves
//     (I + A) W = R,  A_ij = b_i (k_i . k_j) D_ij for j < i,
//     R_i = b_i (v_i - exp(G_i) k_i^T S),
// and
//     o_i = scale (exp(G_i) q_i^T S + sum_{j <= i} (q_i . k_j) D_ij w_j),
//     S'  = exp(G_C) S + sum_i exp(G_C - G_i) k_i w_i^T.
// So a chunk is a few matrix products, and only the state goes from one chunk
// to the next.  M = (I + A)^-1 needs no state: delta_inverse_kernel computes
// it for all chunks at once.  delta_chain_kernel then goes along the chunks,
// a workgroup for a head and a block of the values' columns (columns of S do
// not meet), its state in registers.
//
// Backward, with X = M^T dW the gradient of R:
//     dW = scale P^T dO + exp(G_C - G_i) K dS',  P_ij = (q_i . k_j) D_ij,
//     dS = exp(G_C) dS' + scale (exp(G) Q)^T dO - (b exp(G) K)^T X.
// delta_chain_kernel runs again for the states and W (keeping them would cost
// 1.5 times the inputs' memory until the backward pass), delta_back_kernel
// goes along the chunks in reverse for dS' and X, and delta_grad_kernel
// computes the gradients of all chunks at once from these.
//
// Numbers.  States, sums and everything between the inputs and the outputs
// hold float32's precision.  Operands of the matrix cores are bfloat16; what
// is not one by itself is two, the value rounded and what that leaves, 16 bits
// and more together: 2^-17 of an operand is lost, and 2^-18 of a product of
// two such (the product of the two remainders is left out).  float32 inputs go
// to the float32 matrix instructions.  Sums of log decays are float64, and
// differences of them are taken in two floats, so that a decay keeps its
// precision behind a step that forgot everything.
//
// Documents.  A step where a document starts (its reset flag, or a log decay
// below kForget, whose exponential float32 does not hold) keeps nothing of the
// state, whatever is in it.  A chunk that holds several documents is visited
// once for each, with the rows of the others zero.
#pragma once

#include <hip/hip_runtime.h>

#include "delta_step.hpp"
#include "elements.hpp"
#include "pararnn.h"

namespace pararnn {
namespace delta {

constexpr int kWaves = 8, kThreads = kWaves * kWave;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A tensor indexed [b][h][d][t], strides in elements.
struct Plane {
    void *p;
    int64_t b, h, d, t;
};
struct Args {
    Plane q, k, v, o, dq, dk, dv;     // o: the output, or its gradient
    const float *beta, *decay;        // [b][h][t]; decay may be null
    int64_t gate_b, gate_h, gate_t;
    const uint8_t *resets;            // [B][T] or null
    const float *h0, *g_last;         // [B][Hv][dk][dv] or null
    float *last, *dh0;                // the same
    float *dbeta, *ddecay;            // [B][Hv][T]
    int64_t B, T, chunks;
    int32_t Hk, Hv, key, value;       // key, value: dk, dv
    int32_t value_pad, blocks;        // columns of the workspace's rows; blocks of them
    float scale;
    // workspace
    void *inverse, *inverse_t;        // [b h][chunk][C][C] operands
    float *states, *dstates;          // [b h][chunk][DK][value_pad]
    float *w, *x;                     // [b h][chunk * C][value_pad]
    float *xv;                        // [b h][chunk * C][blocks]: X . V of a block of columns
};

// ---------------------------------------------------------------- numbers ---

// How 8 consecutive elements of an operand are held.  HALF: bfloat16 inputs.
template <bool HALF>
struct Num;

template <>
struct Num<true> {
    static constexpr int kChunk = 64, kPad = 8;
    using Elem = uint16_t;
    using Exact = bf16x8;
    struct Wide {
        bf16x8 hi, lo;
    };
};
template <>
struct Num<false> {
    static constexpr int kChunk = 32, kPad = 4;
    using Elem = float;
    struct Exact {
        float x[8];
    };
    using Wide = Exact;
};
using Bf = Num<true>;
using Fl = Num<false>;

__device__ __forceinline__ f32x4 mma(f32x4 c, bf16x8 a, bf16x8 b)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(f32x4 c, bf16x8 a, const Bf::Wide &b)
{
    return mma(mma(c, a, b.lo), a, b.hi);
}
__device__ __forceinline__ f32x4 mma(f32x4 c, const Bf::Wide &a, bf16x8 b)
{
    return mma(mma(c, a.lo, b), a.hi, b);
}
__device__ __forceinline__ f32x4 mma(f32x4 c, const Bf::Wide &a, const Bf::Wide &b)
{
    return mma(mma(mma(c, a.lo, b.hi), a.hi, b.lo), a.hi, b.hi);
}
// Eight instructions of 4 terms: the j-th takes the j-th element of every
// lane's eight, a permutation of the sum that both operands share.
__device__ __forceinline__ f32x4 mma(f32x4 c, const Fl::Exact &a, const Fl::Exact &b)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x[j], b.x[j], c, 0, 0, 0);
    return c;
}

// A float32 as the bfloat16 next to it and the one next to what that leaves.
__device__ __forceinline__ void split(float x, __bf16 &hi, __bf16 &lo)
{
    hi = (__bf16)x;
    lo = (__bf16)(x - (float)hi);
}
__device__ __forceinline__ Bf::Wide split(const float (&x)[8], Bf::Wide)
{
    Bf::Wide w;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        __bf16 h, l;
        split(x[j], h, l);
        w.hi[j] = h;
        w.lo[j] = l;
    }
    return w;
}
__device__ __forceinline__ Fl::Wide split(const float (&x)[8], Fl::Wide)
{
    Fl::Wide w;
#pragma unroll
    for (int j = 0; j < 8; ++j) w.x[j] = x[j];
    return w;
}

// ------------------------------------------------------------- LDS tiles ---

// ROWS rows of COLS elements side by side, 16 bytes between rows so that 16
// rows start on different banks.
template <bool HALF, int ROWS, int COLS>
struct Tile {
    static constexpr int kPitch = COLS + Num<HALF>::kPad;
    alignas(16) typename Num<HALF>::Elem at[ROWS * kPitch];
};
// The same for values of float32's precision: two bfloat16 planes, or one.
template <bool HALF, int ROWS, int COLS>
struct WideTile {
    static constexpr int kPitch = COLS + Num<HALF>::kPad, kRows = ROWS;
    alignas(16) typename Num<HALF>::Elem at[(HALF ? 2 : 1) * ROWS * kPitch];
};

// Operands of a 16x16 product: lane l holds row (or column) i0 + l % 16 and
// the terms k0 + 8 (l / 16) .. + 7 of the sum.
// along: the terms lie side by side in the tile's rows.
__device__ __forceinline__ bf16x8 operand_along(const uint16_t *at, int pitch, int i0, int k0)
{
    const int lane = threadIdx.x % kWave;
    const uint4 v = *reinterpret_cast<const uint4 *>(at + (i0 + lane % 16) * pitch + k0 + 8 * (lane / 16));
    bf16x8 r;
    __builtin_memcpy(&r, &v, 16);
    return r;
}
__device__ __forceinline__ Fl::Exact operand_along(const float *at, int pitch, int i0, int k0)
{
    const int lane = threadIdx.x % kWave;
    const float *p = at + (i0 + lane % 16) * pitch + k0 + 8 * (lane / 16);
    Fl::Exact r;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p + j);
        r.x[j] = v.x, r.x[j + 1] = v.y, r.x[j + 2] = v.z, r.x[j + 3] = v.w;
    }
    return r;
}
// across: the terms are rows of the tile, the operand's rows its columns.  The
// transposing read takes four elements of a row from each lane of 16 and gives
// lane i the i-th of 16 columns of the four rows.
__device__ __forceinline__ s16x4 read_transposed(const uint16_t *p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4 *)(__attribute__((address_space(3))) void *)p);
}
__device__ __forceinline__ bf16x8 operand_across(const uint16_t *at, int pitch, int i0, int k0)
{
    const int lane = threadIdx.x % kWave, i = lane % 16;
    const uint16_t *p = at + (k0 + 8 * (lane / 16) + i / 4) * pitch + i0 + 4 * (i % 4);
    const s16x4 a = read_transposed(p), b = read_transposed(p + 4 * pitch);
    bf16x8 r;
    __builtin_memcpy(&r, &a, 8);
    __builtin_memcpy(reinterpret_cast<char *>(&r) + 8, &b, 8);
    return r;
}
__device__ __forceinline__ Fl::Exact operand_across(const float *at, int pitch, int i0, int k0)
{
    const int lane = threadIdx.x % kWave;
    const float *p = at + (k0 + 8 * (lane / 16)) * pitch + i0 + lane % 16;
    Fl::Exact r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.x[j] = p[j * pitch];
    return r;
}
template <bool ALONG, bool HALF, int ROWS, int COLS>
__device__ __forceinline__ typename Num<HALF>::Exact operand(const Tile<HALF, ROWS, COLS> &t, int i0, int k0)
{
    if constexpr (ALONG)
        return operand_along(t.at, t.kPitch, i0, k0);
    else
        return operand_across(t.at, t.kPitch, i0, k0);
}
template <bool ALONG, bool HALF, int ROWS, int COLS>
__device__ __forceinline__ typename Num<HALF>::Wide operand(const WideTile<HALF, ROWS, COLS> &t, int i0,
                                                            int k0)
{
    const auto half = [&](int plane) {
        const auto *at = t.at + plane * ROWS * t.kPitch;
        if constexpr (ALONG)
            return operand_along(at, t.kPitch, i0, k0);
        else
            return operand_across(at, t.kPitch, i0, k0);
    };
    if constexpr (HALF)
        return {half(0), half(1)};
    else
        return half(0);
}
// Four values side by side at (row, col), col a multiple of 4.
template <bool HALF, int ROWS, int COLS>
__device__ __forceinline__ void store4(WideTile<HALF, ROWS, COLS> &t, int row, int col, f32x4 x)
{
    auto *p = t.at + row * t.kPitch + col;
    if constexpr (HALF) {
        bf16x4 hi, lo;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            __bf16 h, l;
            split(x[r], h, l);
            hi[r] = h;
            lo[r] = l;
        }
        __builtin_memcpy(p, &hi, 8);
        __builtin_memcpy(p + ROWS * t.kPitch, &lo, 8);
    } else {
        __builtin_memcpy(p, &x, 16);
    }
}
template <bool HALF, int ROWS, int COLS>
__device__ __forceinline__ void clear(WideTile<HALF, ROWS, COLS> &t)
{
    auto *w = reinterpret_cast<uint32_t *>(t.at);
    for (int i = threadIdx.x; i < (int)(sizeof(t.at) / 4); i += blockDim.x) w[i] = 0;
}

// --------------------------------------------------- inputs and documents ---

// A chunk of queries or keys, DK channels of C steps, as 16-byte pieces in
// registers and then in LDS, the steps side by side (TF) or the channels.
// Channels from `key` and steps from T on are zero and not read.
template <bool HALF, int DK, bool TF, int THREADS>
struct Pieces {
    using Elem = typename Num<HALF>::Elem;
    static constexpr int C = Num<HALF>::kChunk, E = 16 / (int)sizeof(Elem);
    static constexpr int kPerRow = (TF ? C : DK) / E, kCount = DK * C / E / THREADS;
    static_assert(kCount >= 1 && DK * C / E % THREADS == 0, "whole pieces a thread");
    using Lds = Tile<HALF, TF ? DK : C, TF ? C : DK>;
    uint4 u[kCount];

    static __device__ __forceinline__ uint32_t element(const Elem *p)
    {
        if constexpr (HALF)
            return *p;
        else
            return __float_as_uint(*p);
    }
    // base: the head's first element; d0: the first channel; t0: the chunk's first step
    __device__ __forceinline__ void load(const Plane &x, const void *base, int d0, int64_t t0, int key, int64_t T)
    {
#pragma unroll
        for (int n = 0; n < kCount; ++n) {
            const int i = n * THREADS + threadIdx.x, row = i / kPerRow, col = i % kPerRow * E;
            const int d = d0 + (TF ? row : col);
            const int64_t t = t0 + (TF ? col : row);
            const Elem *p = static_cast<const Elem *>(base) + d * x.d + t * x.t;
            u[n] = make_uint4(0, 0, 0, 0);
            const bool whole = TF ? d < key && t + E <= T && x.t == 1 : t < T && d + E <= key && x.d == 1;
            if (whole) {
                const Words4 w = *reinterpret_cast<const Words4Any *>(p);
                u[n] = make_uint4(w.x, w.y, w.z, w.w);
            } else if (d < key && t < T) {
                const int64_t step = TF ? x.t : x.d, left = TF ? T - t : key - d;
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (e < left) {
                        if constexpr (HALF)
                            w[e / 2] |= element(p + e * step) << (16 * (e % 2));
                        else
                            w[e] = element(p + e * step);
                    }
                u[n] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    // Steps outside r0 .. r1 - 1 of the chunk are zero.
    __device__ __forceinline__ void store(Lds &lds, int r0, int r1) const
    {
#pragma unroll
        for (int n = 0; n < kCount; ++n) {
            const int i = n * THREADS + threadIdx.x, row = i / kPerRow, col = i % kPerRow * E;
            uint32_t w[4] = {u[n].x, u[n].y, u[n].z, u[n].w};
            if constexpr (TF) {
                if (col < r0 || col + E > r1) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (col + e < r0 || col + e >= r1) {
                            if constexpr (HALF)
                                w[e / 2] &= e % 2 ? 0x0000ffffu : 0xffff0000u;
                            else
                                w[e] = 0;
                        }
                }
            } else if (row < r0 || row >= r1) {
                w[0] = w[1] = w[2] = w[3] = 0;
            }
            *reinterpret_cast<uint4 *>(lds.at + row * lds.kPitch + col) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// Four consecutive steps of one channel: elements at p, p + step, ..., those of
// steps first .. end - 1 (counted from the first of the four); others read as 0.
template <bool HALF>
__device__ __forceinline__ f32x4 load_steps(const void *base, int64_t off, int64_t step, int first, int end)
{
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (first <= 0 && end >= 4 && step == 1) {
        if constexpr (HALF) {
            const Words2 w = *reinterpret_cast<const Words2Any *>(static_cast<const uint16_t *>(base) + off);
            x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xffff0000u);
            x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
            const Words4 w = *reinterpret_cast<const Words4Any *>(static_cast<const float *>(base) + off);
            x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y);
            x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
        }
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r >= first && r < end) x[r] = load_gate<HALF>(base, off + r * step);
    }
    return x;
}
template <bool HALF>
__device__ __forceinline__ void store_steps(void *base, int64_t off, int64_t step, int first, int end, f32x4 x)
{
    if (first <= 0 && end >= 4 && step == 1) {
        if constexpr (HALF) {
            const Words2 w = {bf16_bits(x[0]) | bf16_bits(x[1]) << 16, bf16_bits(x[2]) | bf16_bits(x[3]) << 16};
            *reinterpret_cast<Words2Any *>(static_cast<uint16_t *>(base) + off) = w;
        } else {
            const Words4 w = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                              __float_as_uint(x[3])};
            *reinterpret_cast<Words4Any *>(static_cast<float *>(base) + off) = w;
        }
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r >= first && r < end) store_gate<HALF>(base, off + r * step, x[r]);
    }
}

// The gates of a chunk's steps, one a lane; the same in every wave.
struct StepGates {
    float g, beta;
    uint64_t cut;  // steps that keep nothing of the state before them
    int rows;      // the chunk's steps
};
template <int C>
__device__ __forceinline__ StepGates load_gates(const Args &A, int64_t b, int64_t h, int64_t t0)
{
    const int lane = threadIdx.x % kWave;
    const int64_t t = t0 + lane, at = b * A.gate_b + h * A.gate_h + t * A.gate_t;
    StepGates s = {0.0f, 0.0f, 0, (int)(A.T - t0 < C ? A.T - t0 : C)};
    bool cut = false;
    if (lane < s.rows) {
        if (A.decay) s.g = A.decay[at];
        s.beta = A.beta[at];
        cut = (A.resets && A.resets[b * A.T + t]) || s.g < kForget;
    }
    s.cut = __ballot(cut);
    return s;
}
__device__ __forceinline__ uint64_t steps_below(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }
// The first step after r0 that starts a document, or `rows`.
__device__ __forceinline__ int document_end(uint64_t cut, int r0, int rows)
{
    const uint64_t after = cut & ~steps_below(r0 + 1);
    const int end = after ? __builtin_ctzll(after) : rows;
    return end < rows ? end : rows;
}
// The step at which the document of step r1 - 1 starts in this chunk.
__device__ __forceinline__ int document_start(uint64_t cut, int r1)
{
    const uint64_t upto = cut & steps_below(r1);
    return upto ? 63 - __builtin_clzll(upto) : 0;
}
// Sums of the document's log decays (base 2) up to each step, from its first
// step in the chunk; steps of other documents take the value at their side.
__device__ __forceinline__ double decay_sum(const StepGates &s, int r0, int r1)
{
    const int lane = threadIdx.x % kWave;
    const bool mine = lane >= r0 && lane < r1 && !(s.cut >> lane & 1);
    double G = mine ? (double)s.g * 1.4426950408889634 : 0.0;
#pragma unroll
    for (int off = 1; off < kWave; off *= 2) {
        const double before = __shfl_up(G, off);
        if (lane >= off) G += before;
    }
    return G;
}
// What a visit's steps multiply with, in LDS.
template <int C>
struct alignas(16) Factors {
    float hi[C], lo[C];  // the decay's sum, in two floats
    float start[C];      // exp(G_i)
    float end[C];        // exp(G_C - G_i)
    float beta[C];
    float across[4];     // exp(G_C)
};
template <int C>
__device__ __forceinline__ void write_factors(Factors<C> &F, const StepGates &s, int r0, int r1)
{
    const int lane = threadIdx.x % kWave;
    const double G = decay_sum(s, r0, r1), total = __shfl(G, kWave - 1);
    if (lane < C) {
        const float hi = (float)G;
        F.hi[lane] = hi;
        F.lo[lane] = (float)(G - hi);
        F.start[lane] = ex2(hi);
        F.end[lane] = ex2((float)(total - G));
        F.beta[lane] = lane >= r0 && lane < r1 ? s.beta : 0.0f;
    }
    if (lane == 0) F.across[0] = ex2((float)total);
}
// exp(G_i - G_j)
template <int C>
__device__ __forceinline__ float decay_between(const Factors<C> &F, int i, int j)
{
    return ex2((F.hi[i] - F.hi[j]) + (F.lo[i] - F.lo[j]));
}
__device__ __forceinline__ f32x4 four(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
// x where the step is one of the visit's, else 0, whatever x is.
__device__ __forceinline__ f32x4 only_steps(f32x4 x, int first, int r0, int r1)
{
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = first + r >= r0 && first + r < r1 ? x[r] : 0.0f;
    return x;
}
// The n-th pair (i, j) with j <= i, row by row.
__device__ __forceinline__ void lower_pair(int n, int &i, int &j)
{
    i = n >= 6 ? 3 : n >= 3 ? 2 : n >= 1 ? 1 : 0;
    j = n - i * (i + 1) / 2;
}

// Workgroup -> (head, block of columns): the blocks of a head read the same
// queries and keys, so they go to one XCD (workgroups are dealt to the 8 XCDs
// in turn) where the heads allow it.
__device__ __forceinline__ void head_and_block(int64_t heads, int blocks, int64_t &head, int &block)
{
    const int64_t g = blockIdx.x;
    if (heads % 8 == 0) {
        block = (int)(g / 8 % blocks);
        head = g % 8 + 8 * (g / (8 * (int64_t)blocks));
    } else {
        head = g / blocks;
        block = (int)(g % blocks);
    }
}

// ------------------------------------------------------------ (I + A)^-1 ---

// Float32 products of 16x16 blocks: the four terms k0 + 4 (l / 16) .. + 3 of lane
// l's row or column, side by side in the matrix's rows or across them.
template <bool ALONG>
__device__ __forceinline__ f32x4 block_operand(const float *at, int pitch, int i0, int k0)
{
    const int lane = threadIdx.x % kWave, i = i0 + lane % 16, k = k0 + 4 * (lane / 16);
    if constexpr (ALONG) return four(at + i * pitch + k);
    f32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = at[(k + j) * pitch + i];
    return r;
}
__device__ __forceinline__ f32x4 block_mma(f32x4 c, f32x4 a, f32x4 b)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// A wave for a head's chunk.  K K^T on the matrix cores, 32 channels at a
// time.  The 16x16 blocks of the diagonal are inverted column by column, a
// lane each; then inverses are joined two by two,
//     [L 0; B R]^-1 = [L^-1 0; -R^-1 B L^-1 R^-1],
// in float32 products.  (A lane for a whole column of 64 needs every element
// of A in every lane: 500 wide LDS reads a chunk, or 1600 spilled registers.)
// Entries between documents are set to zero rather than computed.
template <bool HALF, bool TF>
__global__ void __launch_bounds__(kWave) delta_inverse_kernel(Args A)
{
    constexpr int C = Num<HALF>::kChunk, TT = C / 16, kTiles = TT * (TT + 1) / 2, kPitch = C + 4;
    using Keys = Pieces<HALF, 32, TF, kWave>;
    // all by columns: A, its inverse, and a product on the way
    __shared__ union {
        typename Keys::Lds keys;
        struct {
            alignas(16) float a[C * kPitch], m[C * kPitch], p[C / 2 * kPitch];
        };
    } sh;
    __shared__ Factors<C> F;
    const int lane = threadIdx.x, row4 = 4 * (lane / 16), col = lane % 16;
    const int64_t item = blockIdx.x, bh = item / A.chunks, n = item % A.chunks;
    const int64_t b = bh / A.Hv, h = bh % A.Hv, t0 = n * C;
    const StepGates gates = load_gates<C>(A, b, h, t0);
    const auto *keys = static_cast<const typename Num<HALF>::Elem *>(A.k.p) + b * A.k.b + h / (A.Hv / A.Hk) * A.k.h;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

    f32x4 acc[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[i] = zero;
    for (int d0 = 0; d0 < A.key; d0 += 32) {
        Keys raw;
        raw.load(A.k, keys, d0, t0, A.key, A.T);
        __syncthreads();
        raw.store(sh.keys, 0, C);
        __syncthreads();
        typename Num<HALF>::Exact f[TT];
#pragma unroll
        for (int i = 0; i < TT; ++i) f[i] = operand<!TF>(sh.keys, 16 * i, 0);
#pragma unroll
        for (int p = 0, i = 0; i < TT; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j, ++p) acc[p] = mma(acc[p], f[i], f[j]);
    }
    // every document's sums by themselves: a number that is not finite stays in its own
    {
        const int first = document_start(gates.cut, lane + 1);
        double G = lane < gates.rows && !(gates.cut >> lane & 1) ? (double)gates.g * 1.4426950408889634 : 0.0;
#pragma unroll
        for (int off = 1; off < kWave; off *= 2) {
            const double before = __shfl_up(G, off);
            if (lane - off >= first) G += before;
        }
        if (lane < C) {
            F.hi[lane] = (float)G;
            F.lo[lane] = (float)(G - (float)G);
            F.beta[lane] = gates.beta;
        }
    }
    __syncthreads();
    const auto joined = [&](int i, int j) {  // j <= i in one document
        return !(gates.cut & steps_below(i + 1) & ~steps_below(j + 1));
    };
#pragma unroll
    for (int p = 0, it = 0; it < TT; ++it)
#pragma unroll
        for (int jt = 0; jt <= it; ++jt, ++p) {
            const int i = 16 * it + row4, j = 16 * jt + col;
            f32x4 a;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                a[r] = i + r > j && joined(i + r, j) ? F.beta[i + r] * acc[p][r] * decay_between(F, i + r, j) : 0.0f;
            *reinterpret_cast<f32x4 *>(sh.a + j * kPitch + i) = a;
        }
    __syncthreads();
    if (lane < C) {
        const int first = lane / 16 * 16;
        f32x4 m[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i / 4][i % 4] = i == col ? 1.0f : 0.0f;
#pragma unroll
        for (int l = 0; l < 15; ++l) {
            if (l < col) m[l / 4][l % 4] = 0.0f;  // also where an earlier document made it a NaN
#pragma unroll
            for (int i = (l + 1) / 4; i < 4; ++i) {
                const f32x4 a = four(sh.a + (first + l) * kPitch + first + 4 * i);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (4 * i + r > l) m[i][r] = fmaf_(-a[r], m[l / 4][l % 4], m[i][r]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) m[i][r] = 4 * i + r < col ? 0.0f : m[i][r];
            *reinterpret_cast<f32x4 *>(sh.m + lane * kPitch + first + 4 * i) = m[i];
        }
    }
#pragma unroll
    for (int size = 1; size < TT; size *= 2)  // 16x16 blocks of one inverse
#pragma unroll
        for (int at = 0; at < TT; at += 2 * size) {
            __syncthreads();
            // p = B L^-1, rows of the right inverse's blocks
#pragma unroll
            for (int i = 0; i < size; ++i)
#pragma unroll
                for (int j = 0; j < size; ++j) {
                    f32x4 c = zero;
#pragma unroll
                    for (int l = j; l < size; ++l)
                        c = block_mma(c, block_operand<false>(sh.a, kPitch, 16 * (at + size + i), 16 * (at + l)),
                                      block_operand<true>(sh.m, kPitch, 16 * (at + j), 16 * (at + l)));
                    *reinterpret_cast<f32x4 *>(sh.p + (16 * j + col) * kPitch + 16 * i + row4) = c;
                }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < size; ++i)
#pragma unroll
                for (int j = 0; j < size; ++j) {
                    f32x4 c = zero;
#pragma unroll
                    for (int l = 0; l <= i; ++l)
                        c = block_mma(c, block_operand<false>(sh.m, kPitch, 16 * (at + size + i), 16 * (at + size + l)),
                                      block_operand<true>(sh.p, kPitch, 16 * j, 16 * l));
                    *reinterpret_cast<f32x4 *>(sh.m + (16 * (at + j) + col) * kPitch + 16 * (at + size + i) + row4) = -c;
                }
        }
    __syncthreads();
    // rows (and for the backward pass columns) of 8 elements a lane
    const auto put = [&](void *out, bool by_columns) {
        for (int u = lane; u < C * C / 8; u += kWave) {
            const int row = u / (C / 8), c8 = u % (C / 8) * 8;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = by_columns ? c8 + e : row, j = by_columns ? row : c8 + e;
                x[e] = i >= j && joined(i, j) ? sh.m[j * kPitch + i] : 0.0f;
            }
            if constexpr (HALF) {
                const Bf::Wide w = split(x, Bf::Wide());
                __bf16 *p = static_cast<__bf16 *>(out) + 2 * item * C * C + row * C + c8;
                *reinterpret_cast<bf16x8 *>(p) = w.hi;
                *reinterpret_cast<bf16x8 *>(p + C * C) = w.lo;
            } else {
                float *p = static_cast<float *>(out) + item * C * C + row * C + c8;
#pragma unroll
                for (int e = 0; e < 8; e += 4) *reinterpret_cast<f32x4 *>(p + e) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
            }
        }
    };
    put(A.inverse, false);
    if (A.inverse_t) put(A.inverse_t, true);
}
// An operand from such a matrix in memory.
__device__ __forceinline__ Bf::Wide operand_of(const void *m, int64_t item, int i0, int k0, Bf)
{
    constexpr int C = Bf::kChunk;
    const int lane = threadIdx.x % kWave;
    const __bf16 *p = static_cast<const __bf16 *>(m) + 2 * item * C * C + (i0 + lane % 16) * C + k0 + 8 * (lane / 16);
    return {*reinterpret_cast<const bf16x8 *>(p), *reinterpret_cast<const bf16x8 *>(p + C * C)};
}
__device__ __forceinline__ Fl::Wide operand_of(const void *m, int64_t item, int i0, int k0, Fl)
{
    constexpr int C = Fl::kChunk;
    const int lane = threadIdx.x % kWave;
    const float *p = static_cast<const float *>(m) + item * C * C + (i0 + lane % 16) * C + k0 + 8 * (lane / 16);
    Fl::Wide r;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
        const f32x4 v = four(p + j);
        r.x[j] = v[0], r.x[j + 1] = v[1], r.x[j + 2] = v[2], r.x[j + 3] = v[3];
    }
    return r;
}

// A state's tiles in a wave's registers: tile wave + 8 n, of DT x VT.
template <int DK, int VB>
struct State {
    static constexpr int DT = DK / 16, VT = VB / 16, kCount = (DT * VT + kWaves - 1) / kWaves;
    f32x4 s[kCount];
    static __device__ __forceinline__ bool tile(int n, int wave, int &d0, int &v0)
    {
        const int i = wave + kWaves * n;
        d0 = 16 * (i / VT);
        v0 = 16 * (i % VT);
        return i < DT * VT;
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int n = 0; n < kCount; ++n) s[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // rows of `pitch` values, those from `key` and `value` on not there
    __device__ __forceinline__ void load(const float *p, int wave, int lane, int64_t v_first, int key, int64_t value)
    {
        zero();
#pragma unroll
        for (int n = 0; n < kCount; ++n) {
            int d0, v0;
            if (!tile(n, wave, d0, v0)) break;
            const int64_t v = v_first + v0 + lane % 16;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = d0 + 4 * (lane / 16) + r;
                if (d < key && v < value) s[n][r] = p[d * value + v];
            }
        }
    }
    __device__ __forceinline__ void store(float *p, int wave, int lane, int64_t v_first, int key, int64_t value,
                                          int64_t pitch) const
    {
#pragma unroll
        for (int n = 0; n < kCount; ++n) {
            int d0, v0;
            if (!tile(n, wave, d0, v0)) break;
            const int64_t v = v_first + v0 + lane % 16;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = d0 + 4 * (lane / 16) + r;
                if (d < key && v < value) p[d * pitch + v] = s[n][r];
            }
        }
    }
    template <bool HALF>
    __device__ __forceinline__ void to_lds(WideTile<HALF, VB, DK> &t, int wave, int lane) const
    {
#pragma unroll
        for (int n = 0; n < kCount; ++n) {
            int d0, v0;
            if (!tile(n, wave, d0, v0)) break;
            store4(t, v0 + lane % 16, d0 + 4 * (lane / 16), s[n]);
        }
    }
};

// ------------------------------------------------------------- the chain ---

// A workgroup for a head and VB columns, chunk after chunk.  The products'
// tiles are dealt to the waves: a wave that owns a tile of [C][VB] computes
// k^T S, q^T S, then R, W and the output of it, all of them the tiles of P and
// of the state.  STATES: for the backward pass, the states before each chunk
// and W instead of the outputs.
template <bool HALF, int DK, int VB, bool TF, bool STATES>
__global__ void __launch_bounds__(kThreads) delta_chain_kernel(Args A)
{
    using N = Num<HALF>;
    constexpr int C = N::kChunk, TT = C / 16, VT = VB / 16, kOwners = TT * VT;
    using In = Pieces<HALF, DK, TF, kThreads>;
    using St = State<DK, VB>;
    static_assert(kOwners <= kWaves, "a tile a wave");
    __shared__ typename In::Lds keys, queries;
    __shared__ WideTile<HALF, VB, DK> state;
    __shared__ WideTile<HALF, VB, C> rhs, write, carry;
    __shared__ WideTile<HALF, C, C> scores;
    __shared__ Factors<C> F;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, row4 = 4 * (lane / 16), col = lane % 16;
    int64_t bh;
    int block;
    head_and_block(A.B * A.Hv, A.blocks, bh, block);
    const int64_t b = bh / A.Hv, h = bh % A.Hv, hk = h / (A.Hv / A.Hk), v_first = (int64_t)block * VB;
    const bool owner = wave < kOwners;
    const int tt = 16 * (wave / VT), vt = 16 * (wave % VT);  // the owner's tile
    const int64_t v = v_first + vt + col;
    const bool has_v = owner && v < A.value;
    const int64_t v_at = b * A.v.b + h * A.v.h + v * A.v.d, o_at = b * A.o.b + h * A.o.h + v * A.o.d;
    using Elem = typename N::Elem;
    const Elem *const kb = static_cast<const Elem *>(A.k.p) + b * A.k.b + hk * A.k.h;
    const Elem *const qb = static_cast<const Elem *>(A.q.p) + b * A.q.b + hk * A.q.h;

    St S;
    S.zero();
    if (A.h0) S.load(A.h0 + bh * A.key * A.value, wave, lane, v_first, A.key, A.value);
    S.to_lds(state, wave, lane);
    if constexpr (!STATES) clear(scores);
    for (int64_t n = 0; n < A.chunks; ++n) {
        const int64_t t0 = n * C, item = bh * A.chunks + n;
        const StepGates gates = load_gates<C>(A, b, h, t0);
        In k_raw;
        [[maybe_unused]] In q_raw;
        k_raw.load(A.k, kb, 0, t0, A.key, A.T);
        if constexpr (!STATES) q_raw.load(A.q, qb, 0, t0, A.key, A.T);
        if constexpr (STATES)
            S.store(A.states + item * DK * A.value_pad, wave, lane, v_first, DK, A.value_pad, A.value_pad);
        for (int r0 = 0; r0 < gates.rows;) {
            const int r1 = document_end(gates.cut, r0, gates.rows);
            if (gates.cut >> r0 & 1) {
                S.zero();
                S.to_lds(state, wave, lane);
            }
            k_raw.store(keys, r0, r1);
            if constexpr (!STATES) q_raw.store(queries, r0, r1);
            if (wave == 0) write_factors(F, gates, r0, r1);
            f32x4 value = {0.0f, 0.0f, 0.0f, 0.0f};
            if (has_v)
                value = load_steps<HALF>(A.v.p, v_at + (t0 + tt + row4) * A.v.t, A.v.t, r0 - tt - row4,
                                         r1 - tt - row4);
            __syncthreads();

            f32x4 ks = {0.0f, 0.0f, 0.0f, 0.0f};
            [[maybe_unused]] f32x4 qs = ks;
            if (owner) {
#pragma unroll
                for (int d = 0; d < DK; d += 32) {
                    const auto s = operand<true>(state, vt, d);
                    ks = mma(ks, operand<!TF>(keys, tt, d), s);
                    if constexpr (!STATES) qs = mma(qs, operand<!TF>(queries, tt, d), s);
                }
                const f32x4 start = four(F.start + tt + row4), beta = four(F.beta + tt + row4);
                f32x4 r;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    r[e] = beta[e] * fmaf_(-start[e], ks[e], value[e]);
                    if constexpr (!STATES) qs[e] *= A.scale * start[e];
                }
                store4(rhs, vt + col, tt + row4, only_steps(r, tt + row4, r0, r1));
            }
            if constexpr (!STATES) {
                // P by rows of t: its tile (s, t) as keys times queries, four s side by side
                for (int p = wave; p < TT * (TT + 1) / 2; p += kWaves) {
                    int ti, si;
                    lower_pair(p, ti, si);
                    ti *= 16, si *= 16;
                    f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int d = 0; d < DK; d += 32) c = mma(c, operand<!TF>(keys, si, d), operand<!TF>(queries, ti, d));
                    const int t = ti + col, s = si + row4;
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = s + e <= t ? A.scale * c[e] * decay_between(F, t, s + e) : 0.0f;
                    store4(scores, t, s, c);
                }
            }
            __syncthreads();

            if (owner) {
                f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < C; s += 32)
                    if (s <= tt) w = mma(w, operand_of(A.inverse, item, tt, s, N()), operand<true>(rhs, vt, s));
                w = only_steps(w, tt + row4, r0, r1);
                const f32x4 end = four(F.end + tt + row4);
                if constexpr (STATES) {
                    float *p = A.w + (item * C + tt + row4) * A.value_pad + v_first + vt + col;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (tt + row4 + e >= r0 && tt + row4 + e < r1) p[e * A.value_pad] = w[e];
                } else {
                    store4(write, vt + col, tt + row4, w);
                }
                f32x4 c;
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = end[e] * w[e];
                store4(carry, vt + col, tt + row4, only_steps(c, tt + row4, r0, r1));
            }
            __syncthreads();

            if constexpr (!STATES) {
                if (owner) {
#pragma unroll
                    for (int s = 0; s < C; s += 32)
                        if (s <= tt) qs = mma(qs, operand<true>(scores, tt, s), operand<true>(write, vt, s));
                    if (has_v)
                        store_steps<false>(A.o.p, o_at + (t0 + tt + row4) * A.o.t, A.o.t, r0 - tt - row4,
                                           r1 - tt - row4, qs);
                }
            }
            const float across = F.across[0];
#pragma unroll
            for (int i = 0; i < St::kCount; ++i) {
                int d0, v0;
                if (!St::tile(i, wave, d0, v0)) break;
                f32x4 c;
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = across * S.s[i][e];
#pragma unroll
                for (int s = 0; s < C; s += 32) c = mma(c, operand<TF>(keys, d0, s), operand<true>(carry, v0, s));
                S.s[i] = c;
            }
            S.to_lds(state, wave, lane);
            __syncthreads();
            r0 = r1;
        }
    }
    if constexpr (!STATES)
        if (A.last)
            S.store(A.last + bh * A.key * A.value, wave, lane, v_first, A.key, A.value, A.value);
}

// The chain backwards: the gradient of the state, from the last chunk to the
// first, and X, the gradient of R.  Writes the state's gradient behind each
// chunk, X, dV = b X and the rows' sums of X V over the block's columns.
template <bool HALF, int DK, int VB, bool TF>
__global__ void __launch_bounds__(kThreads) delta_back_kernel(Args A)
{
    using N = Num<HALF>;
    constexpr int C = N::kChunk, TT = C / 16, VT = VB / 16, kOwners = TT * VT;
    using In = Pieces<HALF, DK, TF, kThreads>;
    using St = State<DK, VB>;
    static_assert(kOwners <= kWaves, "a tile a wave");
    __shared__ typename In::Lds keys, queries;
    __shared__ WideTile<HALF, VB, DK> state;
    __shared__ WideTile<HALF, VB, C> out, out_q, write, carry;  // dO, its part for S, dW, X's part for S
    __shared__ WideTile<HALF, C, C> scores;                     // P by columns
    __shared__ Factors<C> F;
    __shared__ float products[C * VT];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, row4 = 4 * (lane / 16), col = lane % 16;
    int64_t bh;
    int block;
    head_and_block(A.B * A.Hv, A.blocks, bh, block);
    const int64_t b = bh / A.Hv, h = bh % A.Hv, hk = h / (A.Hv / A.Hk), v_first = (int64_t)block * VB;
    const bool owner = wave < kOwners;
    const int tt = 16 * (wave / VT), vt = 16 * (wave % VT);
    const int64_t v = v_first + vt + col;
    const bool has_v = owner && v < A.value;
    const int64_t v_at = b * A.v.b + h * A.v.h + v * A.v.d, o_at = b * A.o.b + h * A.o.h + v * A.o.d;
    const int64_t dv_at = b * A.dv.b + h * A.dv.h + v * A.dv.d;
    using Elem = typename N::Elem;
    const Elem *const kb = static_cast<const Elem *>(A.k.p) + b * A.k.b + hk * A.k.h;
    const Elem *const qb = static_cast<const Elem *>(A.q.p) + b * A.q.b + hk * A.q.h;

    St S;
    S.zero();
    if (A.g_last) S.load(A.g_last + bh * A.key * A.value, wave, lane, v_first, A.key, A.value);
    S.to_lds(state, wave, lane);
    clear(scores);
    for (int64_t n = A.chunks - 1; n >= 0; --n) {
        const int64_t t0 = n * C, item = bh * A.chunks + n;
        const StepGates gates = load_gates<C>(A, b, h, t0);
        In k_raw, q_raw;
        k_raw.load(A.k, kb, 0, t0, A.key, A.T);
        q_raw.load(A.q, qb, 0, t0, A.key, A.T);
        S.store(A.dstates + item * DK * A.value_pad, wave, lane, v_first, DK, A.value_pad, A.value_pad);
        for (int r1 = gates.rows; r1 > 0;) {
            const int r0 = document_start(gates.cut, r1);
            k_raw.store(keys, r0, r1);
            q_raw.store(queries, r0, r1);
            if (wave == 0) write_factors(F, gates, r0, r1);
            f32x4 value = {0.0f, 0.0f, 0.0f, 0.0f}, go = value;
            if (has_v) {
                value = load_steps<HALF>(A.v.p, v_at + (t0 + tt + row4) * A.v.t, A.v.t, r0 - tt - row4,
                                         r1 - tt - row4);
                if (A.o.p)
                    go = load_steps<false>(A.o.p, o_at + (t0 + tt + row4) * A.o.t, A.o.t, r0 - tt - row4,
                                           r1 - tt - row4);
                go = only_steps(go, tt + row4, r0, r1);
                value = only_steps(value, tt + row4, r0, r1);
            }
            if (owner) store4(out, vt + col, tt + row4, go);
            __syncthreads();

            f32x4 w = {0.0f, 0.0f, 0.0f, 0.0f};
            if (owner) {
#pragma unroll
                for (int d = 0; d < DK; d += 32) w = mma(w, operand<!TF>(keys, tt, d), operand<true>(state, vt, d));
                const f32x4 start = four(F.start + tt + row4), end = four(F.end + tt + row4);
                f32x4 g;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] *= end[e];
                    g[e] = A.scale * start[e] * go[e];
                }
                store4(out_q, vt + col, tt + row4, only_steps(g, tt + row4, r0, r1));
            }
            // P by rows of the keys' steps t: its tile (t, s), s >= t, four s side by side
            for (int p = wave; p < TT * (TT + 1) / 2; p += kWaves) {
                int si, ti;
                lower_pair(p, si, ti);
                si *= 16, ti *= 16;
                f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int d = 0; d < DK; d += 32) c = mma(c, operand<!TF>(queries, si, d), operand<!TF>(keys, ti, d));
                const int t = ti + col, s = si + row4;
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = s + e >= t ? A.scale * c[e] * decay_between(F, s + e, t) : 0.0f;
                store4(scores, t, s, c);
            }
            __syncthreads();

            if (owner) {
#pragma unroll
                for (int s = 0; s < C; s += 32)
                    if (s + 32 > tt) w = mma(w, operand<true>(scores, tt, s), operand<true>(out, vt, s));
                store4(write, vt + col, tt + row4, only_steps(w, tt + row4, r0, r1));
            }
            __syncthreads();

            if (owner) {
                f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < C; s += 32)
                    if (s + 32 > tt) x = mma(x, operand_of(A.inverse_t, item, tt, s, N()), operand<true>(write, vt, s));
                x = only_steps(x, tt + row4, r0, r1);
                const f32x4 start = four(F.start + tt + row4), beta = four(F.beta + tt + row4);
                float *p = A.x + (item * C + tt + row4) * A.value_pad + v_first + vt + col;
                f32x4 c, bx, xv;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (tt + row4 + e >= r0 && tt + row4 + e < r1) p[e * A.value_pad] = x[e];
                    bx[e] = beta[e] * x[e];
                    c[e] = -start[e] * bx[e];
                    xv[e] = x[e] * value[e];
                }
                store4(carry, vt + col, tt + row4, only_steps(c, tt + row4, r0, r1));
                if (has_v)
                    store_steps<HALF>(A.dv.p, dv_at + (t0 + tt + row4) * A.dv.t, A.dv.t, r0 - tt - row4,
                                      r1 - tt - row4, bx);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int o = 1; o < 16; o *= 2) xv[e] += __shfl_xor(xv[e], o);
                    if (col == 0) products[(tt + row4 + e) * VT + vt / 16] = xv[e];
                }
            }
            __syncthreads();

            if ((int)threadIdx.x >= r0 && (int)threadIdx.x < r1) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < VT; ++i) s += products[threadIdx.x * VT + i];
                A.xv[(item * C + threadIdx.x) * A.blocks + block] = s;
            }
            if (gates.cut >> r0 & 1) {  // the state before this document's is no part of it
                S.zero();
            } else {
                const float across = F.across[0];
#pragma unroll
                for (int i = 0; i < St::kCount; ++i) {
                    int d0, v0;
                    if (!St::tile(i, wave, d0, v0)) break;
                    f32x4 c;
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = across * S.s[i][e];
#pragma unroll
                    for (int s = 0; s < C; s += 32) {
                        c = mma(c, operand<TF>(queries, d0, s), operand<true>(out_q, v0, s));
                        c = mma(c, operand<TF>(keys, d0, s), operand<true>(carry, v0, s));
                    }
                    S.s[i] = c;
                }
            }
            S.to_lds(state, wave, lane);
            __syncthreads();
            r1 = r0;
        }
    }
    if (A.dh0) S.store(A.dh0 + bh * A.key * A.value, wave, lane, v_first, A.key, A.value, A.value);
}

// -------------------------------------------------------- the gradients ---

// A workgroup for a key head's chunk: for each value head that shares it, with
// S the state before the chunk and dS' the gradient of the one behind it,
//     U = dO S^T,  Y = X S^T,  Z = W dS'^T                     [C][dk]
//     E_ij = scale (dO_i . w_j) D_ij, j <= i;   H_ij = -(X_i . w_j) D_ij, j < i
//     dQ_i = scale exp(G_i) U_i + sum_j E_ij k_j
//     dK_j = exp(G_C - G_j) Z_j - b_j exp(G_j) Y_j + sum_i E_ij q_i
//            + sum_i b_i H_ij k_i + sum_i b_j H_ji k_i
//     db_i = X_i . v_i - exp(G_i) k_i . Y_i + sum_j H_ij (k_i . k_j)
// and the gradient of G, of which a log decay's is the sum from its step on:
//     dG_i = scale exp(G_i) q_i . U_i - b_i exp(G_i) k_i . Y_i - z_i
//            + sum_j B_ij - sum_j B_ji,  B_ij = E_ij (q_i . k_j) + b_i H_ij (k_i . k_j),
//     z_i = exp(G_C - G_i) k_i . Z_i,  dG_C += sum_i z_i + exp(G_C) <S, dS'>.
template <bool HALF, int DK, bool TF>
__global__ void __launch_bounds__(kThreads) delta_grad_kernel(Args A)
{
    using N = Num<HALF>;
    using Wide = typename N::Wide;
    constexpr int C = N::kChunk, TT = C / 16, DT = DK / 16, kPairs = TT * (TT + 1) / 2;
    constexpr int kD = DT < kWaves ? DT : kWaves, kT = kWaves / kD;  // waves along channels and steps
    constexpr int ND = DT / kD, NT = TT / kT, NP = (kPairs + kWaves - 1) / kWaves;
    static_assert(ND * kD == DT && NT * kT == TT, "whole tiles a wave");
    constexpr int VB = 32;  // columns of the values at a time
    using In = Pieces<HALF, DK, TF, kThreads>;
    __shared__ typename In::Lds keys, queries;
    __shared__ WideTile<HALF, C, C> e_t, h_t;  // E and b H by columns
    __shared__ WideTile<HALF, TF ? VB : C, TF ? C : VB> out;
    __shared__ WideTile<HALF, C, VB> xs, ws;
    __shared__ Factors<C> F;
    __shared__ float row_sum[kPairs * 16], col_sum[kPairs * 16], h_sum[kPairs * 16];
    __shared__ float dots[3][kD][C], inner[kWaves];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, row4 = 4 * (lane / 16), col = lane % 16;
    const int64_t n = blockIdx.x % A.chunks, bk = blockIdx.x / A.chunks, b = bk / A.Hk, hk = bk % A.Hk;
    const int64_t t0 = n * C;
    const int group = A.Hv / A.Hk;
    const int wd = 16 * ND * (wave % kD), wt = 16 * NT * (wave / kD);  // the wave's first channel and step
    using Elem = typename N::Elem;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

    In k_raw, q_raw;
    k_raw.load(A.k, static_cast<const Elem *>(A.k.p) + b * A.k.b + hk * A.k.h, 0, t0, A.key, A.T);
    q_raw.load(A.q, static_cast<const Elem *>(A.q.p) + b * A.q.b + hk * A.q.h, 0, t0, A.key, A.T);
    clear(e_t);
    clear(h_t);
    f32x4 dq[NT][ND], dk[NT][ND];
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int c = 0; c < ND; ++c) dq[a][c] = dk[a][c] = zero;
    for (int head = 0; head < group; ++head) {
        const int64_t h = hk * group + head, bh = b * A.Hv + h, item = bh * A.chunks + n;
        const StepGates gates = load_gates<C>(A, b, h, t0);
        const float *const s_before = A.states + item * DK * A.value_pad;
        const float *const s_behind = A.dstates + item * DK * A.value_pad;
        for (int r0 = 0, r1; r0 < gates.rows; r0 = r1) {
            r1 = document_end(gates.cut, r0, gates.rows);
            const bool before = !(gates.cut >> r0 & 1), behind = r1 == gates.rows;
            __syncthreads();
            k_raw.store(keys, r0, r1);
            q_raw.store(queries, r0, r1);
            if (wave == 0) write_factors(F, gates, r0, r1);

            f32x4 U[NT][ND], Y[NT][ND], Z[NT][ND], ow[NP], xw[NP];
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int c = 0; c < ND; ++c) U[a][c] = Y[a][c] = Z[a][c] = zero;
#pragma unroll
            for (int m = 0; m < NP; ++m) ow[m] = xw[m] = zero;
            float ss = 0.0f;
            for (int v0 = 0; v0 < A.value; v0 += VB) {
                __syncthreads();
                for (int u = threadIdx.x; u < C * VB / 4; u += kThreads) {
                    const int row = u / (VB / 4), v4 = u % (VB / 4) * 4;
                    f32x4 x = zero, w = zero;
                    if (row >= r0 && row < r1) {
                        const int64_t at = (item * C + row) * A.value_pad + v0 + v4;
                        x = four(A.x + at);
                        w = four(A.w + at);
                    }
                    store4(xs, row, v4, x);
                    store4(ws, row, v4, w);
                    x = zero;
                    if constexpr (TF) {
                        const int v = u / (C / 4), t4 = u % (C / 4) * 4;
                        if (A.o.p && v0 + v < A.value)
                            x = load_steps<false>(A.o.p, b * A.o.b + h * A.o.h + (v0 + v) * A.o.d + (t0 + t4) * A.o.t,
                                                  A.o.t, r0 - t4, r1 - t4);
                        store4(out, v, t4, only_steps(x, t4, r0, r1));
                    } else {
                        if (A.o.p && row >= r0 && row < r1)
                            x = load_steps<false>(A.o.p, b * A.o.b + h * A.o.h + (v0 + v4) * A.o.d + (t0 + row) * A.o.t,
                                                  A.o.d, 0, A.value - v0 - v4);
                        store4(out, row, v4, x);
                    }
                }
                __syncthreads();
#pragma unroll
                for (int c = 0; c < ND; ++c) {
                    const int64_t at = (int64_t)(wd + 16 * c + col) * A.value_pad + v0 + 8 * (lane / 16);
                    float s[8], g[8];
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const f32x4 p = before ? four(s_before + at + j) : zero;
                        const f32x4 q = behind ? four(s_behind + at + j) : zero;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[j + e] = p[e];
                            g[j + e] = q[e];
                            ss = fmaf_(p[e], q[e], ss);
                        }
                    }
                    const Wide sw = split(s, Wide()), gw = split(g, Wide());
#pragma unroll
                    for (int a = 0; a < NT; ++a) {
                        U[a][c] = mma(U[a][c], operand<!TF>(out, wt + 16 * a, 0), sw);
                        Y[a][c] = mma(Y[a][c], operand<true>(xs, wt + 16 * a, 0), sw);
                        Z[a][c] = mma(Z[a][c], operand<true>(ws, wt + 16 * a, 0), gw);
                    }
                }
#pragma unroll
                for (int m = 0; m < NP; ++m) {
                    const int p = wave + kWaves * m;
                    if (p >= kPairs) break;
                    int it, jt;
                    lower_pair(p, it, jt);
                    const Wide w = operand<true>(ws, 16 * jt, 0);
                    ow[m] = mma(ow[m], operand<!TF>(out, 16 * it, 0), w);
                    xw[m] = mma(xw[m], operand<true>(xs, 16 * it, 0), w);
                }
            }

            // E and H, and the sums of their rows and columns
#pragma unroll
            for (int m = 0; m < NP; ++m) {
                const int p = wave + kWaves * m;
                if (p >= kPairs) break;
                int it, jt;
                lower_pair(p, it, jt);
                it *= 16, jt *= 16;
                f32x4 qk = zero, kk = zero;
#pragma unroll
                for (int d = 0; d < DK; d += 32) {
                    const auto kj = operand<!TF>(keys, jt, d);
                    qk = mma(qk, operand<!TF>(queries, it, d), kj);
                    kk = mma(kk, operand<!TF>(keys, it, d), kj);
                }
                const int i = it + row4, j = jt + col;
                const f32x4 beta = four(F.beta + i);
                f32x4 E, H, hs, bs;
                float cs = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool mine = i + e >= r0 && i + e < r1 && j >= r0 && j <= i + e;
                    const float d = decay_between(F, i + e, j);
                    E[e] = mine ? A.scale * ow[m][e] * d : 0.0f;
                    H[e] = mine && j < i + e ? -xw[m][e] * d : 0.0f;
                    hs[e] = mine ? H[e] * kk[e] : 0.0f;
                    bs[e] = mine ? fmaf_(E[e], qk[e], beta[e] * hs[e]) : 0.0f;
                    H[e] *= beta[e];
                    cs += bs[e];
                }
                store4(e_t, j, i, E);
                store4(h_t, j, i, H);
#pragma unroll
                for (int o = 1; o < 16; o *= 2)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        hs[e] += __shfl_xor(hs[e], o);
                        bs[e] += __shfl_xor(bs[e], o);
                    }
                cs += __shfl_xor(cs, 16);
                cs += __shfl_xor(cs, 32);
                if (col == 0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h_sum[p * 16 + row4 + e] = hs[e];
                        row_sum[p * 16 + row4 + e] = bs[e];
                    }
                }
                if (lane < 16) col_sum[p * 16 + lane] = cs;
            }
            // the rows' products with U, Y and Z, and these as the gradients' first parts
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                const int t = wt + 16 * a + row4;
                const f32x4 start = four(F.start + t), end = four(F.end + t), beta = four(F.beta + t);
                f32x4 qu = zero, ky = zero, kz = zero;
#pragma unroll
                for (int c = 0; c < ND; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int d = wd + 16 * c + col;
                        const int at = TF ? d * In::Lds::kPitch + t + e : (t + e) * In::Lds::kPitch + d;
                        const float q = load_gate<HALF>(queries.at, at), k = load_gate<HALF>(keys.at, at);
                        qu[e] = fmaf_(q, U[a][c][e], qu[e]);
                        ky[e] = fmaf_(k, Y[a][c][e], ky[e]);
                        kz[e] = fmaf_(k, Z[a][c][e], kz[e]);
                        U[a][c][e] *= A.scale * start[e];
                        Z[a][c][e] = end[e] * Z[a][c][e] - beta[e] * start[e] * Y[a][c][e];
                    }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
#pragma unroll
                    for (int o = 1; o < 16; o *= 2) {
                        qu[e] += __shfl_xor(qu[e], o);
                        ky[e] += __shfl_xor(ky[e], o);
                        kz[e] += __shfl_xor(kz[e], o);
                    }
                    if (col == 0) {
                        dots[0][wave % kD][t + e] = qu[e];
                        dots[1][wave % kD][t + e] = ky[e];
                        dots[2][wave % kD][t + e] = kz[e];
                    }
                }
            }
            if (wt != 0) ss = 0.0f;  // another wave's channels
#pragma unroll
            for (int o = 1; o < kWave; o *= 2) ss += __shfl_xor(ss, o);
            if (lane == 0) inner[wave] = ss;
            __syncthreads();

#pragma unroll
            for (int a = 0; a < NT; ++a) {
                const int t = wt + 16 * a;
#pragma unroll
                for (int c = 0; c < ND; ++c) {
                    const int d = wd + 16 * c;
#pragma unroll
                    for (int s = 0; s < C; s += 32) {
                        const auto k = operand<TF>(keys, d, s);
                        if (s <= t) {
                            U[a][c] = mma(U[a][c], operand<false>(e_t, t, s), k);
                            Z[a][c] = mma(Z[a][c], operand<false>(h_t, t, s), k);
                        }
                        if (s + 32 > t) {
                            Z[a][c] = mma(Z[a][c], operand<true>(e_t, t, s), operand<TF>(queries, d, s));
                            Z[a][c] = mma(Z[a][c], operand<true>(h_t, t, s), k);
                        }
                    }
                    const f32x4 u = only_steps(U[a][c], t + row4, r0, r1), z = only_steps(Z[a][c], t + row4, r0, r1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dq[a][c][e] += u[e];
                        dk[a][c][e] += z[e];
                    }
                }
            }
            if (wave == 0) {
                const int row = lane;
                const bool mine = row >= r0 && row < r1;
                double dG = 0.0, z = 0.0;
                if (mine) {
                    const int tile = row / 16;
                    float qu = 0.0f, ky = 0.0f, kz = 0.0f, hs = 0.0f, xv = 0.0f;
                    for (int w = 0; w < kD; ++w) {
                        qu += dots[0][w][row];
                        ky += dots[1][w][row];
                        kz += dots[2][w][row];
                    }
                    for (int j = 0; j <= tile; ++j) {
                        const int p = (tile * (tile + 1) / 2 + j) * 16 + row % 16;
                        hs += h_sum[p];
                        dG += row_sum[p];
                    }
                    for (int i = tile; i < TT; ++i) dG -= col_sum[(i * (i + 1) / 2 + tile) * 16 + row % 16];
                    for (int j = 0; j < A.blocks; ++j) xv += A.xv[(item * C + row) * A.blocks + j];
                    const float y = F.start[row] * ky;
                    z = (double)F.end[row] * kz;
                    dG += (double)(A.scale * F.start[row]) * qu - (double)F.beta[row] * y - z;
                    A.dbeta[bh * A.T + t0 + row] = xv - y + hs;
                }
                double all = z, suffix;
#pragma unroll
                for (int o = 1; o < kWave; o *= 2) all += __shfl_xor(all, o);
                if (row == r1 - 1) {
                    double inside = 0.0;
                    for (int w = 0; w < kWaves; ++w) inside += inner[w];
                    dG += all + (double)F.across[0] * inside;
                }
                suffix = dG;
#pragma unroll
                for (int o = 1; o < kWave; o *= 2) {
                    const double after = __shfl_down(suffix, o);
                    if (row + o < kWave) suffix += after;
                }
                if (mine && A.ddecay) A.ddecay[bh * A.T + t0 + row] = gates.cut >> row & 1 ? 0.0f : (float)suffix;
            }
        }
    }
    const int64_t dq_at = b * A.dq.b + hk * A.dq.h, dk_at = b * A.dk.b + hk * A.dk.h;
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int c = 0; c < ND; ++c) {
            const int d = wd + 16 * c + col;
            const int64_t t = t0 + wt + 16 * a + row4;
            const int left = (int)(A.T - t < 4 ? A.T - t : 4);
            if (d >= A.key || left <= 0) continue;
            store_steps<HALF>(A.dq.p, dq_at + d * A.dq.d + t * A.dq.t, A.dq.t, 0, left, dq[a][c]);
            store_steps<HALF>(A.dk.p, dk_at + d * A.dk.d + t * A.dk.t, A.dk.t, 0, left, dk[a][c]);
        }
}

}  // namespace delta
}  // namespace pararnn
