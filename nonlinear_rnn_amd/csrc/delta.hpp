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
// Times in these files are of the kernel under the kernel trace, both sides of a
// choice in the same run; from run to run they differ by a tenth (the first calls
// are the slow ones), so a call may take less than its kernels' times together.
//
// Documents.  A step where a document starts (its reset flag, or a log decay
// below kForget, whose exponential float32 does not hold) keeps nothing of the
// state, whatever is in it.  A chunk that holds several documents is visited
// once for each, with the rows of the others zero.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "delta_step.hpp"
#include "elements.hpp"
#include "pararnn.h"

namespace pararnn {
namespace delta {

constexpr int kWaves = 8, kThreads = kWaves * kWave;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
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
    int32_t value_pad, blocks;        // columns of the workspace's rows; the chains' workgroups a head
    float scale;
    // segments of `per` chunks, chained at once (1: the whole chain)
    int32_t segments, per;
    int32_t ends;      // only the segments' maps: their ends from zero, and from the identity
    // workspace
    struct Fragment *inverse, *inverse_t;  // [b h][chunk][slot] operands
    float *states, *dstates;          // [b h][chunk][value_pad][DK]
    float *w, *x;                     // [b h][chunk][value_pad][C]
    float *maps;                      // [b h][segment][DK][value_pad + key_pad]: ends from zero, from the identity
    float *marks;                     // [b h][segment][DK][value_pad]: the state before, the gradient behind
    int32_t *cuts;                    // [b h][segment]: whether a document starts in it
    int32_t key_pad;                  // `key`, whole tiles
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

// A product as the instructions it takes, so that those of several results can take
// turns: one result's wait for each other.  kParts of them, the smallest terms first.
template <class A, class B>
struct Product;
template <>
struct Product<bf16x8, bf16x8> {
    static constexpr int kParts = 1;
    static __device__ __forceinline__ f32x4 part(int, f32x4 c, bf16x8 a, bf16x8 b)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Product<bf16x8, Bf::Wide> {
    static constexpr int kParts = 2;
    static __device__ __forceinline__ f32x4 part(int i, f32x4 c, bf16x8 a, const Bf::Wide &b)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, i == 0 ? b.lo : b.hi, c, 0, 0, 0);
    }
};
template <>
struct Product<Bf::Wide, bf16x8> {
    static constexpr int kParts = 2;
    static __device__ __forceinline__ f32x4 part(int i, f32x4 c, const Bf::Wide &a, bf16x8 b)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(i == 0 ? a.lo : a.hi, b, c, 0, 0, 0);
    }
};
template <>
struct Product<Bf::Wide, Bf::Wide> {
    static constexpr int kParts = 3;
    static __device__ __forceinline__ f32x4 part(int i, f32x4 c, const Bf::Wide &a, const Bf::Wide &b)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(i == 0 ? a.lo : a.hi, i == 1 ? b.lo : b.hi, c, 0, 0, 0);
    }
};
// Eight instructions of 4 terms: the i-th takes the i-th element of every
// lane's eight, a permutation of the sum that both operands share.
template <>
struct Product<Fl::Exact, Fl::Exact> {
    static constexpr int kParts = 8;
    static __device__ __forceinline__ f32x4 part(int i, f32x4 c, const Fl::Exact &a, const Fl::Exact &b)
    {
        return __builtin_amdgcn_mfma_f32_16x16x4f32(a.x[i], b.x[i], c, 0, 0, 0);
    }
};
template <class A, class B>
__device__ __forceinline__ f32x4 mma(f32x4 c, const A &a, const B &b)
{
#pragma unroll
    for (int i = 0; i < Product<A, B>::kParts; ++i) c = Product<A, B>::part(i, c, a, b);
    return c;
}
// c_t + a_t b for several t
template <class A, class B, int M>
__device__ __forceinline__ void mma_rows(f32x4 (&c)[M], const A (&a)[M], const B &b)
{
#pragma unroll
    for (int i = 0; i < Product<A, B>::kParts; ++i)
#pragma unroll
        for (int t = 0; t < M; ++t) c[t] = Product<A, B>::part(i, c[t], a[t], b);
}

// Results that are used behind a branch.  They can be read 8 (bfloat16) or 10
// wait states after the instruction; the compiler does not count these along a
// branch that is taken at once (rows 3 of 4 came out without their last terms).
template <int M>
__device__ __forceinline__ void settle(f32x4 (&x)[M])
{
    static_assert(M == 1 || M == 2 || M == 4 || M == 8 || M == 16, "one statement for all");
    if constexpr (M == 16)
        asm volatile("s_nop 9"
                     : "+v"(x[0]), "+v"(x[1]), "+v"(x[2]), "+v"(x[3]), "+v"(x[4]), "+v"(x[5]), "+v"(x[6]), "+v"(x[7]),
                       "+v"(x[8]), "+v"(x[9]), "+v"(x[10]), "+v"(x[11]), "+v"(x[12]), "+v"(x[13]), "+v"(x[14]),
                       "+v"(x[15]));
    else if constexpr (M == 8)
        asm volatile("s_nop 9"
                     : "+v"(x[0]), "+v"(x[1]), "+v"(x[2]), "+v"(x[3]), "+v"(x[4]), "+v"(x[5]), "+v"(x[6]), "+v"(x[7]));
    else if constexpr (M == 4)
        asm volatile("s_nop 9" : "+v"(x[0]), "+v"(x[1]), "+v"(x[2]), "+v"(x[3]));
    else if constexpr (M == 2)
        asm volatile("s_nop 9" : "+v"(x[0]), "+v"(x[1]));
    else
        asm volatile("s_nop 9" : "+v"(x[0]));
}

// A stride as if it were new here: what a rare path makes of it is then computed
// there, and not kept in registers through the loops around.
__device__ __forceinline__ int64_t afresh(int64_t stride)
{
    asm volatile("" : "+s"(stride));
    return stride;
}
// The same for the addresses in LDS: without it the loops keep dozens of them in
// registers, spill some, and every reload waits for the loads under way.
template <class T>
__device__ __forceinline__ T &lds_afresh(T &shared)
{
    auto *p = (__attribute__((address_space(3))) T *)&shared;
    asm volatile("" : "+s"(p));
    return *(T *)p;
}
__device__ __forceinline__ int lane_afresh(int lane)
{
    asm volatile("" : "+v"(lane));
    return lane;
}

// Two float32 as the bfloat16 next to them and the ones next to what that leaves.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t rounded(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ void split(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = rounded(a, b);
    lo = rounded(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
__device__ __forceinline__ Bf::Wide split(const float (&x)[8], Bf::Wide)
{
    Words4 hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h, l;
        split(x[2 * j], x[2 * j + 1], h, l);
        hi[j] = h;
        lo[j] = l;
    }
    return {__builtin_bit_cast(bf16x8, hi), __builtin_bit_cast(bf16x8, lo)};
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

// Operands of a 16x16 product over 32 terms: lane l holds row (or column) i0 +
// l % 16 and, with g = l / 16, the terms k0 + 4 g .. + 3 and k0 + 16 + 4 g .. + 3.
// This order is that of two results one above the other (lane l of a result
// holds column l % 16, rows 4 g .. + 3), so what a wave has computed it can
// multiply with, without the LDS.
// along: the terms lie side by side in the tile's rows.
__device__ __forceinline__ bf16x8 operand_along(const uint16_t *at, int pitch, int i0, int k0)
{
    const int lane = threadIdx.x % kWave;
    const uint16_t *p = at + (i0 + lane % 16) * pitch + k0 + 4 * (lane / 16);
    bf16x8 r;
    __builtin_memcpy(&r, p, 8);
    __builtin_memcpy(reinterpret_cast<char *>(&r) + 8, p + 16, 8);
    return r;
}
__device__ __forceinline__ Fl::Exact operand_along(const float *at, int pitch, int i0, int k0)
{
    const int lane = threadIdx.x % kWave;
    const float *p = at + (i0 + lane % 16) * pitch + k0 + 4 * (lane / 16);
    Fl::Exact r;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p + 4 * j);
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
    const uint16_t *p = at + (k0 + 4 * (lane / 16) + i / 4) * pitch + i0 + 4 * (i % 4);
    const s16x4 a = read_transposed(p), b = read_transposed(p + 16 * pitch);
    bf16x8 r;
    __builtin_memcpy(&r, &a, 8);
    __builtin_memcpy(reinterpret_cast<char *>(&r) + 8, &b, 8);
    return r;
}
__device__ __forceinline__ Fl::Exact operand_across(const float *at, int pitch, int i0, int k0)
{
    const int lane = threadIdx.x % kWave;
    const float *p = at + (k0 + 4 * (lane / 16)) * pitch + i0 + lane % 16;
    Fl::Exact r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.x[j] = p[(j < 4 ? j : 12 + j) * pitch];
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
// One value.
template <bool HALF, int ROWS, int COLS>
__device__ __forceinline__ float value_at(const WideTile<HALF, ROWS, COLS> &t, int row, int col)
{
    const int at = row * t.kPitch + col;
    if constexpr (HALF)
        return __uint_as_float((uint32_t)t.at[at] << 16) + __uint_as_float((uint32_t)t.at[ROWS * t.kPitch + at] << 16);
    else
        return t.at[at];
}
// Four values side by side at (row, col), col a multiple of 4.
template <bool HALF, int ROWS, int COLS>
__device__ __forceinline__ void store4(WideTile<HALF, ROWS, COLS> &t, int row, int col, f32x4 x)
{
    auto *p = t.at + row * t.kPitch + col;
    if constexpr (HALF) {
        uint32_t hi[2], lo[2];
        split(x[0], x[1], hi[0], lo[0]);
        split(x[2], x[3], hi[1], lo[1]);
        __builtin_memcpy(p, hi, 8);
        __builtin_memcpy(p + ROWS * t.kPitch, lo, 8);
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

// A wide operand as it lies in the lanes' registers, in LDS or in memory.
struct Fragment {
    uint4 a[kWave], b[kWave];  // the rounded values and what that leaves; of float32 the two halves
};
__device__ __forceinline__ void store_fragment(Fragment &f, const Bf::Wide &w)
{
    const int lane = threadIdx.x % kWave;
    __builtin_memcpy(&f.a[lane], &w.hi, 16);
    __builtin_memcpy(&f.b[lane], &w.lo, 16);
}
__device__ __forceinline__ void store_fragment(Fragment &f, const Fl::Wide &w)
{
    const int lane = threadIdx.x % kWave;
    __builtin_memcpy(&f.a[lane], w.x, 16);
    __builtin_memcpy(&f.b[lane], w.x + 4, 16);
}
__device__ __forceinline__ Bf::Wide load_fragment(const Fragment &f, Bf)
{
    const uint4 a = f.a[threadIdx.x % kWave], b = f.b[threadIdx.x % kWave];
    Bf::Wide w;
    __builtin_memcpy(&w.hi, &a, 16);
    __builtin_memcpy(&w.lo, &b, 16);
    return w;
}
__device__ __forceinline__ Fl::Wide load_fragment(const Fragment &f, Fl)
{
    const uint4 a = f.a[threadIdx.x % kWave], b = f.b[threadIdx.x % kWave];
    Fl::Wide w;
    __builtin_memcpy(w.x, &a, 16);
    __builtin_memcpy(w.x + 4, &b, 16);
    return w;
}
// Two results one above the other as an operand.
template <bool HALF>
__device__ __forceinline__ typename Num<HALF>::Wide stacked(f32x4 a, f32x4 b)
{
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return split(x, typename Num<HALF>::Wide());
}
// Operands of a triangular matrix [C][C], 16 rows and 32 terms each: those that
// are not zero, row by row.  lower: terms up to the row; upper: from the row on.
template <int C>
struct Slots {
    static constexpr int kCount = C == 64 ? 6 : 2;
    static_assert(C == 64 || C == 32, "chunks");
    static constexpr int lower(int row, int terms) { return C == 32 || row < 2 ? row : 2 * row - 2 + terms; }
    static constexpr int upper(int row, int terms) { return C == 32 ? row : row < 2 ? 2 * row + terms : 2 + row; }
    static constexpr bool in_lower(int row, int terms) { return 2 * terms <= row; }
    static constexpr bool in_upper(int row, int terms) { return 2 * terms + 1 >= row; }
};

// --------------------------------------------------- inputs and documents ---

// A chunk of queries or keys, DK channels of C steps, as 16-byte pieces in
// THREADS threads' registers and then in LDS, the steps side by side (TF) or the
// channels.
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
    // base: the head's first element; d0: the first channel; t0: the chunk's first
    // step.  Nothing here depends on the lane but addresses, which are kept inside
    // the tensor, so that all loads are under way at once; store() drops what lies
    // outside.
    __device__ __forceinline__ void load(const Plane &x, const Elem *base, int d0, int64_t t0, int key, int64_t T,
                                         int tid)
    {
        constexpr int kRows = THREADS / kPerRow;  // between a thread's pieces
        static_assert(THREADS % kPerRow == 0, "a thread's pieces in one column");
        const int row = tid / kPerRow, col = tid % kPerRow * E;
        const int64_t stride = TF ? x.d : x.t;
        if (t0 + C <= T && (TF ? x.t == 1 : x.d == 1 && key % E == 0) && stride < 1 << 24) {
            // one address for the workgroup, 32 bits a lane
            const char *p = reinterpret_cast<const char *>(base + (TF ? d0 * x.d + t0 : d0 + t0 * x.t));
            const uint32_t at = (uint32_t)(row * (int)stride + col) * (uint32_t)sizeof(Elem);
            const bool all = d0 + DK <= key;
#pragma unroll
            for (int n = 0; n < kCount; ++n) {
                // (a piece whose channels are not there takes the first ones)
                const bool here = all || (TF ? d0 + row + n * kRows < key : d0 + col < key);
                const Words4 w = *reinterpret_cast<const Words4Any *>(
                    p + (here ? at : 0u) + (TF && !here ? 0 : n * kRows * stride * (int64_t)sizeof(Elem)));
                u[n] = make_uint4(w.x, w.y, w.z, w.w);
            }
            return;
        }
        const int64_t by_d = afresh(x.d), by_t = afresh(x.t), last = afresh(T) - 1;
        const int top = (int)afresh(key) - 1;
#pragma unroll
        for (int n = 0; n < kCount; ++n) {
            const int d = d0 + (TF ? row + n * kRows : col);
            const int64_t t = t0 + (TF ? col : row + n * kRows);
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int de = min(TF ? d : d + e, top);
                const uint32_t v = element(base + de * by_d + min(TF ? t + e : t, last) * by_t);
                if constexpr (HALF)
                    w[e / 2] |= v << (16 * (e % 2));
                else
                    w[e] = v;
            }
            u[n] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    // To LDS; steps outside r0 .. r1 - 1 of the chunk and channels from `key` on
    // (counted from the tile's first) are zero.
    __device__ __forceinline__ void store(Lds &lds, int r0, int r1, int key, int tid) const
    {
        constexpr int kRows = THREADS / kPerRow;
        const int row = tid / kPerRow, col = tid % kPerRow * E;
        auto *const p = lds.at + row * lds.kPitch + col;
        if (r0 == 0 && r1 == C && key >= DK) {
#pragma unroll
            for (int n = 0; n < kCount; ++n) *reinterpret_cast<uint4 *>(p + n * kRows * lds.kPitch) = u[n];
            return;
        }
        const int first = TF ? r0 : 0, end = TF ? r1 : key;  // of the piece's own direction
#pragma unroll
        for (int n = 0; n < kCount; ++n) {
            uint32_t w[4] = {u[n].x, u[n].y, u[n].z, u[n].w};
            const int r = row + n * kRows;
            const bool out = TF ? r >= key : r < r0 || r >= r1;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const bool in = !out & (col + e >= first) & (col + e < end);
                if constexpr (HALF)
                    w[e / 2] &= in ? ~0u : e % 2 ? 0x0000ffffu : 0xffff0000u;
                else
                    w[e] = in ? w[e] : 0;
            }
            *reinterpret_cast<uint4 *>(p + n * kRows * lds.kPitch) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// A wave's 16 columns of C steps as results hold them: lane l has column l % 16
// and, of each 16 steps, 4 (l / 16) .. + 3.  Kept as loaded, so that nothing waits
// for them before their use.  As above, all loads are under way at once.
template <bool HALF, int C>
struct Columns {
    static constexpr int TT = C / 16;
    using Elem = typename Num<HALF>::Elem;
    uint32_t w[TT][HALF ? 2 : 4];
    // base: the lane's column (one that is there); t0: the chunk's first step
    __device__ __forceinline__ void load(const Elem *base, int64_t step, int64_t t0, int64_t T)
    {
        const int row4 = threadIdx.x % kWave / 16 * 4;
        if (t0 + C <= T && step == 1) {
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                const Elem *p = base + t0 + 16 * i + row4;
                if constexpr (HALF) {
                    const Words2 v = *reinterpret_cast<const Words2Any *>(p);
                    w[i][0] = v.x, w[i][1] = v.y;
                } else {
                    const Words4 v = *reinterpret_cast<const Words4Any *>(p);
                    w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
                }
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            const int64_t t = t0 + 16 * i + row4;
            uint32_t e[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const Elem *p = base + min(t + r, T - 1) * step;
                if constexpr (HALF)
                    e[r] = *p;
                else
                    e[r] = __float_as_uint(*p);
            }
            if constexpr (HALF)
                w[i][0] = e[0] | e[1] << 16, w[i][1] = e[2] | e[3] << 16;
            else
                w[i][0] = e[0], w[i][1] = e[1], w[i][2] = e[2], w[i][3] = e[3];
        }
    }
    __device__ __forceinline__ f32x4 get(int i) const
    {
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (HALF)
                x[r] = __uint_as_float(r % 2 ? w[i][r / 2] & 0xffff0000u : w[i][r / 2] << 16);
            else
                x[r] = __uint_as_float(w[i][r]);
        }
        return x;
    }
};
// Four values at p, p + step, ...; those of `first` .. `end` - 1 are there.
__device__ __forceinline__ f32x4 load_four(const float *p, int64_t step, int first, int end)
{
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (r >= first && r < end) x[r] = p[r * step];
    return x;
}
// Four results to the lane's column: rows t .. t + 3, `step` elements apart, as far
// as they are rows r0 .. r1 - 1.  whole: they all are.
template <bool HALF>
__device__ __forceinline__ void store_column(typename Num<HALF>::Elem *base, int64_t step, int t, int r0, int r1,
                                             bool whole, f32x4 x)
{
    if (whole && step == 1) {
        if constexpr (HALF) {
            const Words2 w = {rounded(x[0], x[1]), rounded(x[2], x[3])};
            *reinterpret_cast<Words2Any *>(base + t) = w;
        } else {
            const Words4 w = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                              __float_as_uint(x[3])};
            *reinterpret_cast<Words4Any *>(base + t) = w;
        }
    } else {
        step = afresh(step);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (whole || (t + r >= r0 && t + r < r1)) store_gate<HALF>(base, (t + r) * step, x[r]);
    }
}

// Steps r0 .. r1 - 1 (whole: all) of a wave's columns to a workspace's rows of a
// chunk's steps.
template <int TT>
__device__ __forceinline__ void store_rows(float *p, int64_t v, int r0, int r1, bool whole, const f32x4 (&x)[TT])
{
#pragma unroll
    for (int t = 0; t < TT; ++t)
        store_column<false>(p + v * 16 * TT, 1, 16 * t + threadIdx.x % kWave / 16 * 4, r0, r1, whole, x[t]);
}

// The gates of a chunk's steps, one a lane; the same in every wave.
struct StepGates {
    float g, beta;
    uint64_t cut;  // steps that keep nothing of the state before them
    int rows;      // the chunk's steps
};
struct LoadedGates {
    float g, beta;
    uint32_t reset;
};
// (lanes without a step read another's, and use_gates() drops it)
__device__ __forceinline__ LoadedGates fetch_gates(const Args &A, int64_t b, int64_t h, int64_t t0)
{
    const int64_t t = min(t0 + threadIdx.x % kWave, A.T - 1), at = b * A.gate_b + h * A.gate_h + t * A.gate_t;
    LoadedGates l = {0.0f, A.beta[at], 0};
    if (A.decay) l.g = A.decay[at];
    if (A.resets) l.reset = A.resets[b * A.T + t];
    return l;
}
template <int C>
__device__ __forceinline__ StepGates use_gates(const Args &A, const LoadedGates &l, int64_t t0)
{
    const int lane = threadIdx.x % kWave;
    const bool here = lane < C && t0 + lane < A.T;
    return {here ? l.g : 0.0f, here ? l.beta : 0.0f, __ballot(here && (l.reset != 0 || l.g < kForget)),
            (int)(A.T - t0 < C ? A.T - t0 : C)};
}
template <int C>
__device__ __forceinline__ StepGates load_gates(const Args &A, int64_t b, int64_t h, int64_t t0)
{
    return use_gates<C>(A, fetch_gates(A, b, h, t0), t0);
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
// Sums over the lanes up to each lane: by rows of 16, then across them.
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double x)
{
    const uint64_t u = __double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return __longlong_as_double((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double sum_upto(double x)
{
    x += moved<0x111, 0xf>(x);  // from 1, 2, 4 and 8 lanes below
    x += moved<0x112, 0xf>(x);
    x += moved<0x114, 0xf>(x);
    x += moved<0x118, 0xf>(x);
    x += moved<0x142, 0xa>(x);  // the row's last lane to the next row
    x += moved<0x143, 0xc>(x);  // lane 31 to the upper half
    return x;
}
// Sums of the document's log decays (base 2) up to each step, from its first
// step in the chunk; steps of other documents take the value at their side.
__device__ __forceinline__ double decay_sum(const StepGates &s, int r0, int r1)
{
    const int lane = threadIdx.x % kWave;
    const bool mine = lane >= r0 && lane < r1 && !(s.cut >> lane & 1);
    return sum_upto(mine ? (double)s.g * 1.4426950408889634 : 0.0);
}
// What a visit's steps multiply with, in LDS.
template <int C>
struct alignas(16) Factors {
    float hi[C], lo[C];  // the decay's sum, in two floats
    float start[C];      // exp(G_i)
    float end[C];        // exp(G_C - G_i)
    float back[C];       // exp(-G_i), if all sums are near zero
    float beta[C];
    float across[4];     // exp(G_C)
};
// Within 2^+-kNear, where a factor exp(G_i - G_j) may be the product of two: with an
// exponential for each, 8 x 4096 x 8 heads take 231 us instead of 226, 4 x 16384 x 32
// heads 1157 instead of 1114.
constexpr double kNear = 32.0;
// 2^x, its argument's rounding made good
__device__ __forceinline__ float power_of_two(double x)
{
    const float hi = (float)x, f = ex2(hi);
    return fmaf_(f, 0.6931472f * (float)(x - hi), f);
}
// Returns whether all sums are near zero.
template <int C>
__device__ __forceinline__ bool write_factors(Factors<C> &F, const StepGates &s, int r0, int r1)
{
    const int lane = threadIdx.x % kWave;
    const double G = decay_sum(s, r0, r1), total = __shfl(G, kWave - 1);
    const bool near = !__ballot(!(fabs(G) <= kNear));
    if (lane < C) {
        const float hi = (float)G;
        F.hi[lane] = hi;
        F.lo[lane] = (float)(G - hi);
        F.start[lane] = power_of_two(G);
        F.end[lane] = power_of_two(total - G);
        F.back[lane] = power_of_two(-G);
        F.beta[lane] = lane >= r0 && lane < r1 ? s.beta : 0.0f;
    }
    if (lane == 0) F.across[0] = power_of_two(total);
    return near;
}
__device__ __forceinline__ f32x4 four(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }
// exp(G_i - G_j) for i .. i + 3, and for j .. j + 3.  An exponential takes as long
// as four products.
template <int C>
__device__ __forceinline__ f32x4 decays_from(const Factors<C> &F, int i, int j, bool near = false)
{
    if (near) return four(F.start + i) * F.back[j];
    const f32x4 hi = four(F.hi + i), lo = four(F.lo + i);
    const float h = F.hi[j], l = F.lo[j];
    f32x4 d;
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = ex2((hi[e] - h) + (lo[e] - l));
    return d;
}
template <int C>
__device__ __forceinline__ f32x4 decays_to(const Factors<C> &F, int i, int j, bool near = false)
{
    if (near) return four(F.back + j) * F.start[i];
    const f32x4 hi = four(F.hi + j), lo = four(F.lo + j);
    const float h = F.hi[i], l = F.lo[i];
    f32x4 d;
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = ex2((h - hi[e]) + (l - lo[e]));
    return d;
}
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

// Four waves for a head's chunk.  K K^T on the matrix cores, 64 channels at a
// time.  The 16x16 blocks of the diagonal are inverted column by column, a
// lane each; then inverses are joined two by two,
//     [L 0; B R]^-1 = [L^-1 0; -R^-1 B L^-1 R^-1],
// in float32 products, in the matrix's own place.  (A lane for a whole column of
// 64 needs every element of A in every lane: 500 wide LDS reads a chunk, or 1600
// spilled registers.)  Entries between documents are set to zero rather than
// computed.  Bound by vector instructions (650 a wave, twice that while every wave
// inverted a block and every element asked for its document): 4096 chunks of 64
// steps, 128 channels 38 us, 32768 of them 209 us, 0.7 GB at 3.2 TB/s.
constexpr int kInverseThreads = 4 * kWave;
template <bool HALF, bool TF>
__global__ void __launch_bounds__(kInverseThreads, 5) delta_inverse_kernel(Args A)
{
    using N = Num<HALF>;
    using S = Slots<N::kChunk>;
    constexpr int C = N::kChunk, TT = C / 16, kTiles = TT * (TT + 1) / 2, kPitch = C + 4, kMine = (kTiles + 3) / 4;
    using Keys = Pieces<HALF, 64, TF, kInverseThreads>;
    __shared__ union {
        typename Keys::Lds keys;
        struct {
            alignas(16) float m[C * kPitch], p[C / 2 * kPitch];  // by columns: A, then its inverse; a product
        };
    } sh;
    __shared__ Factors<C> F;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x % kWave, row4 = 4 * (lane / 16), col = lane % 16;
    const unsigned chunks = (unsigned)A.chunks, heads = (unsigned)A.Hv, shared = heads / (unsigned)A.Hk;
    const unsigned head = blockIdx.x / chunks;
    const int64_t item = blockIdx.x, n = blockIdx.x % chunks, b = head / heads, h = head % heads, t0 = n * C;
    const LoadedGates loaded = fetch_gates(A, b, h, t0);
    const auto *keys = static_cast<const typename N::Elem *>(A.k.p) + b * A.k.b + head % heads / shared * A.k.h;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

    f32x4 acc[kMine];
#pragma unroll
    for (int m = 0; m < kMine; ++m) acc[m] = zero;
    const int gates_rows = (int)min((int64_t)C, A.T - t0);
    Keys raw;
    raw.load(A.k, keys, 0, t0, A.key, A.T, threadIdx.x);
    for (int d0 = 0; d0 < A.key; d0 += 64) {
        __syncthreads();
        raw.store(sh.keys, 0, gates_rows, A.key - d0, threadIdx.x);
        if (d0 + 64 < A.key) raw.load(A.k, keys, d0 + 64, t0, A.key, A.T, threadIdx.x);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int p = wave + 4 * m;
            if (p >= kTiles) break;
            int i, j;
            lower_pair(p, i, j);
#pragma unroll
            for (int d = 0; d < 64; d += 32)
                acc[m] = mma(acc[m], operand<!TF>(sh.keys, 16 * i, d), operand<!TF>(sh.keys, 16 * j, d));
        }
    }
    const StepGates gates = use_gates<C>(A, loaded, t0);
    if (wave == 0) {  // every document's sums by themselves: a number that is not finite stays in its own
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
    const bool several = (gates.cut & ~1ull) != 0;  // documents
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int p = wave + 4 * m;
        if (p >= kTiles) break;
        int it, jt;
        lower_pair(p, it, jt);
        const int i = 16 * it + row4, j = 16 * jt + col;
        const f32x4 d = decays_from(F, i, j), beta = four(F.beta + i);
        f32x4 a;
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = i + r > j ? beta[r] * acc[m][r] * d[r] : 0.0f;
        if (several)
#pragma unroll
            for (int r = 0; r < 4; ++r) a[r] = joined(i + r, j) ? a[r] : 0.0f;
        *reinterpret_cast<f32x4 *>(sh.m + j * kPitch + i) = a;
    }
    __syncthreads();
    if (wave == 3 && lane < C) {  // all 16 x 16 blocks in one wave: the instructions bound this kernel
        const int first = lane - col;
        f32x4 m[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i / 4][i % 4] = i == col ? 1.0f : 0.0f;
#pragma unroll
        for (int l = 0; l < 15; ++l) {
            if (l < col) m[l / 4][l % 4] = 0.0f;  // also where an earlier document made it a NaN
#pragma unroll
            for (int i = (l + 1) / 4; i < 4; ++i) {
                const f32x4 a = four(sh.m + (first + l) * kPitch + first + 4 * i);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (4 * i + r > l) m[i][r] = fmaf_(-a[r], m[l / 4][l % 4], m[i][r]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) m[i][r] = 4 * i + r < col ? 0.0f : m[i][r];
            *reinterpret_cast<f32x4 *>(sh.m + (first + col) * kPitch + first + 4 * i) = m[i];
        }
    }
    // inverses of `size` blocks joined: a wave for a tile of the block below the diagonal
#pragma unroll
    for (int size = 1; size < TT; size *= 2) {
        const int per = size * size, at = wave / per * 2 * size, i = wave % per / size, j = wave % size;
        const bool mine = at < TT;
        __syncthreads();
        if (mine) {
            f32x4 c = zero;
            for (int l = j; l < size; ++l)
                c = block_mma(c, block_operand<false>(sh.m, kPitch, 16 * (at + size + i), 16 * (at + l)),
                              block_operand<true>(sh.m, kPitch, 16 * (at + j), 16 * (at + l)));
            *reinterpret_cast<f32x4 *>(sh.p + (16 * (at / 2 + j) + col) * kPitch + 16 * i + row4) = c;
        }
        __syncthreads();
        if (mine) {
            f32x4 c = zero;
            for (int l = 0; l <= i; ++l)
                c = block_mma(c, block_operand<false>(sh.m, kPitch, 16 * (at + size + i), 16 * (at + size + l)),
                              block_operand<true>(sh.p, kPitch, 16 * (at / 2 + j), 16 * l));
            *reinterpret_cast<f32x4 *>(sh.m + (16 * (at + j) + col) * kPitch + 16 * (at + size + i) + row4) = -c;
        }
    }
    __syncthreads();
    // as operands: its own rows, and for the backward pass its columns
    for (int f = wave; f < (A.inverse_t ? 2 : 1) * S::kCount; f += 4) {
        const bool columns = f >= S::kCount;
        const int s = columns ? f - S::kCount : f;
        int rt = s, kt = 0;
        if constexpr (C == 64) {
            rt = columns ? (s < 4 ? s / 2 : s - 2) : s < 2 ? s : s / 2 + 1;
            kt = columns ? (s < 4 ? s % 2 : 1) : s < 2 ? 0 : s % 2;
        }
        const int row = 16 * rt + col;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int k = 32 * kt + row4 + (e < 4 ? e : 12 + e), i = columns ? k : row, j = columns ? row : k;
            x[e] = i >= j ? sh.m[j * kPitch + i] : 0.0f;
            if (several && !joined(i, j)) x[e] = 0.0f;
        }
        Fragment *const out = (columns ? A.inverse_t : A.inverse) + item * S::kCount + s;
        store_fragment(*out, split(x, typename N::Wide()));
    }
}

// A state's 16 columns in a wave's registers, DT tiles of 16 channels.
template <int DK>
struct State {
    static constexpr int DT = DK / 16;
    f32x4 s[DT];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < DT; ++i) s[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // S <- across S + channels times w
    template <class Exact, class Wide, int KC>
    __device__ __forceinline__ void advance(float across, const Exact (&k)[KC][DT], const Wide (&w)[KC])
    {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[d][r] *= across;
#pragma unroll
        for (int i = 0; i < KC; ++i) mma_rows(s, k[i], w[i]);
    }
    // column j of the identity
    __device__ __forceinline__ void identity(int j)
    {
        const int row4 = threadIdx.x % kWave / 16 * 4;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[i][r] = 16 * i + row4 + r == j ? 1.0f : 0.0f;
    }
    // rows of `pitch` values; channels from `key` on, and all without `here`, are not there
    __device__ __forceinline__ void load(const float *p, int64_t v, bool here, int key, int64_t pitch)
    {
        const int row4 = threadIdx.x % kWave / 16 * 4;
        zero();
        if (!here) return;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (16 * i + row4 + r < key) s[i][r] = p[(16 * i + row4 + r) * pitch + v];
    }
    // column v as a row of DK values
    __device__ __forceinline__ void store_row(float *p, int64_t v, bool here) const
    {
        const int row4 = threadIdx.x % kWave / 16 * 4;
        if (!here) return;
#pragma unroll
        for (int i = 0; i < DT; ++i) *reinterpret_cast<f32x4 *>(p + v * DK + 16 * i + row4) = s[i];
    }
    __device__ __forceinline__ void store(float *p, int64_t v, bool here, int key, int64_t pitch) const
    {
        const int row4 = threadIdx.x % kWave / 16 * 4;
        pitch = afresh(pitch);
        const uint32_t at = (uint32_t)(row4 * (int)pitch + (int)v) * 4u;  // dv <= 2^20
        if (!here) return;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (16 * i + row4 + r < key)
                    *reinterpret_cast<float *>(reinterpret_cast<char *>(p + (16 * i + r) * pitch) + at) = s[i][r];
    }
};

// Products whose operands are read from LDS all at once, before the first is used:
// left to itself the compiler reads two, waits for the LDS and multiplies.
// x_t = the rows 16 t .. of a tile of steps times s(0) .. s(KD - 1), over the channels.
// `meanwhile` is what else is to be read meanwhile.
template <bool ALONG, int KD, class In, int TT, class S, class F>
__device__ __forceinline__ void times(f32x4 (&x)[TT], const In &tile, const S &s, const F &meanwhile)
{
    constexpr int B = KD < 4 ? KD : 4;  // the registers of 16 operands at a time
    decltype(operand<ALONG>(tile, 0, 0)) k[B][TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) x[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int d0 = 0; d0 < KD; d0 += B) {
#pragma unroll
        for (int d = 0; d < B; ++d)
#pragma unroll
            for (int t = 0; t < TT; ++t) k[d][t] = operand<ALONG>(tile, 16 * t, 32 * (d0 + d));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < B; ++d) {
            mma_rows(x, k[d], s(d0 + d));
            if (d0 + d == KD - 2) {  // half of the operands' registers are free
                __builtin_amdgcn_sched_barrier(0);
                meanwhile();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (d0 + B < KD) __builtin_amdgcn_sched_barrier(0);
    }
    settle(x);
}
// x_t = the rows of a triangular matrix [C][C] times `s`; LOWER, or its transpose
template <bool LOWER, int C, class Wide, int TT, int KC>
__device__ __forceinline__ void triangle_times(f32x4 (&x)[TT], const Wide (&m)[Slots<C>::kCount], const Wide (&s)[KC])
{
    using Sl = Slots<C>;
    using P = Product<Wide, Wide>;
#pragma unroll
    for (int k = 0; k < KC; ++k)
#pragma unroll
        for (int i = 0; i < P::kParts; ++i)
#pragma unroll
            for (int t = 0; t < TT; ++t)
                if (LOWER ? Sl::in_lower(t, k) : Sl::in_upper(t, k))
                    x[t] = P::part(i, x[t], m[LOWER ? Sl::lower(t, k) : Sl::upper(t, k)], s[k]);
    settle(x);
}
// The operands of a tile's channels, their terms the steps.
template <bool ALONG, class In, class Exact, int DT, int KC>
__device__ __forceinline__ void read_channels(Exact (&k)[KC][DT], const In &tile)
{
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int s = 0; s < KC; ++s) k[s][d] = operand<ALONG>(tile, 16 * d, 32 * s);
}

// ------------------------------------------------------------- the chain ---

// The chains' waves.  A workgroup has a head and 16 NC columns of the values: NC
// waves with 16 columns of the state each in their registers, and others that
// bring the next keys and queries to LDS and take over the products that the
// state does not need (Roles below).  A wave multiplies what it has computed from
// its registers, so between two chunks only the state itself is waited for.  A
// `visit` is a chunk, or one document of it.
//
// Bound by a visit's way through the state's wave: three products one after the
// other, each with its operands' split into two bfloat16 between (about 500 vector
// instructions and 82 matrix instructions of 16 cycles), two barriers and the LDS
// reads: 3.5 us of 64 steps and 32 columns (8 x 4096 x 8 heads of 128 x 128
// bfloat16: 226 us, 5 us a visit before every wave's registers sufficed: a spilled
// address was reloaded behind all loads under way).  The matrix cores are busy 17%
// of the time, LDS 38%.  4 x 16384 x 32 heads: 1020 us, 2.1 TB/s.

// A workgroup's head, columns and segment.
struct Place {
    int64_t bh, b, h, hk;
    int first;    // its first 16 columns
    int seg;
    int n0, n1;   // chunks n0 .. n1 - 1
};
template <int NC>
__device__ __forceinline__ Place place_of(const Args &A)
{
    Place p;
    int block;
    int64_t chain;
    head_and_block(A.B * A.Hv * A.segments, A.blocks, chain, block);
    p.bh = chain / A.segments;
    p.seg = (int)(chain % A.segments);
    p.b = p.bh / A.Hv;
    p.h = p.bh % A.Hv;
    p.hk = p.h / (A.Hv / A.Hk);
    p.first = block * NC;
    p.n0 = p.seg * A.per;
    p.n1 = (int)min((int64_t)p.n0 + A.per, A.chunks);
    return p;
}

// A visit: steps r0 .. r1 - 1 of chunk n (-1: no more).
struct Visit {
    int n, r0, r1, flags;
    // starts a document; the chunk's first, its last; sums of log decays near zero
    static constexpr int kFresh = 1, kEnters = 2, kLeaves = 4, kNear = 8;
    __device__ __forceinline__ bool here() const { return n >= 0; }
    __device__ __forceinline__ bool fresh() const { return flags & kFresh; }
    __device__ __forceinline__ bool enters() const { return flags & kEnters; }
    __device__ __forceinline__ bool leaves() const { return flags & kLeaves; }
    __device__ __forceinline__ bool near() const { return flags & kNear; }
};
__device__ __forceinline__ Visit read_visit(const Visit &v)
{
    return {__builtin_amdgcn_readfirstlane(v.n), __builtin_amdgcn_readfirstlane(v.r0),
            __builtin_amdgcn_readfirstlane(v.r1), __builtin_amdgcn_readfirstlane(v.flags)};
}
// The wave that finds the visits one after the other, for all of its workgroup.
template <int C, bool BACK>
struct Planner {
    int n, r0, r1;
    StepGates gates;
    LoadedGates next;  // of the chunk after this one
    bool cut;  // a document has started
    __device__ __forceinline__ bool beyond(const Place &at) const { return BACK ? n > at.n0 : n + 1 < at.n1; }
    __device__ __forceinline__ void start(const Args &A, const Place &at)
    {
        n = BACK ? at.n1 - 1 : at.n0;
        cut = false;
        gates = load_gates<C>(A, at.b, at.h, (int64_t)n * C);
        enter(A, at);
    }
    __device__ __forceinline__ void enter(const Args &A, const Place &at)
    {
        r0 = BACK ? document_start(gates.cut, gates.rows) : 0;
        r1 = BACK ? gates.rows : document_end(gates.cut, 0, gates.rows);
        cut |= gates.cut != 0;
        if (beyond(at)) next = fetch_gates(A, at.b, at.h, (int64_t)(BACK ? n - 1 : n + 1) * C);
    }
    __device__ __forceinline__ void advance(const Args &A, const Place &at)
    {
        if (BACK ? r0 > 0 : r1 < gates.rows) {
            if (BACK)
                r1 = r0, r0 = document_start(gates.cut, r1);
            else
                r0 = r1, r1 = document_end(gates.cut, r0, gates.rows);
        } else if (beyond(at)) {
            n += BACK ? -1 : 1;
            gates = use_gates<C>(A, next, (int64_t)n * C);
            enter(A, at);
        } else {
            n = -1;
        }
    }
    // waits for the next chunk's gates, so that what is loaded from here on is not
    // waited for with them
    __device__ __forceinline__ void settle() { asm volatile("" : "+v"(next.g), "+v"(next.beta), "+v"(next.reset)); }
    // to LDS: the visit, and what its steps multiply with
    __device__ __forceinline__ void write(Visit &v, Factors<C> &F) const
    {
        const bool near = n >= 0 && write_factors(F, gates, r0, r1);
        const bool first = BACK ? r1 == gates.rows : r0 == 0, last = BACK ? r0 == 0 : r1 == gates.rows;
        if (threadIdx.x % kWave == 0)
            v = {n, r0, r1,
                 (gates.cut >> r0 & 1 ? Visit::kFresh : 0) | (first ? Visit::kEnters : 0) |
                     (last ? Visit::kLeaves : 0) | (near ? Visit::kNear : 0)};
    }
};

// What the chains' waves share: keys and queries of two visits (with 256
// channels there is room for one), their factors, and what passes between a
// state's wave and its helper.
template <bool HALF, int DK, int NC, bool TF>
struct Staged {
    static constexpr int C = Num<HALF>::kChunk, TT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32;
    static constexpr bool kTwo = DK < 256;
    using In = Pieces<HALF, DK, TF, NC * kWave>;
    typename In::Lds keys[kTwo ? 2 : 1];
    Factors<C> factors[2];
    Visit visits[2];
    __device__ __forceinline__ typename In::Lds &keys_of(int buffer) { return keys[kTwo ? buffer : 0]; }
};
template <bool HALF, int DK, int NC, bool TF>
struct Forward : Staged<HALF, DK, NC, TF> {
    using Base = Staged<HALF, DK, NC, TF>;
    typename Base::In::Lds queries[1];
    Fragment scores[Slots<Base::C>::kCount], state[NC][Base::KD], write[NC][Base::KC];
    __device__ __forceinline__ typename Base::In::Lds &queries_of(int) { return queries[0]; }
};
template <bool HALF, int DK, int NC, bool TF>
struct Backward : Staged<HALF, DK, NC, TF> {
    using Base = Staged<HALF, DK, NC, TF>;
    typename Base::In::Lds queries[Base::kTwo ? 2 : 1];
    Fragment scores[Slots<Base::C>::kCount];
    f32x4 by_scores[NC][Base::TT][kWave], by_queries[NC][Base::DT][kWave];
    __device__ __forceinline__ typename Base::In::Lds &queries_of(int buffer)
    {
        return queries[Base::kTwo ? buffer : 0];
    }
};
template <bool BACK, bool HALF, int DK, int NC, bool TF>
using Chained = std::conditional_t<BACK, Backward<HALF, DK, NC, TF>, Forward<HALF, DK, NC, TF>>;
template <bool HALF>
__device__ __forceinline__ const typename Num<HALF>::Elem *head_of(const Plane &x, int64_t b, int64_t h)
{
    return static_cast<const typename Num<HALF>::Elem *>(x.p) + b * x.b + h * x.h;
}

// P = scale (q . k) D as operands, slots first .. end - 1: its tile (s, t) as keys times
// queries, row t of the operand, four s.  BACK: P^T, as queries times keys.
template <bool BACK, bool HALF, int DK, int NC, bool TF>
__device__ __forceinline__ void make_scores(const Args &A, Chained<BACK, HALF, DK, NC, TF> &sh, int buffer, bool near,
                                            int first, int end)
{
    using N = Num<HALF>;
    constexpr int C = N::kChunk, KD = DK / 32;
    const int lane = threadIdx.x % kWave, row4 = 4 * (lane / 16), col = lane % 16;
    const Factors<C> &F = sh.factors[buffer];
    const auto &rows = BACK ? sh.queries_of(buffer) : sh.keys_of(buffer);
    const auto &columns = BACK ? sh.keys_of(buffer) : sh.queries_of(buffer);
    for (int s = first; s < end; ++s) {
        int tt = s, ss = 0;
        if constexpr (C == 64) {
            tt = BACK ? (s < 4 ? s / 2 : s - 2) : s < 2 ? s : s / 2 + 1;
            ss = BACK ? (s < 4 ? s % 2 : 1) : s < 2 ? 0 : s % 2;
        }
        f32x4 p[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
        typename N::Exact c[KD], r[KD][2];
#pragma unroll
        for (int d = 0; d < KD; ++d) {
            c[d] = operand<!TF>(columns, 16 * tt, 32 * d);
            r[d][0] = operand<!TF>(rows, 32 * ss, 32 * d);
            r[d][1] = operand<!TF>(rows, 32 * ss + 16, 32 * d);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = 0; d < KD; ++d) mma_rows(p, r[d], c[d]);
        settle(p);
        const int t = 16 * tt + col;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = 32 * ss + 16 * i + row4;
            const f32x4 d = BACK ? decays_from(F, j, t, near) : decays_to(F, t, j, near);
#pragma unroll
            for (int e = 0; e < 4; ++e) p[i][e] = (BACK ? j + e >= t : j + e <= t) ? A.scale * p[i][e] * d[e] : 0.0f;
        }
        store_fragment(sh.scores[s], stacked<HALF>(p[0], p[1]));
    }
}

// How the chains' waves share the work.  NC state's waves; as many that compute the
// outputs (backwards: help); and with NC = 2 four that bring keys and queries and plan
// the visits, which may wait for memory (they have 8 pieces a tensor each with 128
// channels) while the others do not.  With NC = 4 the waves of the outputs do this
// too, as there is no room for more waves' registers, and so with 256 channels: there
// four waves have 512 registers each, and eight would spill hundreds of their 256.
// Without outputs there are two servers or four.
template <int DK, int NC, bool OUTPUT>
struct Roles {
    static constexpr bool kApart = OUTPUT && NC == 2 && DK < 256;
    static constexpr int kServers = kApart ? 4 : NC;
    static constexpr int kServer = kApart ? 2 * NC : NC;  // their first wave
    static constexpr int kWaves = OUTPUT && !kApart ? 2 * NC : kServer + kServers;
};

// Brings keys and queries (QUERIES), plans the visits.
template <bool BACK, bool HALF, int DK, int NC, bool TF, bool QUERIES>
struct Server {
    using Lds = Chained<BACK, HALF, DK, NC, TF>;
    using In = Pieces<HALF, DK, TF, Roles<DK, NC, QUERIES>::kServers * kWave>;
    static constexpr int C = Num<HALF>::kChunk;
    In k_raw, q_raw;
    Planner<C, BACK> plan;
    Place at_;
    __device__ __forceinline__ void load(const Args &A, int64_t n, int tid)
    {
        k_raw.load(A.k, head_of<HALF>(A.k, at_.b, at_.hk), 0, n * C, A.key, A.T, tid);
        if constexpr (QUERIES) q_raw.load(A.q, head_of<HALF>(A.q, at_.b, at_.hk), 0, n * C, A.key, A.T, tid);
    }
    __device__ __forceinline__ void stage(const Args &A, Lds &sh, int buffer, const Visit &v, int tid)
    {
        k_raw.store(sh.keys_of(buffer), v.r0, v.r1, A.key, tid);
        if constexpr (QUERIES) q_raw.store(sh.queries_of(buffer), v.r0, v.r1, A.key, tid);
        plan.settle();
    }
    // what the visit after v has; in the visit's first half, as in the second the others
    // wait for stage()
    __device__ __forceinline__ void fetch(const Args &A, const Visit &v, int tid)
    {
        // (also where the next visit has the same chunk: see the state's wave)
        load(A, v.leaves() ? (BACK ? max(v.n - 1, at_.n0) : min(v.n + 1, at_.n1 - 1)) : v.n, tid);
    }
    __device__ __forceinline__ Visit start(const Args &A, Lds &sh, const Place &at, int c, int tid)
    {
        at_ = at;
        load(A, BACK ? at.n1 - 1 : at.n0, tid);
        if (c == 0) {
            plan.start(A, at);
            plan.write(sh.visits[0], sh.factors[0]);
        }
        __syncthreads();
        const Visit now = read_visit(sh.visits[0]);
        stage(A, sh, 0, now, tid);
        __syncthreads();
        return now;
    }
    __device__ __forceinline__ void look(const Args &A, Lds &sh, int buffer, int c)
    {
        if (c != 0) return;
        plan.advance(A, at_);
        plan.write(sh.visits[buffer ^ 1], sh.factors[buffer ^ 1]);
        if (!BACK && A.ends && plan.n < 0 && at_.first == 0 && threadIdx.x % kWave == 0)
            A.cuts[at_.bh * A.segments + at_.seg] = plan.cut;
    }
};
template <bool BACK, bool HALF, int DK, int NC, bool TF, bool QUERIES>
__device__ __forceinline__ void chain_server(const Args &A, Chained<BACK, HALF, DK, NC, TF> &shared, const Place &at,
                                             int c)
{
    const int tid = c * kWave + threadIdx.x % kWave;
    constexpr bool kSix = Slots<Num<HALF>::kChunk>::kCount == 6;
    // its slots of the scores: none to the first, which plans; of six one each and two to
    // the last (the waves of the outputs have two), backwards two each; of two one each
    const int s0 = c == 0 ? 0 : BACK && kSix ? 2 * c - 2 : min(c - 1, kSix ? 6 : 2);
    const int s1 = c == 0 ? 0 : kSix ? (BACK ? 2 * c : c == 3 ? 4 : c) : min(c, 2);
    Server<BACK, HALF, DK, NC, TF, QUERIES> server;
    Visit now = server.start(A, shared, at, c, tid);
    for (int buffer = 0; now.here(); buffer ^= 1) {
        auto &sh = lds_afresh(shared);
        server.look(A, sh, buffer, c);
        server.fetch(A, now, tid);
        if constexpr (QUERIES) make_scores<BACK, HALF, DK, NC, TF>(A, sh, buffer, now.near(), s0, s1);
        __syncthreads();
        if constexpr (BACK) __syncthreads();
        const Visit then = read_visit(sh.visits[buffer ^ 1]);
        if (!sh.kTwo) __syncthreads();
        if (then.here()) server.stage(A, sh, buffer ^ 1, then, tid);
        __syncthreads();
        now = then;
    }
}
// P, q^T S and the outputs, from S and W as operands in LDS.  SERVES: also what a
// server does.
template <bool HALF, int DK, int NC, bool TF, bool SERVES>
__device__ __forceinline__ void chain_output(const Args &A, Forward<HALF, DK, NC, TF> &shared, const Place &at, int c)
{
    using N = Num<HALF>;
    using Wide = typename N::Wide;
    constexpr int C = N::kChunk, TT = C / 16, KC = C / 32, KD = DK / 32, kSlots = Slots<C>::kCount;
    const int lane = threadIdx.x % kWave, row4 = 4 * (lane / 16), col = lane % 16, tid = c * kWave + lane;
    const int64_t v = 16 * (int64_t)(at.first + c) + col;
    const bool has_v = v < A.value;
    float *const o = static_cast<float *>(A.o.p) + at.b * A.o.b + at.h * A.o.h + v * A.o.d;
    // its slots of P: with servers one of the last two of six; else a share of all, of
    // four waves none to the one that plans
    constexpr bool kSix = kSlots == 6;
    int s0 = kSix ? 4 + c : 0, s1 = kSix ? 5 + c : 0;
    if constexpr (SERVES && NC == 2) s0 = kSlots / 2 * c, s1 = s0 + kSlots / 2;
    if constexpr (SERVES && NC == 4) {
        s0 = kSix ? max(2 * c - 2, 0) : min(max(c - 1, 0), 2);
        s1 = c == 0 ? s0 : min(s0 + (kSix ? 2 : 1), kSlots);
    }
    [[maybe_unused]] Server<false, HALF, DK, NC, TF, true> server;
    Visit now;
    if constexpr (SERVES) {
        now = server.start(A, shared, at, c, tid);
    } else {
        __syncthreads();
        now = read_visit(shared.visits[0]);
        __syncthreads();
    }
    for (int buffer = 0; now.here(); buffer ^= 1) {
        auto &sh = lds_afresh(shared);
        const Factors<C> &F = sh.factors[buffer];
        if constexpr (SERVES) {
            server.look(A, sh, buffer, c);
            server.fetch(A, now, tid);
        }
        make_scores<false, HALF, DK, NC, TF>(A, sh, buffer, now.near(), s0, s1);
        f32x4 out[TT];
        {
            Wide s[KD];
#pragma unroll
            for (int d = 0; d < KD; ++d) s[d] = load_fragment(sh.state[c][d], N());
            f32x4 start[TT];
            times<!TF, KD>(out, sh.queries_of(buffer), [&](int d) { return s[d]; }, [&]() {
#pragma unroll
                for (int t = 0; t < TT; ++t) start[t] = four(F.start + 16 * t + row4);
            });
#pragma unroll
            for (int t = 0; t < TT; ++t) out[t] *= A.scale * start[t];
        }
        __syncthreads();
        const Visit then = read_visit(sh.visits[buffer ^ 1]);
        Wide x[KC], p[kSlots];
#pragma unroll
        for (int s = 0; s < KC; ++s) x[s] = load_fragment(sh.write[c][s], N());
#pragma unroll
        for (int s = 0; s < kSlots; ++s) p[s] = load_fragment(sh.scores[s], N());
        if constexpr (SERVES)
            if (sh.kTwo && then.here()) server.stage(A, sh, buffer ^ 1, then, tid);
        triangle_times<true, C>(out, p, x);
        const bool whole = now.r0 == 0 && now.r1 == C;
        if (has_v)
#pragma unroll
            for (int t = 0; t < TT; ++t)
                store_column<false>(o + (int64_t)now.n * C * A.o.t, A.o.t, 16 * t + row4, now.r0,
                                    now.r1, whole, out[t]);
        if (!sh.kTwo) {
            __syncthreads();
            if constexpr (SERVES)
                if (then.here()) server.stage(A, sh, buffer ^ 1, then, tid);
        }
        __syncthreads();
        now = then;
    }
}
// A state's wave: k^T S, R, W, S'.  OUTPUT: S and W for the helper, and the last
// state; else for the backward pass, the states before each chunk and W to memory.
template <bool HALF, int DK, int NC, bool TF, bool OUTPUT>
__device__ __forceinline__ void chain_state(const Args &A, Forward<HALF, DK, NC, TF> &shared, const Place &at, int c)
{
    using N = Num<HALF>;
    using Wide = typename N::Wide;
    constexpr int C = N::kChunk, TT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32;
    using Sl = Slots<C>;
    const int lane = threadIdx.x % kWave, row4 = 4 * (lane / 16), col = lane % 16;
    const int64_t v = 16 * (int64_t)(at.first + c) + col;
    const bool has_v = v < A.value, in_row = v < A.value_pad && !A.ends;
    constexpr bool kEarly = DK < 256 && NC == 2 && !OUTPUT;  // registers for all of the keys' operands, of 512
    State<DK> S;
    Wide operands[KD], inverse[Sl::kCount];
    Columns<HALF, C> value;
    const auto *const values = head_of<HALF>(A.v, at.b, at.h) + min(v, (int64_t)A.value - 1) * A.v.d;
    const auto load_value = [&](int64_t n) { value.load(values, A.v.t, n * C, A.T); };
    const auto load_inverse = [&](int64_t n) {
#pragma unroll
        for (int s = 0; s < Sl::kCount; ++s)
            inverse[s] = load_fragment(A.inverse[(at.bh * A.chunks + n) * Sl::kCount + s], N());
    };
    const auto make_operands = [&](Forward<HALF, DK, NC, TF> &sh) {
#pragma unroll
        for (int d = 0; d < KD; ++d) {
            operands[d] = stacked<HALF>(S.s[2 * d], S.s[2 * d + 1]);
            if constexpr (OUTPUT) store_fragment(sh.state[c][d], operands[d]);
        }
    };
    const auto keep = [&](int64_t n) {
        S.store_row(A.states + (at.bh * A.chunks + n) * DK * A.value_pad, v, in_row);
    };

    if (!OUTPUT && A.ends) {
        S.identity((int)min(v - A.value_pad, (int64_t)A.key));  // zero in the values' columns
    } else if (A.segments > 1) {
        S.load(A.marks + (at.bh * A.segments + at.seg) * DK * A.value_pad, v, v < A.value_pad, DK, A.value_pad);
    } else {
        S.load(A.h0 + at.bh * A.key * A.value, v, A.h0 && has_v, A.key, A.value);
    }
    load_value(at.n0);
    load_inverse(at.n0);
    if constexpr (!OUTPUT) keep(at.n0);
    __syncthreads();
    Visit now = read_visit(shared.visits[0]);
    if (now.fresh()) S.zero();
    make_operands(shared);
    __syncthreads();
    for (int buffer = 0; now.here(); buffer ^= 1) {
        auto &sh = lds_afresh(shared);
        const Factors<C> &F = sh.factors[buffer];
        const auto &K = sh.keys_of(buffer);
        const bool whole = now.r0 == 0 && now.r1 == C;
        // what the next visit reads, also where it is what this one has: a load that
        // may not be under way would have everything behind it waited for
        const int64_t after = now.leaves() && now.n + 1 < at.n1 ? now.n + 1 : now.n;
        f32x4 x[TT];
        f32x4 start[TT], beta[TT];
        typename N::Exact kt[KC][DT];
        times<!TF, KD>(x, K, [&](int d) { return operands[d]; }, [&]() {
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                start[t] = four(F.start + 16 * t + row4);
                beta[t] = four(F.beta + 16 * t + row4);
            }
            if (kEarly) read_channels<TF>(kt, K);
        });
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const f32x4 val = value.get(t);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] = beta[t][e] * fmaf_(-start[t][e], x[t][e], has_v ? val[e] : 0.0f);
        }
        if (!whole)
#pragma unroll
            for (int t = 0; t < TT; ++t) x[t] = only_steps(x[t], 16 * t + row4, now.r0, now.r1);
        if (!kEarly) read_channels<TF>(kt, K);
        Wide rhs[KC];
#pragma unroll
        for (int s = 0; s < KC; ++s) rhs[s] = stacked<HALF>(x[2 * s], x[2 * s + 1]);
#pragma unroll
        for (int t = 0; t < TT; ++t) x[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        triangle_times<true, C>(x, inverse, rhs);
        if (!whole)
#pragma unroll
            for (int t = 0; t < TT; ++t) x[t] = only_steps(x[t], 16 * t + row4, now.r0, now.r1);
        load_value(after);
        load_inverse(after);
        if constexpr (OUTPUT) {
#pragma unroll
            for (int s = 0; s < KC; ++s) store_fragment(sh.write[c][s], stacked<HALF>(x[2 * s], x[2 * s + 1]));
        } else {
            if (in_row)
                store_rows(A.w + (at.bh * A.chunks + now.n) * C * A.value_pad, v, now.r0, now.r1, whole, x);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) x[t] *= four(F.end + 16 * t + row4);
        if (!whole)
#pragma unroll
            for (int t = 0; t < TT; ++t) x[t] = only_steps(x[t], 16 * t + row4, now.r0, now.r1);
        Wide carry[KC];
#pragma unroll
        for (int s = 0; s < KC; ++s) carry[s] = stacked<HALF>(x[2 * s], x[2 * s + 1]);
        __syncthreads();
        const Visit then = read_visit(sh.visits[buffer ^ 1]);
        const float across = F.across[0];
        S.advance(across, kt, carry);
        if (then.here()) {
            if constexpr (!OUTPUT)
                if (then.enters()) keep(then.n);
            if (then.fresh()) S.zero();
            make_operands(sh);
        }
        if (!sh.kTwo) __syncthreads();
        __syncthreads();
        now = then;
    }
    if constexpr (OUTPUT) {
        if (A.last && at.n1 == A.chunks) S.store(A.last + at.bh * A.key * A.value, v, has_v, A.key, A.value);
    } else if (A.ends) {
        const int columns = A.value_pad + A.key_pad;
        S.store(A.maps + (at.bh * A.segments + at.seg) * DK * columns, v, v < columns, DK, columns);
    }
}
template <bool HALF, int DK, int NC, bool TF, bool OUTPUT>
__global__ void __launch_bounds__((Roles<DK, NC, OUTPUT>::kWaves * kWave)) delta_chain_kernel(Args A)
{
    __shared__ Forward<HALF, DK, NC, TF> sh;
    using R = Roles<DK, NC, OUTPUT>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Place at = place_of<NC>(A);
    if (A.chunks == 0) {  // the state goes through
        State<DK> S;
        const int64_t v = 16 * (int64_t)(at.first + wave) + threadIdx.x % 16;
        const bool here = wave < NC && v < A.value && A.last;
        S.load(A.h0 + at.bh * A.key * A.value, v, here && A.h0, A.key, A.value);
        S.store(A.last + at.bh * A.key * A.value, v, here, A.key, A.value);
        return;
    }
    if (wave < NC) {
        chain_state<HALF, DK, NC, TF, OUTPUT>(A, sh, at, wave);
    } else if constexpr (!OUTPUT) {
        chain_server<false, HALF, DK, NC, TF, false>(A, sh, at, wave - NC);
    } else if constexpr (R::kApart) {
        if (wave < R::kServer)
            chain_output<HALF, DK, NC, TF, false>(A, sh, at, wave - NC);
        else
            chain_server<false, HALF, DK, NC, TF, true>(A, sh, at, wave - R::kServer);
    } else {
        chain_output<HALF, DK, NC, TF, true>(A, sh, at, wave - NC);
    }
}

// Another lane's value, of the 16 of a group: rotated by 8 or 4 lanes, of the mirrored
// lane of 8, and of a neighbour (the instruction set's codes).
constexpr int kRotate8 = 0x128, kRotate4 = 0x124, kMirror8 = 0x141, kNext = 0xb1, kNext2 = 0x4e;
template <int CODE>
__device__ __forceinline__ float from_lane(float x)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CODE, 0xf, 0xf, true));
}
// Sums over the 16 lanes of a group, of M values each: at the end a lane holds
// the sum of value `which` (with M < 16 several lanes the same one, to the last bit:
// they all write it to one place).  Half of the values go to another lane at each
// step, first to one whose lower bits differ too.
template <int M>
__device__ __forceinline__ float sum_columns(float (&x)[M], int &which)
{
    static_assert(M == 8 || M == 4, "halves");
    const int lane = threadIdx.x % kWave;
    which = 0;
    const auto halve = [&](auto half, auto code, int bit) {
        constexpr int m = decltype(half)::value;
        const bool upper = lane & bit;
        which += upper ? m : 0;
#pragma unroll
        for (int i = 0; i < m; ++i)
            x[i] = (upper ? x[i + m] : x[i]) + from_lane<decltype(code)::value>(upper ? x[i] : x[i + m]);
    };
    if constexpr (M == 8) halve(std::integral_constant<int, 4>(), std::integral_constant<int, kMirror8>(), 4);
    halve(std::integral_constant<int, 2>(), std::integral_constant<int, kNext>(), 1);
    halve(std::integral_constant<int, 1>(), std::integral_constant<int, kNext2>(), 2);
    // (lanes 8 apart first: the sums of both pairs are then the same in either order)
    x[0] += from_lane<kRotate8>(x[0]);
    return M == 4 ? x[0] + from_lane<kRotate4>(x[0]) : x[0];
}

// The chain backwards: the gradient of the state, from the last chunk to the
// first, and X, the gradient of R.  A helper: P^T dO, which the state's wave needs
// in the middle of a visit, and scale (exp(G) Q)^T dO, which joins the state a
// visit later.  SERVES: also what a server does.
// Bound like the forward chain, three barriers a visit: 8 x 4096 x 8 heads of 128 x
// 128 bfloat16 324 us, 5 a chunk (the inverses through LDS instead of the state's
// wave's own loads: 410 us instead of 345).
template <bool HALF, int DK, int NC, bool TF, bool SERVES>
__device__ __forceinline__ void back_helper(const Args &A, Backward<HALF, DK, NC, TF> &shared, const Place &at, int c)
{
    using N = Num<HALF>;
    using Wide = typename N::Wide;
    constexpr int C = N::kChunk, TT = C / 16, KC = C / 32, DT = DK / 16, kSlots = Slots<C>::kCount;
    const int lane = threadIdx.x % kWave, row4 = 4 * (lane / 16), col = lane % 16, tid = c * kWave + lane;
    const int64_t v = 16 * (int64_t)(at.first + c) + col;
    const bool has_o = v < A.value && A.o.p, all_o = 16 * (at.first + c + 1) <= A.value && A.o.p;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    // its slots of P^T: with servers none; else a share, the smallest to the one that plans
    constexpr bool kSix = kSlots == 6;
    int s0 = 0, s1 = 0;
    if constexpr (SERVES && NC == 2) s0 = kSix ? 2 * c : c, s1 = kSix ? 2 + 4 * c : c + 1;
    if constexpr (SERVES && NC == 4) {
        s0 = kSix ? max(2 * c - 2, 0) : min(max(c - 1, 0), 2);
        s1 = c == 0 ? s0 : min(s0 + (kSix ? 2 : 1), kSlots);
    }
    Columns<false, C> go;
    const float *const gos = head_of<false>(A.o, at.b, at.h) + min(v, (int64_t)A.value - 1) * A.o.d;
    const auto load_go = [&](int64_t n) {
        if (A.o.p) go.load(gos, A.o.t, n * C, A.T);
    };
    [[maybe_unused]] Server<true, HALF, DK, NC, TF, true> server;
    Visit now;
    load_go(at.n1 - 1);
    if constexpr (SERVES) {
        now = server.start(A, shared, at, c, tid);
    } else {
        __syncthreads();
        now = read_visit(shared.visits[0]);
        __syncthreads();
    }
    for (int buffer = 0; now.here(); buffer ^= 1) {
        auto &sh = lds_afresh(shared);
        const Factors<C> &F = sh.factors[buffer];
        if constexpr (SERVES) {
            server.look(A, sh, buffer, c);
            server.fetch(A, now, tid);
        }
        make_scores<true, HALF, DK, NC, TF>(A, sh, buffer, now.near(), s0, s1);
        const bool whole = now.r0 == 0 && now.r1 == C;
        f32x4 x[TT];
        Wide g[KC];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            x[t] = go.get(t);
            if (!whole || !all_o) x[t] = only_steps(x[t], 16 * t + row4, has_o ? now.r0 : C, now.r1);
        }
#pragma unroll
        for (int s = 0; s < KC; ++s) g[s] = stacked<HALF>(x[2 * s], x[2 * s + 1]);
        __syncthreads();
        {
            Wide p[kSlots];
            f32x4 y[TT];
#pragma unroll
            for (int s = 0; s < kSlots; ++s) p[s] = load_fragment(sh.scores[s], N());
#pragma unroll
            for (int t = 0; t < TT; ++t) y[t] = zero;
            triangle_times<false, C>(y, p, g);
#pragma unroll
            for (int t = 0; t < TT; ++t) sh.by_scores[c][t][lane] = y[t];
        }
        __syncthreads();
        const Visit then = read_visit(sh.visits[buffer ^ 1]);
        if constexpr (SERVES)
            if (sh.kTwo && then.here()) server.stage(A, sh, buffer ^ 1, then, tid);
        load_go(then.here() ? then.n : now.n);
        if (!now.fresh()) {
            typename N::Exact qt[KC][DT];
            f32x4 start[TT], part[DT];
#pragma unroll
            for (int t = 0; t < TT; ++t) start[t] = four(F.start + 16 * t + row4);
            read_channels<TF>(qt, sh.queries_of(buffer));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                x[t] *= A.scale * start[t];
                if (!whole) x[t] = only_steps(x[t], 16 * t + row4, now.r0, now.r1);
            }
#pragma unroll
            for (int s = 0; s < KC; ++s) g[s] = stacked<HALF>(x[2 * s], x[2 * s + 1]);
#pragma unroll
            for (int d = 0; d < DT; ++d) part[d] = zero;
#pragma unroll
            for (int s = 0; s < KC; ++s) mma_rows(part, qt[s], g[s]);
            settle(part);
#pragma unroll
            for (int d = 0; d < DT; ++d) sh.by_queries[c][d][lane] = part[d];
        }
        if (!sh.kTwo) {
            __syncthreads();
            if constexpr (SERVES)
                if (then.here()) server.stage(A, sh, buffer ^ 1, then, tid);
        }
        __syncthreads();
        now = then;
    }
}
// A state's wave: K dS', X, dS.  Writes dS' behind each chunk, X and dV = b X.
template <bool HALF, int DK, int NC, bool TF>
__device__ __forceinline__ void back_state(const Args &A, Backward<HALF, DK, NC, TF> &shared, const Place &at, int c)
{
    using N = Num<HALF>;
    using Wide = typename N::Wide;
    constexpr int C = N::kChunk, TT = C / 16, KC = C / 32, DT = DK / 16, KD = DK / 32;
    using Sl = Slots<C>;
    const int lane = threadIdx.x % kWave, row4 = 4 * (lane / 16), col = lane % 16;
    const int64_t v = 16 * (int64_t)(at.first + c) + col;
    const bool has_v = v < A.value && !A.ends, in_row = v < A.value_pad && !A.ends;
    auto *const dv = static_cast<typename N::Elem *>(A.dv.p) + at.b * A.dv.b + at.h * A.dv.h;
    State<DK> S;
    Wide inverse[Sl::kCount];
    const auto load_inverse = [&](int64_t n) {
#pragma unroll
        for (int s = 0; s < Sl::kCount; ++s)
            inverse[s] = load_fragment(A.inverse_t[(at.bh * A.chunks + n) * Sl::kCount + s], N());
    };
    bool behind = false;  // the helper has a part of the state's gradient
    const auto join = [&](Backward<HALF, DK, NC, TF> &sh) {
        if (behind)
#pragma unroll
            for (int d = 0; d < DT; ++d) S.s[d] += sh.by_queries[c][d][lane];
    };

    if (A.ends) {
        S.zero();
    } else if (A.segments > 1) {
        S.load(A.marks + (at.bh * A.segments + at.seg) * DK * A.value_pad, v, in_row, DK, A.value_pad);
    } else {
        S.load(A.g_last + at.bh * A.key * A.value, v, A.g_last && has_v, A.key, A.value);
    }
    load_inverse(at.n1 - 1);
    __syncthreads();
    Visit now = read_visit(shared.visits[0]);
    __syncthreads();
    for (int buffer = 0; now.here(); buffer ^= 1) {
        auto &sh = lds_afresh(shared);
        const int64_t item = at.bh * A.chunks + now.n;
        const Factors<C> &F = sh.factors[buffer];
        const auto &K = sh.keys_of(buffer);
        const bool whole = now.r0 == 0 && now.r1 == C;
        const int64_t after = now.leaves() && now.n > at.n0 ? now.n - 1 : now.n;
        f32x4 x[TT];
        join(sh);
        f32x4 end[TT];
        times<!TF, KD>(x, K, [&](int d) { return stacked<HALF>(S.s[2 * d], S.s[2 * d + 1]); }, [&]() {
#pragma unroll
            for (int t = 0; t < TT; ++t) end[t] = four(F.end + 16 * t + row4);
        });
        __syncthreads();  // (the scores are there, for the helper)
        __syncthreads();
        const Visit then = read_visit(sh.visits[buffer ^ 1]);
        Wide p[KC];
        {
            f32x4 y[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) y[t] = sh.by_scores[c][t][lane];
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[t][e] = fmaf_(end[t][e], x[t][e], y[t][e]);
        }
        typename N::Exact kt[KC][DT];
        read_channels<TF>(kt, K);
        if (!whole)
#pragma unroll
            for (int t = 0; t < TT; ++t) x[t] = only_steps(x[t], 16 * t + row4, now.r0, now.r1);
#pragma unroll
        for (int s = 0; s < KC; ++s) p[s] = stacked<HALF>(x[2 * s], x[2 * s + 1]);
#pragma unroll
        for (int t = 0; t < TT; ++t) x[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        triangle_times<false, C>(x, inverse, p);
        if (!whole)
#pragma unroll
            for (int t = 0; t < TT; ++t) x[t] = only_steps(x[t], 16 * t + row4, now.r0, now.r1);
        f32x4 start[TT], beta[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            start[t] = four(F.start + 16 * t + row4);
            beta[t] = four(F.beta + 16 * t + row4);
        }
        // (not before the product: what is stored would be waited for with the inverse)
        if (now.enters()) S.store_row(A.dstates + item * DK * A.value_pad, v, in_row);
        if (in_row) store_rows(A.x + item * C * A.value_pad, v, now.r0, now.r1, whole, x);
        auto *const dv_column = dv + (int64_t)now.n * C * A.dv.t + v * afresh(A.dv.d);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            f32x4 bx;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                bx[e] = beta[t][e] * x[t][e];
                x[t][e] = -start[t][e] * bx[e];
            }
            if (has_v)
                store_column<HALF>(dv_column, A.dv.t, 16 * t + row4, now.r0, now.r1, whole, bx);
            if (!whole) x[t] = only_steps(x[t], 16 * t + row4, now.r0, now.r1);
        }
        if (now.fresh()) {  // the state before this document's is no part of it
            S.zero();
        } else {
#pragma unroll
            for (int s = 0; s < KC; ++s) p[s] = stacked<HALF>(x[2 * s], x[2 * s + 1]);
            S.advance(F.across[0], kt, p);
        }
        load_inverse(after);
        behind = !now.fresh();
        if (!sh.kTwo) __syncthreads();
        __syncthreads();
        now = then;
    }
    join(shared);
    if (A.ends) {
        const int columns = A.value_pad + A.key_pad;
        S.store(A.maps + (at.bh * A.segments + at.seg) * DK * columns, v, v < A.value_pad, DK, columns);
    } else if (A.dh0 && at.n0 == 0) {
        S.store(A.dh0 + at.bh * A.key * A.value, v, has_v, A.key, A.value);
    }
}
template <bool HALF, int DK, int NC, bool TF>
__global__ void __launch_bounds__((Roles<DK, NC, true>::kWaves * kWave)) delta_back_kernel(Args A)
{
    __shared__ Backward<HALF, DK, NC, TF> sh;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const Place at = place_of<NC>(A);
    if (A.chunks == 0) {
        State<DK> S;
        const int64_t v = 16 * (int64_t)(at.first + wave) + threadIdx.x % 16;
        const bool here = wave < NC && v < A.value && A.dh0;
        S.load(A.g_last + at.bh * A.key * A.value, v, here && A.g_last, A.key, A.value);
        S.store(A.dh0 + at.bh * A.key * A.value, v, here, A.key, A.value);
        return;
    }
    using R = Roles<DK, NC, true>;
    if (wave < NC)
        back_state<HALF, DK, NC, TF>(A, sh, at, wave);
    else if (R::kApart && wave >= R::kServer)
        chain_server<true, HALF, DK, NC, TF, true>(A, sh, at, wave - R::kServer);
    else
        back_helper<HALF, DK, NC, TF, !R::kApart>(A, sh, at, wave - NC);
}

// ------------------------------------------------------------ segments ---

// Long chains of few heads, chained in segments at once.  A segment takes the state
// S before it to M S + N: with `ends` the forward chain computes N as its end from
// zero and M, in further columns without values, as its end from the identity; the
// backward chain's map has M transposed.  This kernel goes along the segments and
// leaves the state before each (BACK: the state's gradient behind each) in `marks`;
// then the chains run again from there.  Where a document starts in a segment
// nothing of S is kept, whatever is in it.  A workgroup for a head and 16 columns,
// float32 products.  Bound by the way along the segments, 0.9 us each (the next one's
// map is read meanwhile, else 1.6): 64 of them, 64 x 64, 60 us.
template <int DK, bool BACK>
__global__ void __launch_bounds__(4 * kWave) delta_segments_kernel(Args A)
{
    constexpr int DT = DK / 16, kMine = (DT + 3) / 4, kPitch = DK + 4;
    __shared__ f32x4 state4[16 * kPitch / 4];
    float *const state = reinterpret_cast<float *>(state4);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = threadIdx.x % kWave, row4 = 4 * (lane / 16), col = lane % 16;
    const int tiles = A.value_pad / 16;
    const int64_t bh = blockIdx.x / tiles, v = 16 * (blockIdx.x % tiles) + col;
    const float *const first = BACK ? A.g_last : A.h0;
    // the state by columns, in LDS: rows of DK channels
    f32x4 S[kMine];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int d0 = 16 * (wave + 4 * m) + row4;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[m][r] = first && d0 + r < A.key && v < A.value ? first[(bh * A.key + d0 + r) * A.value + v] : 0.0f;
    }
    // a segment's map: N's rows that the wave has, and M's as operands
    struct Map {
        f32x4 n[kMine], m[kMine][DT];
        int cut;
        __device__ __forceinline__ void load(const Args &A, int64_t seg, int64_t v, int wave)
        {
            const int lane = threadIdx.x % kWave, row4 = 4 * (lane / 16), col = lane % 16;
            const int columns = A.value_pad + A.key_pad;
            const float *const map = A.maps + seg * DK * columns;
            cut = A.cuts[seg];
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int d0 = min(16 * (wave + 4 * i), DK - 16);
#pragma unroll
                for (int r = 0; r < 4; ++r) n[i][r] = map[(int64_t)(d0 + row4 + r) * columns + v];
#pragma unroll
                for (int t = 0; t < DT; ++t) {
                    const int d = min(d0 + col, A.key_pad - 1), k = min(16 * t + row4, A.key_pad - 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        m[i][t][e] = map[(int64_t)(BACK ? k + e : d) * columns + A.value_pad + (BACK ? d : k + e)];
                }
            }
        }
    };
    constexpr bool kAhead = DK < 256;  // registers for the next one's
    Map map, next;
    const auto segment = [&](int i) {
        const int at = min(i, A.segments - 1);
        return bh * A.segments + (BACK ? A.segments - 1 - at : at);
    };
    if (kAhead) next.load(A, segment(0), v, wave);
    for (int i = 0; i < A.segments; ++i) {
        const int64_t seg = segment(i);
        if (kAhead) {
            map = next;
            next.load(A, segment(i + 1), v, wave);
        } else {
            map.load(A, seg, v, wave);
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int d0 = 16 * (wave + 4 * m) + row4;
            if (d0 >= DK) break;
            *reinterpret_cast<f32x4 *>(state + col * kPitch + d0) = S[m];
#pragma unroll
            for (int r = 0; r < 4; ++r) A.marks[(seg * DK + d0 + r) * A.value_pad + v] = S[m][r];
            S[m] = map.n[m];
        }
        __syncthreads();
        if (map.cut) continue;
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            if (16 * (wave + 4 * m) >= A.key_pad) break;
#pragma unroll
            for (int t = 0; t < DT; ++t)
                if (16 * t < A.key_pad)
                    S[m] = block_mma(S[m], map.m[m][t], four(state + col * kPitch + 16 * t + row4));
        }
        settle(S);
    }
}

// Four steps t .. t + 3 of channel d of a tile of queries or keys.
template <bool TF, bool HALF, int ROWS, int COLS>
__device__ __forceinline__ f32x4 steps_of(const Tile<HALF, ROWS, COLS> &x, int d, int t)
{
    f32x4 r;
    if constexpr (TF && HALF) {
        uint32_t w[2];
        __builtin_memcpy(w, x.at + d * x.kPitch + t, 8);
        r = f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                  __uint_as_float(w[1] & 0xffff0000u)};
    } else if constexpr (TF) {
        r = four(x.at + d * x.kPitch + t);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = load_gate<HALF>(x.at, (t + e) * x.kPitch + d);
    }
    return r;
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
// Two halves of the steps by four parts of the channels: a wave's rows of dO, X and
// W are read once for all its channels (a wave for a part of the channels and all
// steps reads twice as much from LDS, which bounds it then).  32 columns of the
// values at a time; the next ones are loaded meanwhile.  The workspace's rows are
// columns of the values, as the chains' waves hold them, who store 16 bytes a lane.
// SHARED: several value heads share a key head, whose gradients are summed in
// registers.
// Bound by latency: one workgroup fits a CU, and its phases (loads, four blocks of
// columns, E and H, the last products, the stores: 50000 cycles) wait for one
// another.  4096 chunks of 128 x 128 bfloat16, 1.2 GB: 510 us, 2.4 TB/s (1066 us
// while it spilled registers).  float32 80 x 100, 288 workgroups of three heads
// each: 181 us, two rounds for 32 of them.  With 256 channels it spills 66 to 320
// registers: 8 x 4096 x 8 heads of 256 x 128 bfloat16 take 3.8 ms a call, 1.1 of 128.
template <bool HALF, int DK, bool TF>
struct Gradients {
    using N = Num<HALF>;
    static constexpr int C = N::kChunk, TT = C / 16, DT = DK / 16, VB = 32, kT = 2, kD = 4, kPairs = TT * kD;
    using In = Pieces<HALF, DK, TF, kThreads>;
    typename In::Lds keys, queries;
    static constexpr bool kBoth = DK < 256;  // room for both states' columns
    union {
        struct {
            WideTile<HALF, TF ? VB : C, TF ? C : VB> out;
            WideTile<HALF, VB, C> x, w;
            WideTile<HALF, VB, DK> s[kBoth ? 2 : 1];
        } block;
        struct {
            WideTile<HALF, C, C> e, h;  // E and b H by columns
        } t;
    };
    Factors<C> F;
    float row_sum[kPairs * 16], col_sum[kPairs * 16], h_sum[kPairs * 16];
    float dots[3][kD][C], xv[kWaves][C], inner[kWaves];
};
template <bool HALF, int DK, bool TF, bool SHARED>
__global__ void __launch_bounds__(kThreads) delta_grad_kernel(Args A)
{
    using N = Num<HALF>;
    using Wide = typename N::Wide;
    using Exact = typename N::Exact;
    using L = Gradients<HALF, DK, TF>;
    using In = typename L::In;
    constexpr int C = L::C, TT = L::TT, KC = C / 32, KD = DK / 32, kT = L::kT, kD = L::kD, VB = L::VB;
    constexpr int ND = L::DT / kD, NT = TT / kT;
    constexpr int kStates = VB * DK / 4 / kThreads;  // a thread's pieces of a state's columns
    __shared__ L sh;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), pd = wave % kD, pt = wave / kD;
    const unsigned chunks = (unsigned)A.chunks, heads = (unsigned)A.Hk, bk = blockIdx.x / chunks;
    const int64_t n = blockIdx.x % chunks, b = bk / heads, hk = bk % heads, t0 = n * C;
    const int group = SHARED ? A.Hv / A.Hk : 1;
    const int wd = 16 * ND * pd, wt = 16 * NT * pt;  // the wave's first channel and step
    using Elem = typename N::Elem;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    Elem *const dq_at = static_cast<Elem *>(A.dq.p) + b * A.dq.b + hk * A.dq.h + t0 * A.dq.t;
    Elem *const dk_at = static_cast<Elem *>(A.dk.p) + b * A.dk.b + hk * A.dk.h + t0 * A.dk.t;

    [[maybe_unused]] f32x4 dq[NT][ND], dk[NT][ND];
    if constexpr (SHARED)
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int c = 0; c < ND; ++c) dq[a][c] = dk[a][c] = zero;
    for (int head = 0; head < group; ++head) {
        const int64_t h = hk * group + head, bh = b * A.Hv + h, item = bh * A.chunks + n;
        const LoadedGates loaded = fetch_gates(A, b, h, t0);
        StepGates gates;
        const int rows = (int)min((int64_t)C, A.T - t0);
        const float *const s_before = A.states + item * DK * A.value_pad;
        const float *const s_behind = A.dstates + item * DK * A.value_pad;
        // (without a gradient of the output its place is read all the same: a load that may
        // not be under way would be waited for)
        const bool has_go = A.o.p != nullptr;
        const Plane go = {has_go ? A.o.p : A.x, has_go ? A.o.b : 0, has_go ? A.o.h : 0, has_go ? A.o.d : 0,
                          has_go ? A.o.t : 0};
        const float *const x_at = A.x + item * C * A.value_pad, *const w_at = A.w + item * C * A.value_pad;
        for (int r0 = 0, r1; r0 < rows; r0 = r1) {
            const int lane = lane_afresh(threadIdx.x % kWave), row4 = 4 * (lane / 16), col = lane % 16;
            // 32 columns as loaded, four values a piece: X and W, (v, t); dO and V as
            // they lie side by side, (v, t) or (t, v); the states, (v, d)
            constexpr bool kAll = C * VB / 4 == kThreads;  // a piece for every thread
            const int u = wave * kWave + lane;
            const bool loads = kAll || u < C * VB / 4;
            const int pv = u / (C / 4), pt4 = u % (C / 4) * 4, prow = u / (VB / 4), pv4 = u % (VB / 4) * 4;
            f32x4 xr, wr, orr, sr[kStates], gr[kStates];
            uint32_t vr[HALF ? 2 : 4];
            // four elements side by side, or `step` apart from `first` to `last`
            const auto load_four = [&](auto *p, int64_t step, bool beside, int first, int64_t last, uint32_t *w) {
                using E = std::remove_cv_t<std::remove_pointer_t<decltype(p)>>;
                if (beside) {
                    if constexpr (sizeof(E) == 2) {
                        const Words2 q = *reinterpret_cast<const Words2Any *>(p + first);
                        w[0] = q.x, w[1] = q.y;
                    } else {
                        const Words4 q = *reinterpret_cast<const Words4Any *>(p + first);
                        w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
                    }
                    return;
                }
                step = afresh(step);
                uint32_t e4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const E *const at = p + min((int64_t)first + e, last) * step;
                    if constexpr (sizeof(E) == 2)
                        e4[e] = *at;
                    else
                        e4[e] = __float_as_uint(*at);
                }
                if constexpr (sizeof(E) == 2)
                    w[0] = e4[0] | e4[1] << 16, w[1] = e4[2] | e4[3] << 16;
                else
                    w[0] = e4[0], w[1] = e4[1], w[2] = e4[2], w[3] = e4[3];
            };
            const auto load_plane = [&](const Plane &x, const auto *base, int v0, uint32_t *w) {
                if constexpr (TF)
                    load_four(base + min(v0 + pv, A.value - 1) * x.d + t0 * x.t, x.t, x.t == 1 && t0 + C <= A.T, pt4,
                              A.T - 1 - t0, w);
                else
                    load_four(base + (t0 + min((int64_t)prow, A.T - 1 - t0)) * x.t + v0 * x.d, x.d,
                              x.d == 1 && v0 + VB <= A.value, pv4, A.value - 1 - v0, w);
            };
            const auto load_block = [&](int v0) {
                if (loads) {
                    xr = four(x_at + (int64_t)v0 * C + 4 * u);
                    wr = four(w_at + (int64_t)v0 * C + 4 * u);
                    uint32_t w[4];
                    load_plane(go, head_of<false>(go, b, h), v0, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) orr[e] = __uint_as_float(w[e]);
                    load_plane(A.v, head_of<HALF>(A.v, b, h), v0, vr);
                }
#pragma unroll
                for (int i = 0; i < kStates; ++i) {
                    const int64_t at = (int64_t)v0 * DK + 4 * (u + i * kThreads);
                    sr[i] = four(s_before + at);
                    gr[i] = four(s_behind + at);
                }
            };
            In k_raw, q_raw;
            k_raw.load(A.k, head_of<HALF>(A.k, b, hk), 0, t0, A.key, A.T, u);
            q_raw.load(A.q, head_of<HALF>(A.q, b, hk), 0, t0, A.key, A.T, u);
            load_block(0);
            if (r0 == 0) gates = use_gates<C>(A, loaded, t0);
            r1 = document_end(gates.cut, r0, rows);
            const bool before = !(gates.cut >> r0 & 1), behind = r1 == rows, whole = r0 == 0 && r1 == C;
            __syncthreads();
            if (wave == 0) write_factors(sh.F, gates, r0, r1);
            k_raw.store(sh.keys, r0, r1, A.key, u);
            q_raw.store(sh.queries, r0, r1, A.key, u);
            const Factors<C> &F = sh.F;
            auto &B = sh.block;

            f32x4 U[NT][ND], Y[NT][ND], Z[NT][ND], ow[NT], xw[NT], xv = zero;
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                ow[a] = xw[a] = zero;
#pragma unroll
                for (int c = 0; c < ND; ++c) U[a][c] = Y[a][c] = Z[a][c] = zero;
            }
            float ss = 0.0f;
            const auto values = [&]() {
                f32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (HALF)
                        x[e] = __uint_as_float(e % 2 ? vr[e / 2] & 0xffff0000u : vr[e / 2] << 16);
                    else
                        x[e] = __uint_as_float(vr[e]);
                }
                return x;
            };
            const auto store_state = [&](int tile, const f32x4 (&x)[kStates], bool there) {
#pragma unroll
                for (int i = 0; i < kStates; ++i) {
                    const int at = u + i * kThreads;
                    store4(B.s[tile], at / (DK / 4), at % (DK / 4) * 4, there ? x[i] : zero);
                }
            };
            for (int v0 = 0; v0 < A.value; v0 += VB) {
                if (v0 > 0) __syncthreads();
                if (loads) {
                    if (!whole) xr = only_steps(xr, pt4, r0, r1), wr = only_steps(wr, pt4, r0, r1);
                    store4(B.x, pv, pt4, xr);
                    store4(B.w, pv, pt4, wr);
                    f32x4 o;
                    if constexpr (TF) {
                        const bool here = v0 + pv < A.value;
                        f32x4 val = here ? values() : zero;
                        o = here && has_go ? orr : zero;
                        if (!whole) o = only_steps(o, pt4, r0, r1), val = only_steps(val, pt4, r0, r1);
#pragma unroll
                        for (int e = 0; e < 4; ++e) xv[e] = fmaf_(xr[e], val[e], xv[e]);
                        store4(B.out, pv, pt4, o);
                    } else {
                        const bool here = prow >= r0 && prow < r1;
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = here && has_go && v0 + pv4 + e < A.value ? orr[e] : 0.0f;
                        store4(B.out, prow, pv4, o);
                    }
                }
#pragma unroll
                for (int i = 0; i < kStates; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) ss = before && behind ? fmaf_(sr[i][e], gr[i][e], ss) : 0.0f;
                store_state(0, sr, before);
                if (L::kBoth) store_state(L::kBoth ? 1 : 0, gr, behind);
                __syncthreads();
                if constexpr (!TF)
                    if (loads) {
                        const f32x4 val = values();
                        const bool here = prow >= r0 && prow < r1;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (here && v0 + pv4 + e < A.value) xv[0] = fmaf_(value_at(B.x, pv4 + e, prow), val[e], xv[0]);
                    }
                const bool more = v0 + VB < A.value;
                if (L::kBoth && more) load_block(v0 + VB);
                using P = Product<Wide, Wide>;
                const auto multiply_behind = [&]() {
                    Wide gw[ND];
#pragma unroll
                    for (int c = 0; c < ND; ++c) gw[c] = operand<false>(B.s[L::kBoth ? 1 : 0], wd + 16 * c, 0);
#pragma unroll
                    for (int a = 0; a < NT; ++a) {
                        const Wide wo = operand<false>(B.w, wt + 16 * a, 0);
#pragma unroll
                        for (int i = 0; i < P::kParts; ++i)
#pragma unroll
                            for (int c = 0; c < ND; ++c) Z[a][c] = P::part(i, Z[a][c], wo, gw[c]);
                    }
                };
                Wide sw[ND];
#pragma unroll
                for (int c = 0; c < ND; ++c) sw[c] = operand<false>(B.s[0], wd + 16 * c, 0);
                const Wide wj = operand<false>(B.w, 16 * (pd < TT ? pd : 0), 0);
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    const Wide oo = operand<!TF>(B.out, wt + 16 * a, 0), xo = operand<false>(B.x, wt + 16 * a, 0);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < P::kParts; ++i) {
#pragma unroll
                        for (int c = 0; c < ND; ++c) {
                            U[a][c] = P::part(i, U[a][c], oo, sw[c]);
                            Y[a][c] = P::part(i, Y[a][c], xo, sw[c]);
                        }
                        ow[a] = P::part(i, ow[a], oo, wj);
                        xw[a] = P::part(i, xw[a], xo, wj);
                    }
                }
                if (!L::kBoth) {
                    __syncthreads();
                    store_state(0, gr, behind);
                    if (more) load_block(v0 + VB);
                    __syncthreads();
                }
                multiply_behind();
            }
            if constexpr (TF) {
#pragma unroll
                for (int o = C / 4; o < kWave; o *= 2)
#pragma unroll
                    for (int e = 0; e < 4; ++e) xv[e] += __shfl_xor(xv[e], o);
                if (lane < C / 4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sh.xv[wave][4 * lane + e] = xv[e];
            } else {
#pragma unroll
                for (int o = 1; o < VB / 4; o *= 2) xv[0] += __shfl_xor(xv[0], o);
                if (loads && u % (VB / 4) == 0) sh.xv[0][prow] = xv[0];
            }
            settle(ow);
            settle(xw);

            // E and H of the wave's rows and 16 columns, the sums of their rows and
            // columns (the LDS of the blocks is theirs from here)
            __syncthreads();
            for (int i = u; i < (int)(sizeof(sh.t) / 16); i += kThreads)
                reinterpret_cast<uint4 *>(&sh.t)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                const int it = pt * NT + a, jt = pd;
                if (jt > it) continue;
                f32x4 qk[1] = {zero}, kk[1] = {zero};
                Exact kj[KD], qi[KD], ki[KD];
#pragma unroll
                for (int d = 0; d < KD; ++d) {
                    kj[d] = operand<!TF>(sh.keys, 16 * jt, 32 * d);
                    qi[d] = operand<!TF>(sh.queries, 16 * it, 32 * d);
                    ki[d] = operand<!TF>(sh.keys, 16 * it, 32 * d);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int d = 0; d < KD; ++d) {
                    qk[0] = mma(qk[0], qi[d], kj[d]);
                    kk[0] = mma(kk[0], ki[d], kj[d]);
                }
                const int i = 16 * it + row4, j = 16 * jt + col, p = (it * kD + jt) * 16;
                const f32x4 beta = four(F.beta + i), d = decays_from(F, i, j);
                f32x4 E, H;
                float hs[4], bs[4], cs = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool in = i + e >= r0 && i + e < r1 && j >= r0 && j <= i + e;
                    E[e] = in ? A.scale * ow[a][e] * d[e] : 0.0f;
                    H[e] = in && j < i + e ? -xw[a][e] * d[e] : 0.0f;
                    hs[e] = in ? H[e] * kk[0][e] : 0.0f;
                    bs[e] = in ? fmaf_(E[e], qk[0][e], beta[e] * hs[e]) : 0.0f;
                    H[e] *= beta[e];
                    cs += bs[e];
                }
                store4(sh.t.e, j, i, E);
                store4(sh.t.h, j, i, H);
                int which;
                const float hsum = sum_columns(hs, which), bsum = sum_columns(bs, which);
                sh.h_sum[p + row4 + which] = hsum;
                sh.row_sum[p + row4 + which] = bsum;
                cs += __shfl_xor(cs, 16);
                cs += __shfl_xor(cs, 32);
                if (lane < 16) sh.col_sum[p + lane] = cs;
            }
            // the rows' products with U, Y and Z, and these as the gradients' first parts
            {
                float qu[4 * NT], ky[4 * NT], kz[4 * NT];
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    const int t = wt + 16 * a + row4;
                    const f32x4 start = four(F.start + t), end = four(F.end + t), beta = four(F.beta + t);
#pragma unroll
                    for (int e = 0; e < 4; ++e) qu[4 * a + e] = ky[4 * a + e] = kz[4 * a + e] = 0.0f;
#pragma unroll
                    for (int c = 0; c < ND; ++c) {
                        const f32x4 q = steps_of<TF>(sh.queries, wd + 16 * c + col, t);
                        const f32x4 k = steps_of<TF>(sh.keys, wd + 16 * c + col, t);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            qu[4 * a + e] = fmaf_(q[e], U[a][c][e], qu[4 * a + e]);
                            ky[4 * a + e] = fmaf_(k[e], Y[a][c][e], ky[4 * a + e]);
                            kz[4 * a + e] = fmaf_(k[e], Z[a][c][e], kz[4 * a + e]);
                        }
                        U[a][c] *= A.scale * start;
                        Z[a][c] = end * Z[a][c] - beta * start * Y[a][c];
                    }
                }
                int which;
                const float sums[3] = {sum_columns(qu, which), sum_columns(ky, which), sum_columns(kz, which)};
                const int t = wt + 16 * (which / 4) + row4 + which % 4;
#pragma unroll
                for (int i = 0; i < 3; ++i) sh.dots[i][pd][t] = sums[i];
            }
#pragma unroll
            for (int o = 1; o < kWave; o *= 2) ss += __shfl_xor(ss, o);
            if (lane == 0) sh.inner[wave] = ss;
            __syncthreads();

            Exact kt[KC][ND], qt[KC][ND];
#pragma unroll
            for (int s = 0; s < KC; ++s)
#pragma unroll
                for (int c = 0; c < ND; ++c) {
                    kt[s][c] = operand<TF>(sh.keys, wd + 16 * c, 32 * s);
                    qt[s][c] = operand<TF>(sh.queries, wd + 16 * c, 32 * s);
                }
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                const int t = wt + 16 * a;
                using P = Product<Wide, Exact>;
                // steps up to the tile's own, and from it on: the first 32 and the last 32
                // always, and of 64 the others of the tile's own half
                constexpr int kLast = KC - 1;
                const auto earlier = [&](const Wide &e, const Wide &h, int s) {
#pragma unroll
                    for (int i = 0; i < P::kParts; ++i)
#pragma unroll
                        for (int c = 0; c < ND; ++c) {
                            U[a][c] = P::part(i, U[a][c], e, kt[s][c]);
                            Z[a][c] = P::part(i, Z[a][c], h, kt[s][c]);
                        }
                };
                const auto later = [&](const Wide &e, const Wide &h, int s) {
#pragma unroll
                    for (int i = 0; i < P::kParts; ++i)
#pragma unroll
                        for (int c = 0; c < ND; ++c) {
                            Z[a][c] = P::part(i, Z[a][c], e, qt[s][c]);
                            Z[a][c] = P::part(i, Z[a][c], h, kt[s][c]);
                        }
                };
                const Wide e0 = operand<false>(sh.t.e, t, 0), h0 = operand<false>(sh.t.h, t, 0);
                const Wide e1 = operand<true>(sh.t.e, t, 32 * kLast), h1 = operand<true>(sh.t.h, t, 32 * kLast);
                __builtin_amdgcn_sched_barrier(0);
                earlier(e0, h0, 0);
                later(e1, h1, kLast);
                if constexpr (KC == 2) {
                    if (pt == 0)
                        later(operand<true>(sh.t.e, t, 0), operand<true>(sh.t.h, t, 0), 0);
                    else
                        earlier(operand<false>(sh.t.e, t, 32), operand<false>(sh.t.h, t, 32), 1);
                }
            }
#pragma unroll
            for (int c = 0; c < ND; ++c) {
                const int64_t q_step = afresh(A.dq.d), k_step = afresh(A.dk.d);
                f32x4 rows[2][NT];
#pragma unroll
                for (int a = 0; a < NT; ++a) rows[0][a] = U[a][c], rows[1][a] = Z[a][c];
                settle(rows[0]);
                settle(rows[1]);
                const int d = wd + 16 * c + col;
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    if constexpr (SHARED) {
                        dq[a][c] += only_steps(rows[0][a], wt + 16 * a + row4, r0, r1);
                        dk[a][c] += only_steps(rows[1][a], wt + 16 * a + row4, r0, r1);
                    } else if (d < A.key) {
                        store_column<HALF>(dq_at + d * q_step, A.dq.t, wt + 16 * a + row4, r0, r1, whole, rows[0][a]);
                        store_column<HALF>(dk_at + d * k_step, A.dk.t, wt + 16 * a + row4, r0, r1, whole, rows[1][a]);
                    }
                }
            }
            if (wave == 0) {
                const int row = lane;
                const bool in = row >= r0 && row < r1;
                double dG = 0.0, z = 0.0;
                if (in) {
                    const int tile = row / 16;
                    float qu = 0.0f, ky = 0.0f, kz = 0.0f, hs = 0.0f, xs = 0.0f;
                    for (int w = 0; w < kD; ++w) {
                        qu += sh.dots[0][w][row];
                        ky += sh.dots[1][w][row];
                        kz += sh.dots[2][w][row];
                    }
                    for (int j = 0; j <= tile; ++j) {
                        hs += sh.h_sum[(tile * kD + j) * 16 + row % 16];
                        dG += sh.row_sum[(tile * kD + j) * 16 + row % 16];
                    }
                    for (int i = tile; i < TT; ++i) dG -= sh.col_sum[(i * kD + tile) * 16 + row % 16];
                    for (int w = 0; w < (TF ? kWaves : 1); ++w) xs += sh.xv[w][row];
                    const float y = F.start[row] * ky;
                    z = (double)F.end[row] * kz;
                    dG += (double)(A.scale * F.start[row]) * qu - (double)F.beta[row] * y - z;
                    A.dbeta[bh * A.T + t0 + row] = xs - y + hs;
                }
                double all = z, suffix;
#pragma unroll
                for (int o = 1; o < kWave; o *= 2) all += __shfl_xor(all, o);
                if (row == r1 - 1) {
                    double inside = 0.0;
                    for (int w = 0; w < kWaves; ++w) inside += sh.inner[w];
                    dG += all + (double)F.across[0] * inside;
                }
                suffix = dG;
#pragma unroll
                for (int o = 1; o < kWave; o *= 2) {
                    const double after = __shfl_down(suffix, o);
                    if (row + o < kWave) suffix += after;
                }
                if (in && A.ddecay) A.ddecay[bh * A.T + t0 + row] = gates.cut >> row & 1 ? 0.0f : (float)suffix;
            }
        }
    }
    if constexpr (SHARED) {
        const int lane = threadIdx.x % kWave, row4 = 4 * (lane / 16), col = lane % 16;
        const int rows = (int)min((int64_t)C, A.T - t0);
#pragma unroll
        for (int c = 0; c < ND; ++c) {
            const int d = wd + 16 * c + col;
            if (d >= A.key) continue;
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                store_column<HALF>(dq_at + d * A.dq.d, A.dq.t, wt + 16 * a + row4, 0, rows, rows == C, dq[a][c]);
                store_column<HALF>(dk_at + d * A.dk.d, A.dk.t, wt + 16 * a + row4, 0, rows, rows == C, dk[a][c]);
            }
        }
    }
}

}  // namespace delta
}  // namespace pararnn
