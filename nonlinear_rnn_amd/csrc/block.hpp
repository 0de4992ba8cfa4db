// Block boundary: gate, norm, scale and add the states of one block to the
// residual stream, and norm the stream for the next block.  Per step, over D
// channels:
//     v = h silu(g),  n1 = v r1,  r1 = 1 / sqrt(mean v^2 + eps)
//     y = x + scale n1 w_post,  n2 = y r2,  r2 = 1 / sqrt(mean y^2 + eps)
//     z = n2 w_pre
// and backwards, from gy, gz (q = gz w_pre):
//     dx = gy + r2 (q - n2 mean(q n2)),       dw_pre  = sum gz n2
//     p = scale dx w_post
//     dv = r1 (p - n1 mean(p n1)),            dw_post = sum scale dx n1
//     dh = dv silu(g),  dg = dv h sig(g) (1 + g (1 - sig(g)))
// Everything is float32 until it is stored: z, and the next block's norm,
// see the unrounded y.
//
// The states and the gate are channel-major (a channel's steps contiguous),
// the stream is time-major (a step's channels contiguous).  A workgroup takes
// consecutive steps of one row.  A lane holds some steps of its channels (one
// channel in the strip kernels, pairs of neighbours in the register kernels),
// so channel-major loads use a lane's contiguous steps and time-major ones the
// wave's contiguous channels, and no transpose goes through LDS.
#pragma once

#include "elements.hpp"

namespace pararnn {

struct BlockArgs {
    const float *h;
    const void *gate;
    const void *x;
    const float *w_post, *w_pre;
    const float *rstd_in;
    const void *gy, *gz;
    void *y, *z;
    float *rstd;
    float *dh;
    void *dgate, *dx;
    float *part;  // backward: [workgroups][2][D] partial sums of dw_post, dw_pre
    float *dw_post, *dw_pre;
    float scale, eps;
    int64_t B, T, D;
    int64_t hsb, hsd, hst, gsb, gsd, gst, xsb, xst, zsb, zst;
    int64_t tiles, tiles_per_row;
    int32_t gate_bf16, x_bf16, z_bf16;
    int32_t has_gate, has_gy, has_gz;  // register kernels: else read but dropped
    int32_t groups;
};

__device__ __forceinline__ float load_any(const void *p, int64_t i, bool bf16)
{
    return bf16 ? load_gate<true>(p, i) : load_gate<false>(p, i);
}
__device__ __forceinline__ void store_any(void *p, int64_t i, float v, bool bf16)
{
    if (bf16)
        store_gate<true>(p, i, v);
    else
        store_gate<false>(p, i, v);
}

// Sums of TT values over the workgroup, in every thread; a fixed order.
// `lds`: TT * waves floats, free to be written once every wave is here.
template <int TT, int WAVES>
__device__ __forceinline__ void group_sum(float (&v)[TT], float *lds)
{
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TT; ++k) {
        const float s = wave_sum_to_last(v[k]);
        if (lane == kWave - 1) lds[k * WAVES + wave] = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TT; ++k) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += lds[k * WAVES + w];
        v[k] = s;
    }
}

// Tile of a workgroup: contiguous ranges of tiles on each of the 8 XCDs.
__device__ __forceinline__ int64_t tile_of(int64_t group, int64_t tiles)
{
    return (group & 7) * ((tiles + 7) >> 3) + (group >> 3);
}

constexpr int kBlockThreads = 256;
constexpr int kBlockWaves = kBlockThreads / kWave;

// h silu(g) and, backwards, d v / d g.
__device__ __forceinline__ float gated_value(float h, float g, bool has_gate)
{
    return has_gate ? h * (g * sigmoid_q(-kLog2e * g)) : h;
}

// Any width: the channels are taken in strips of the workgroup's lanes, and
// read once for each of the two norms and once more for the result.  What the
// kernels below cannot hold comes here: one channel, more than 8192, planes
// that reach past 32 bits.  Bound by the re-reads and 4-byte loads: B=8 T=4096
// D=1024 takes 1099 us here, 129 below.
template <int TT>
__global__ void __launch_bounds__(kBlockThreads) block_strip_kernel(BlockArgs A)
{
    __shared__ float lds[TT * kBlockWaves];
    const bool gb = A.gate_bf16, xb = A.x_bf16, zb = A.z_bf16;
    const float over_d = 1.0f / (float)A.D;
    for (int64_t tile = blockIdx.x; tile < A.tiles; tile += gridDim.x) {
        const int64_t b = tile / A.tiles_per_row, t0 = (tile - b * A.tiles_per_row) * TT;
        const int nt = (int)min((int64_t)TT, A.T - t0);
        const int64_t ho = b * A.hsb + t0 * A.hst, go = b * A.gsb + t0 * A.gst;
        const int64_t xo = b * A.xsb + t0 * A.xst, zo = b * A.zsb + t0 * A.zst;
        float r1[TT], r2[TT];
#pragma unroll
        for (int k = 0; k < TT; ++k) r1[k] = r2[k] = 0.0f;
        if (A.h) {
            for (int64_t d = threadIdx.x; d < A.D; d += kBlockThreads)
#pragma unroll
                for (int k = 0; k < TT; ++k) {
                    if (k >= nt) continue;
                    const float h = A.h[ho + d * A.hsd + k * A.hst];
                    const float g = A.gate ? load_any(A.gate, go + d * A.gsd + k * A.gst, gb) : 0.0f;
                    const float v = gated_value(h, g, A.gate);
                    r1[k] = fmaf_(v, v, r1[k]);
                }
            group_sum<TT, kBlockWaves>(r1, lds);
#pragma unroll
            for (int k = 0; k < TT; ++k) r1[k] = 1.0f / sqrtf(fmaf_(r1[k], over_d, A.eps));
        }
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t d = threadIdx.x; d < A.D; d += kBlockThreads) {
                const float wp = A.h ? A.scale * A.w_post[d] : 0.0f, wn = A.w_pre[d];
#pragma unroll
                for (int k = 0; k < TT; ++k) {
                    if (k >= nt) continue;
                    float y = load_any(A.x, xo + d + k * A.xst, xb);
                    if (A.h) {
                        const float h = A.h[ho + d * A.hsd + k * A.hst];
                        const float g =
                            A.gate ? load_any(A.gate, go + d * A.gsd + k * A.gst, gb) : 0.0f;
                        y = fmaf_(gated_value(h, g, A.gate) * r1[k], wp, y);
                    }
                    if (pass == 0) {
                        r2[k] = fmaf_(y, y, r2[k]);
                        if (A.y) store_any(A.y, xo + d + k * A.xst, y, xb);
                    } else {
                        store_any(A.z, zo + d + k * A.zst, y * r2[k] * wn, zb);
                    }
                }
            }
            if (pass == 0) {
                group_sum<TT, kBlockWaves>(r2, lds);
#pragma unroll
                for (int k = 0; k < TT; ++k) r2[k] = 1.0f / sqrtf(fmaf_(r2[k], over_d, A.eps));
            }
        }
        if (A.rstd && threadIdx.x == 0)
            for (int k = 0; k < nt; ++k) {
                if (A.h) A.rstd[b * A.T + t0 + k] = r1[k];
                A.rstd[(A.B + b) * A.T + t0 + k] = r2[k];
            }
    }
}

// Backward, any width; a lane's partial weight gradients are kept in `part`,
// in the workgroup's own row, between one tile and the next.  B=16 T=2048 D=4096
// takes 19.6 ms here, 1.0 below.
template <int TT>
__global__ void __launch_bounds__(kBlockThreads) block_strip_adjoint_kernel(BlockArgs A)
{
    __shared__ float lds[TT * kBlockWaves];
    const bool gb = A.gate_bf16, xb = A.x_bf16, zb = A.z_bf16;
    const float over_d = 1.0f / (float)A.D;
    float *part = A.part + (int64_t)blockIdx.x * 2 * A.D;
    for (int64_t d = threadIdx.x; d < A.D; d += kBlockThreads) part[d] = part[A.D + d] = 0.0f;
    for (int64_t tile = blockIdx.x; tile < A.tiles; tile += gridDim.x) {
        const int64_t b = tile / A.tiles_per_row, t0 = (tile - b * A.tiles_per_row) * TT;
        const int nt = (int)min((int64_t)TT, A.T - t0);
        const int64_t ho = b * A.hsb + t0 * A.hst, go = b * A.gsb + t0 * A.gst;
        const int64_t xo = b * A.xsb + t0 * A.xst, zo = b * A.zsb + t0 * A.zst;
        float r1[TT], r2[TT], m1[TT], m2[TT];
#pragma unroll
        for (int k = 0; k < TT; ++k) {
            m1[k] = m2[k] = 0.0f;
            r1[k] = A.h && k < nt ? A.rstd_in[b * A.T + t0 + k] : 0.0f;
            r2[k] = k < nt ? A.rstd_in[(A.B + b) * A.T + t0 + k] : 0.0f;
        }
        // pass 0: mean(q n2); pass 1: mean(p n1); pass 2: the results
        for (int pass = A.gz ? 0 : A.h ? 1 : 2; pass < 3; ++pass) {
            if (pass == 1 && !A.h) continue;
            for (int64_t d = threadIdx.x; d < A.D; d += kBlockThreads) {
                const float wp = A.h ? A.scale * A.w_post[d] : 0.0f, wn = A.w_pre[d];
                float s_post = 0.0f, s_pre = 0.0f;
#pragma unroll
                for (int k = 0; k < TT; ++k) {
                    if (k >= nt) continue;
                    float h = 0.0f, g = 0.0f;
                    if (A.h) h = A.h[ho + d * A.hsd + k * A.hst];
                    if (A.h && A.gate) g = load_any(A.gate, go + d * A.gsd + k * A.gst, gb);
                    const float n1 = gated_value(h, g, A.gate) * r1[k];
                    const float y = fmaf_(n1, wp, load_any(A.x, xo + d + k * A.xst, xb));
                    const float n2 = y * r2[k];
                    const float gz = A.gz ? load_any(A.gz, zo + d + k * A.zst, zb) : 0.0f;
                    const float q = gz * wn;
                    if (pass == 0) {
                        m2[k] = fmaf_(q, n2, m2[k]);
                        continue;
                    }
                    const float gy = A.gy ? load_any(A.gy, xo + d + k * A.xst, xb) : 0.0f;
                    const float dx = fmaf_(r2[k], fmaf_(-n2, m2[k], q), gy);
                    const float p = dx * wp;
                    if (pass == 1) {
                        m1[k] = fmaf_(p, n1, m1[k]);
                        continue;
                    }
                    store_any(A.dx, xo + d + k * A.xst, dx, xb);
                    s_pre = fmaf_(gz, n2, s_pre);
                    if (!A.h) continue;
                    s_post = fmaf_(dx, n1, s_post);
                    const float dv = r1[k] * fmaf_(-n1, m1[k], p);
                    const float sg = A.gate ? sigmoid_q(-kLog2e * g) : 1.0f;
                    A.dh[ho + d * A.hsd + k * A.hst] = A.gate ? dv * (g * sg) : dv;
                    if (A.gate)
                        store_any(A.dgate, go + d * A.gsd + k * A.gst,
                                  dv * h * (sg * fmaf_(g, 1.0f - sg, 1.0f)), gb);
                }
                if (pass == 2) {
                    part[d] = fmaf_(A.scale, s_post, part[d]);
                    part[A.D + d] += s_pre;
                }
            }
            if (pass == 0) group_sum<TT, kBlockWaves>(m2, lds);
            if (pass == 1) group_sum<TT, kBlockWaves>(m1, lds);
#pragma unroll
            for (int k = 0; k < TT; ++k) {
                if (pass == 0) m2[k] *= over_d;
                if (pass == 1) m1[k] *= over_d;
            }
        }
    }
}

// ------------------------------------------------------- tile in registers ---
// Up to 8192 channels: a workgroup keeps its tile of 4 TG steps in registers
// from the first load to the last store, so that every tensor is read once.
// A lane owns pairs of channels (NP pairs, the workgroup's pairs apart) and 4
// steps; TG neighbouring lanes own the same pairs and 4 steps each.  Channel-
// major loads are 16 bytes (8 in bf16) along a lane's steps, 16 TG together;
// time-major ones two channels wide, 64 / TG pairs of a step together.
//
// No load is conditional: a lane past the last channel reads the last pair
// again, is left out of the sums, and stores what that pair's lane stores; a
// row's last tile is moved back to end with the row, and the steps it shares
// with the one before are computed but neither stored nor summed.  A gradient
// or gate that is not given is read from a tensor that is, and dropped.  A
// tile's base is uniform (scalar registers), a lane's offset from it 32 bits;
// the host sends planes that reach further to the strip kernels.
//
// Planes whose steps are not contiguous, or fewer steps than a tile, load
// their 4 steps one by one (QUADS false); a missing step repeats the last one.
//
// Workgroups are dealt to the 8 XCDs in turn: each XCD takes a contiguous
// range of tiles, so that the tiles that share a channel's cache lines (4 or
// 8 of a line's 32 float32 steps each) run together on one L2.
//
// Forward, B=8 T=4096 D=1024 bf16 gate and z, float32 stream: 129 us, 4.2 of a
// copy's 5.1 TB/s (one step of 64 requests: 6 us on the device, one launch).
// Bound by HBM, and by the channel-major planes' 16- to 64-byte runs: the two
// channels of a pair are two lines.
constexpr int kTileSteps = 4;  // steps of a lane

// The types of a launch: known when it is compiled (gate, stream and normed
// stream each float32 or bf16), or read from the arguments.
constexpr int kGateBf16 = 1, kStreamBf16 = 2, kNormedBf16 = 4, kTypesFromArgs = 8;
constexpr int kNoStates = 16;  // without h: the stream's norm alone
template <int TYPES>
struct BlockTypes {
    static constexpr bool known = (TYPES & kTypesFromArgs) == 0;
    bool gate, stream, normed;
    __device__ __forceinline__ explicit BlockTypes(const BlockArgs &A)
        : gate(known ? (TYPES & kGateBf16) != 0 : A.gate_bf16 != 0),
          stream(known ? (TYPES & kStreamBf16) != 0 : A.x_bf16 != 0),
          normed(known ? (TYPES & kNormedBf16) != 0 : A.z_bf16 != 0)
    {
    }
};

__device__ __forceinline__ uint32_t opaque_bits(uint32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}
// `bytes` past a uniform address.  The address goes through an empty asm as a
// scalar register pair in the global address space: the compiler would add
// the lane's offset to the tensor's address first, to share that sum between
// rows, and hold 64 vector bits for each tensor.
#define PARARNN_GLOBAL __attribute__((address_space(1)))
template <class T>
__device__ __forceinline__ T load_at(const void *base, uint32_t bytes)
{
    uint64_t a = reinterpret_cast<uint64_t>(base);
    asm("" : "+s"(a));
    return *(const PARARNN_GLOBAL T *)((const PARARNN_GLOBAL char *)a + bytes);
}
template <class T>
__device__ __forceinline__ T load_once(const void *base, uint32_t bytes)
{
    uint64_t a = reinterpret_cast<uint64_t>(base);
    asm("" : "+s"(a));
    return __builtin_nontemporal_load((const PARARNN_GLOBAL T *)((const PARARNN_GLOBAL char *)a + bytes));
}
template <class T, class V>
__device__ __forceinline__ void store_once(void *base, uint32_t bytes, V v)
{
    uint64_t a = reinterpret_cast<uint64_t>(base);
    asm("" : "+s"(a), "+v"(bytes));
    __builtin_nontemporal_store((T)v, (PARARNN_GLOBAL T *)((PARARNN_GLOBAL char *)a + bytes));
}
template <class T, class V>
__device__ __forceinline__ void store_at(void *base, uint32_t bytes, V v)
{
    uint64_t a = reinterpret_cast<uint64_t>(base);
    asm("" : "+s"(a), "+v"(bytes));  // the offset too: it is widened where it is used
    *(PARARNN_GLOBAL T *)((PARARNN_GLOBAL char *)a + bytes) = v;
}
__device__ __forceinline__ const void *element_at(const void *p, int64_t i, bool bf16)
{
    return static_cast<const char *>(p) + (i << (bf16 ? 1 : 2));
}
__device__ __forceinline__ void *element_at(void *p, int64_t i, bool bf16)
{
    return static_cast<char *>(p) + (i << (bf16 ? 1 : 2));
}

struct Quad {  // 4 steps of a channel, as loaded: bf16 in two words, float32 in four
    uint32_t w[4];
};
// `row`: the uniform address of the lane's channel group at the tile's first
// step; step k is `step[k]` elements on.
template <bool QUADS>
__device__ __forceinline__ Quad load_quad(const void *row, uint32_t off, const int64_t (&step)[4],
                                          bool bf16)
{
    Quad q = {{0u, 0u, 0u, 0u}};
    if constexpr (QUADS) {
        if (bf16) {
            const Words2 v = load_at<Words2Any>(row, off);
            q.w[0] = v.x, q.w[1] = v.y;
        } else {
            const Words4 v = load_at<Words4Any>(row, off);
            q.w[0] = v.x, q.w[1] = v.y, q.w[2] = v.z, q.w[3] = v.w;
        }
    } else if (bf16) {
        uint32_t e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = load_at<uint16_t>(element_at(row, step[k], true), off);
        q.w[0] = e[0] | e[1] << 16, q.w[1] = e[2] | e[3] << 16;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            q.w[k] = load_at<uint32_t>(element_at(row, step[k], false), off);
    }
    return q;
}
__device__ __forceinline__ float quad_value(const Quad &q, int k, bool bf16)
{
    if (bf16) return __uint_as_float(k & 1 ? q.w[k / 2] & 0xffff0000u : q.w[k / 2] << 16);
    return __uint_as_float(q.w[k]);
}
template <bool QUADS>
__device__ __forceinline__ void store_quad(void *row, uint32_t off, const int64_t (&step)[4],
                                           const bool (&own)[4], bool all, bool bf16,
                                           const float (&v)[4])
{
    if (QUADS && all) {
        if (bf16) {
            store_at<Words2Any>(row, off, Words2{bf16_bits(v[0]) | bf16_bits(v[1]) << 16,
                                                    bf16_bits(v[2]) | bf16_bits(v[3]) << 16});
        } else {
            store_at<Words4Any>(row, off, Words4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                    __float_as_uint(v[2]), __float_as_uint(v[3])});
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (!own[k]) continue;
            void *e = element_at(row, step[k], bf16);
            if (bf16)
                store_at<uint16_t>(e, off, (uint16_t)bf16_bits(v[k]));
            else
                store_at<float>(e, off, v[k]);
        }
    }
}
// Two neighbouring channels of a step.  The stream goes past the L2's other
// contents (non-temporal), unless it is read again (`kept`): the lines of the
// channel-major planes have to stay there until all tiles that share one have
// read or written their part.  B=8 T=4096 D=1024 backward 279 -> 262 us; with
// the planes themselves non-temporal it takes twice as long.
__device__ __forceinline__ Words2 load_pair(const void *row, uint32_t off, bool bf16,
                                            bool kept = false)
{
    if (kept) {
        if (bf16) return Words2{load_at<Word1Any>(row, off), 0u};
        return load_at<Words2Any>(row, off);
    }
    if (bf16) return Words2{load_once<Word1Any>(row, off), 0u};
    return load_once<Words2Any>(row, off);
}
__device__ __forceinline__ float pair_value(Words2 w, int i, bool bf16)
{
    if (bf16) return __uint_as_float(i ? w.x & 0xffff0000u : w.x << 16);
    return __uint_as_float(i ? w.y : w.x);
}
__device__ __forceinline__ void store_pair(void *row, uint32_t off, bool bf16, float a, float b)
{
    if (bf16)
        store_once<Word1Any>(row, off, bf16_bits(a) | bf16_bits(b) << 16);
    else
        store_once<Words2Any>(row, off, Words2{__float_as_uint(a), __float_as_uint(b)});
}

// Sums of N values a lane over the lanes that share its steps (every TG-th
// lane of the workgroup).  Each row of 16 lanes by DPP, then a wave for each
// sum over the workgroup's rows, through LDS.
template <int N, int TG, int WAVES>
struct TileSums {
    float part[N * TG][WAVES * 4];
    float total[TG][(N + 3) / 4 * 4];
    __device__ __forceinline__ void sum(float (&v)[N])
    {
        const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, group = threadIdx.x % TG;
        // opaque: else the compiler sinks the sums' products below the stores
        // here, one sum's after another's, and keeps all their factors
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = opaque(v[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x = v[i];
            if constexpr (TG == 1) x += dppf<0x111>(0.0f, x);
            if constexpr (TG <= 2) x += dppf<0x112>(0.0f, x);
            x += dppf<0x114>(0.0f, x);
            x += dppf<0x118>(0.0f, x);
            if (lane % 16 >= 16 - TG) part[i * TG + group][threadIdx.x / 16] = x;
        }
        __syncthreads();
        for (int r = wave; r < N * TG; r += WAVES) {
            const float x = wave_sum_to_last(lane < WAVES * 4 ? part[r][lane] : 0.0f);
            if (lane == kWave - 1) total[r % TG][r / TG] = x;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = total[group][i];
    }
};

// A tile's place: row b, first step t, the lane's steps own[k] (all: every one).
template <int TG, bool QUADS>
struct TileAt {
    int64_t b, t;
    int group;             // the lane's 4 of the tile's steps
    int64_t k_of[4];       // offset from t of step k (of group 0 where QUADS)
    bool own[4], all;
    __device__ __forceinline__ TileAt(const BlockArgs &A, int64_t tile)
    {
        constexpr int TT = kTileSteps * TG;
        static_assert(QUADS || TG == 1, "single steps: one group");
        // tiles fit in 32 bits; the division leaves vector registers, so the
        // row is made uniform again
        const uint32_t row = __builtin_amdgcn_readfirstlane((uint32_t)tile / (uint32_t)A.tiles_per_row);
        b = row;
        const int64_t want = (tile - b * A.tiles_per_row) * TT;
        t = QUADS ? min(want, A.T - TT) : want;
        group = TG > 1 ? (int)(threadIdx.x % TG) : 0;
        all = true;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            k_of[k] = QUADS ? k : min((int64_t)k, A.T - 1 - t);
            own[k] = QUADS ? t + group * kTileSteps + k >= want : t + k < A.T;
            all = all && own[k];
        }
    }
    __device__ __forceinline__ void steps(int64_t stride, int64_t (&s)[4]) const
    {
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = k_of[k] * stride;
    }
};

// The lane's channel pair p.  Past the end, and where the last channel of an
// odd number stands alone, the pair is (D - 2, D - 1).
template <int WAVES, int TG>
struct PairAt {
    uint32_t d, group;
    bool first, second;  // which of its channels no other lane has
    __device__ __forceinline__ PairAt(const BlockArgs &A, int p)
    {
        // opaque: what follows from it is cheaper again than kept over a tile
        const uint32_t thread = opaque_bits(threadIdx.x);
        const uint32_t D = (uint32_t)A.D, want = 2u * (thread / TG + p * (WAVES * kWave / TG));
        group = thread % TG;
        d = min(want, D - 2);
        first = want + 1 < D;
        second = want < D;
    }
    // Byte offsets from the tile's base.
    __device__ __forceinline__ uint32_t in_plane(int64_t stride_d, bool bf16) const
    {
        return (d * (uint32_t)stride_d + kTileSteps * group) << (bf16 ? 1 : 2);
    }
    __device__ __forceinline__ uint32_t in_row(int64_t stride_t, bool bf16) const
    {
        return (d + group * kTileSteps * (uint32_t)stride_t) << (bf16 ? 1 : 2);
    }
};

template <int WAVES, int TG, int NP, bool QUADS, int TYPES>
__global__ void __launch_bounds__(WAVES * kWave) block_tile_kernel(BlockArgs A)
{
    __shared__ TileSums<4, TG, WAVES> sums[2];
    const int64_t tile = tile_of(blockIdx.x, A.tiles);
    if (tile >= A.tiles) return;
    const TileAt<TG, QUADS> at(A, tile);
    const BlockTypes<TYPES> types(A);
    const bool gb = types.gate, xb = types.stream, zb = types.normed;
    constexpr bool kStates = (TYPES & kNoStates) == 0;
    [[maybe_unused]] const bool has_gate = A.has_gate;
    const float over_d = 1.0f / (float)A.D;
    int64_t hk[4], gk[4], xk[4], zk[4];
    at.steps(A.hst, hk), at.steps(A.gst, gk), at.steps(A.xst, xk), at.steps(A.zst, zk);
    const int64_t xo = at.b * A.xsb + at.t * A.xst, zo = at.b * A.zsb + at.t * A.zst;

    Quad h[NP][2], g[NP][2];
    Words2 x[NP][4];
    float wp[NP][2], wn[NP][2];
    const float *h_row = A.h + at.b * A.hsb + at.t * A.hst;
    const void *g_row = element_at(A.gate, at.b * A.gsb + at.t * A.gst, gb);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const PairAt<WAVES, TG> c(A, p);
        const uint32_t hoff = c.in_plane(A.hsd, false), goff = c.in_plane(A.gsd, gb);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (kStates) {
                h[p][i] = load_quad<QUADS>(h_row + i * A.hsd, hoff, hk, false);
                g[p][i] = load_quad<QUADS>(element_at(g_row, i * A.gsd, gb), goff, gk, gb);
            }
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const PairAt<WAVES, TG> c(A, p);
        const uint32_t xoff = c.in_row(A.xst, xb);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[p][k] = load_pair(element_at(A.x, xo + xk[k], xb), xoff, xb);
        wn[p][0] = A.w_pre[c.d], wn[p][1] = A.w_pre[c.d + 1];
        if constexpr (kStates)
            wp[p][0] = A.scale * A.w_post[c.d], wp[p][1] = A.scale * A.w_post[c.d + 1];
    }
    float v[NP][2][4], r1[4] = {0.0f, 0.0f, 0.0f, 0.0f}, r2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (kStates) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const PairAt<WAVES, TG> c(A, p);
                const bool counts = i ? c.second : c.first;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[p][i][k] = gated_value(quad_value(h[p][i], k, false),
                                             quad_value(g[p][i], k, gb), has_gate);
                    const float s = counts ? v[p][i][k] : 0.0f;
                    r1[k] = fmaf_(s, s, r1[k]);
                }
            }
        sums[0].sum(r1);
#pragma unroll
        for (int k = 0; k < 4; ++k) r1[k] = 1.0f / sqrtf(fmaf_(r1[k], over_d, A.eps));
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const PairAt<WAVES, TG> c(A, p);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float y = pair_value(x[p][k], i, xb);
                if constexpr (kStates) y = fmaf_(v[p][i][k] * r1[k], wp[p][i], y);
                const float s = (i ? c.second : c.first) ? y : 0.0f;
                r2[k] = fmaf_(s, s, r2[k]);
                v[p][i][k] = y;
            }
            if (A.y && (at.all || at.own[k]))
                store_pair(element_at(A.y, xo + xk[k], xb), c.in_row(A.xst, xb), xb, v[p][0][k],
                           v[p][1][k]);
        }
    }
    sums[1].sum(r2);
#pragma unroll
    for (int k = 0; k < 4; ++k) r2[k] = 1.0f / sqrtf(fmaf_(r2[k], over_d, A.eps));
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const uint32_t zoff = PairAt<WAVES, TG>(A, p).in_row(A.zst, zb);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (at.all || at.own[k])
                store_pair(element_at(A.z, zo + zk[k], zb), zoff, zb, v[p][0][k] * r2[k] * wn[p][0],
                           v[p][1][k] * r2[k] * wn[p][1]);
    }
    if (A.rstd && threadIdx.x < TG)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (at.own[k]) {
                const int64_t t = at.t + at.group * 4 + k;
                if (kStates) A.rstd[at.b * A.T + t] = r1[k];
                A.rstd[(A.B + at.b) * A.T + t] = r2[k];
            }
}

// Backward.  The means of both norms come from one round of sums: with
// e = gy + r2 q (dx without its mean),
//     mean(p n1) = scale (mean(w_post n1 e) - r2 mean(q n2) mean(w_post n1 n2)).
// The workgroup stays, takes every (groups / 8)-th tile of its XCD's range, and
// keeps its channels' weight gradients.  The states and the gate stay in
// registers between the sums and the results, e waits in LDS, and x is read
// again (just read, and in long runs).  The channel pairs follow one another,
// the next one's loads issued before the current one is computed.
//
// B=16 T=2048 D=4096: 997 us of 684 at a copy's rate.  4.5 GB go instead of
// 3.5, at 4.5 TB/s: x twice, and dh and dgate in parts of lines (without their
// stores 726 us).  A CU's registers hold 8 steps of 4096 channels, 32 bytes of
// a line, and the L2 has to put the parts together.  B=3 T=1531 D=2000 float32:
// 101 us of 54, 576 tiles on 256 CUs.  Tiles of 4 steps that keep x too took
// 1141 us of the first, reading the gradients again as well 1880, a kernel for
// the sums and one to apply them 1404.
//
// 4097 to 8192 channels: 16 waves, and 128 registers a lane for them; 18 to 86
// are spilled.  B=4 T=2048 D=8192 bf16 gate, float32 stream 706 us (strip
// kernel 6243), forward, which spills none, 311 (2979).  With a float32 normed
// stream, types read from the arguments, the tilings of 8 pairs spill 7 to 19 of
// 256; with float32 gate and stream those of 2048 and 4096 channels 3 and 4.
struct StreamPair {
    Words2 x[4], gy[4], gz[4];
    float wp[2], wn[2];
};

template <int WAVES, int TG, int NP, bool QUADS, int TYPES>
__global__ void __launch_bounds__(WAVES * kWave, 2) block_tile_adjoint_kernel(BlockArgs A)
{
    __shared__ TileSums<12, TG, WAVES> sums;
    __shared__ float4 e_lds[NP * 2][WAVES * kWave];
    const BlockTypes<TYPES> types(A);
    const bool gb = types.gate, xb = types.stream, zb = types.normed;
    constexpr bool kStates = (TYPES & kNoStates) == 0;
    [[maybe_unused]] const bool has_gate = A.has_gate;
    const bool has_gy = A.has_gy, has_gz = A.has_gz;
    const float over_d = 1.0f / (float)A.D;
    const int64_t per = (A.tiles + 7) >> 3, begin = (blockIdx.x & 7) * per;
    const int64_t end = min(A.tiles, begin + per);
    float s_post[NP][2], s_pre[NP][2];
#pragma unroll
    for (int p = 0; p < NP; ++p) s_post[p][0] = s_post[p][1] = s_pre[p][0] = s_pre[p][1] = 0.0f;

    for (int64_t tile = begin + (blockIdx.x >> 3); tile < end; tile += A.groups >> 3) {
        const TileAt<TG, QUADS> at(A, tile);
        int64_t hk[4], gk[4], xk[4], zk[4];
        at.steps(A.hst, hk), at.steps(A.gst, gk), at.steps(A.xst, xk), at.steps(A.zst, zk);
        const int64_t ho = at.b * A.hsb + at.t * A.hst, go = at.b * A.gsb + at.t * A.gst;
        const int64_t xo = at.b * A.xsb + at.t * A.xst, zo = at.b * A.zsb + at.t * A.zst;
        const auto load_stream = [&](int p, bool again) {
            const PairAt<WAVES, TG> c(A, p);
            const uint32_t xoff = c.in_row(A.xst, xb), zoff = c.in_row(A.zst, zb);
            StreamPair v;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v.x[k] = load_pair(element_at(A.x, xo + xk[k], xb), xoff, xb, !again);
                if (again) continue;
                v.gy[k] = load_pair(element_at(A.gy, xo + xk[k], xb), xoff, xb);
                v.gz[k] = load_pair(element_at(A.gz, zo + zk[k], zb), zoff, zb);
            }
            if (!again) {
                const Words2 w = load_at<Words2Any>(A.w_pre, c.d * 4);
                v.wn[0] = __uint_as_float(w.x), v.wn[1] = __uint_as_float(w.y);
            }
            if constexpr (kStates) {
                const Words2 w = load_at<Words2Any>(A.w_post, c.d * 4);
                v.wp[0] = __uint_as_float(w.x), v.wp[1] = __uint_as_float(w.y);
            }
            return v;
        };
        Quad h[NP][2], g[NP][2];
        if constexpr (kStates)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const PairAt<WAVES, TG> c(A, p);
                const uint32_t hoff = c.in_plane(A.hsd, false), goff = c.in_plane(A.gsd, gb);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    h[p][i] = load_quad<QUADS>(A.h + ho + i * A.hsd, hoff, hk, false);
                    g[p][i] = load_quad<QUADS>(element_at(A.gate, go + i * A.gsd, gb), goff, gk, gb);
                }
            }
        // a step that is not the tile's own has no norms, so it adds nothing to
        // the weight gradients
        float r1[4], r2[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t t = at.t + at.group * kTileSteps + at.k_of[k];
            const float r = kStates ? A.rstd_in[at.b * A.T + t] : 0.0f;
            const float q = A.rstd_in[(A.B + at.b) * A.T + t];
            r1[k] = at.own[k] ? r : 0.0f;
            r2[k] = at.own[k] ? q : 0.0f;
        }
        float s[12];
#pragma unroll
        for (int i = 0; i < 12; ++i) s[i] = 0.0f;
        StreamPair now = load_stream(0, false);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            StreamPair next;
            if (p + 1 < NP) next = load_stream(p + 1, false);
            __builtin_amdgcn_sched_barrier(0);
            const PairAt<WAVES, TG> c(A, p);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool counts = i ? c.second : c.first;
                const float wp = kStates ? A.scale * now.wp[i] : 0.0f;
                float e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float n1w = 0.0f;
                    if constexpr (kStates)
                        n1w = gated_value(quad_value(h[p][i], k, false), quad_value(g[p][i], k, gb),
                                          has_gate) * r1[k] * wp;
                    const float n2 = (n1w + pair_value(now.x[k], i, xb)) * r2[k];
                    const float z = has_gz ? pair_value(now.gz[k], i, zb) : 0.0f, q = z * now.wn[i];
                    e[k] = fmaf_(r2[k], q, has_gy ? pair_value(now.gy[k], i, xb) : 0.0f);
                    s_pre[p][i] = fmaf_(z, n2, s_pre[p][i]);
                    s[k] = fmaf_(counts ? q : 0.0f, n2, s[k]);
                    if constexpr (kStates) {
                        n1w = counts ? n1w : 0.0f;
                        s[4 + k] = fmaf_(n1w, e[k], s[4 + k]);
                        s[8 + k] = fmaf_(n1w, n2, s[8 + k]);
                    }
                }
                e_lds[2 * p + i][threadIdx.x] = make_float4(e[0], e[1], e[2], e[3]);
            }
            // opaque: else the sums' products sink below the next pair, and
            // their factors are kept
#pragma unroll
            for (int i = 0; i < 12; ++i) s[i] = opaque(s[i]);
            s_pre[p][0] = opaque(s_pre[p][0]), s_pre[p][1] = opaque(s_pre[p][1]);
            now = next;
        }
        now = load_stream(0, true);
        sums.sum(s);
        float m1[4], m2[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m2[k] = r2[k] * r2[k] * (s[k] * over_d);
            m1[k] = over_d * fmaf_(-r2[k] * (s[k] * over_d), s[8 + k], s[4 + k]);
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            StreamPair next;
            if (p + 1 < NP) next = load_stream(p + 1, true);
            __builtin_amdgcn_sched_barrier(0);
            const PairAt<WAVES, TG> c(A, p);
            float dx[4][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 e4 = e_lds[2 * p + i][threadIdx.x];
                const float e[4] = {e4.x, e4.y, e4.z, e4.w};
                const float wp = kStates ? A.scale * now.wp[i] : 0.0f;
                float dh[4], dg[4];
                // opaque: the sigmoids are cheaper again than kept since the sums
                if constexpr (kStates)
#pragma unroll
                    for (int j = 0; j < (gb ? 2 : 4); ++j) g[p][i].w[j] = opaque_bits(g[p][i].w[j]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float hv = 0.0f, gv = 0.0f, sg = 1.0f, act = 1.0f, n1 = 0.0f;
                    float y = pair_value(now.x[k], i, xb);
                    if constexpr (kStates) {
                        hv = quad_value(h[p][i], k, false), gv = quad_value(g[p][i], k, gb);
                        if (has_gate) sg = sigmoid_q(-kLog2e * gv), act = gv * sg;
                        n1 = hv * act * r1[k];
                        y = fmaf_(n1, wp, y);
                    }
                    dx[k][i] = fmaf_(-m2[k], y, e[k]);
                    if constexpr (kStates) {
                        s_post[p][i] = fmaf_(dx[k][i], n1, s_post[p][i]);
                        const float dv = r1[k] * fmaf_(-n1, m1[k], dx[k][i] * wp);
                        dh[k] = dv * act;
                        dg[k] = dv * hv * (sg * fmaf_(gv, 1.0f - sg, 1.0f));
                    }
                }
                if constexpr (kStates) {
                    store_quad<QUADS>(A.dh + ho + i * A.hsd, c.in_plane(A.hsd, false), hk, at.own,
                                      at.all, false, dh);
                    if (has_gate)
                        store_quad<QUADS>(element_at(A.dgate, go + i * A.gsd, gb),
                                          c.in_plane(A.gsd, gb), gk, at.own, at.all, gb, dg);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (at.all || at.own[k])
                    store_pair(element_at(A.dx, xo + xk[k], xb), c.in_row(A.xst, xb), xb, dx[k][0],
                               dx[k][1]);
            s_post[p][0] = opaque(s_post[p][0]), s_post[p][1] = opaque(s_post[p][1]);
            now = next;
        }
    }
    float *part = A.part + (int64_t)blockIdx.x * 2 * A.D;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const PairAt<WAVES, TG> c(A, p);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float a = s_post[p][i], b = s_pre[p][i];
#pragma unroll
            for (int o = 1; o < TG; o *= 2) {  // the groups hold the same channels
                a += __shfl_xor(a, o);
                b += __shfl_xor(b, o);
            }
            if (threadIdx.x % TG == 0 && (i ? c.second : c.first)) {
                part[c.d + i] = A.scale * a;
                part[A.D + c.d + i] = b;
            }
        }
    }
}

// dw_post and dw_pre: the workgroups' partial sums, 64 columns a workgroup,
// its waves each a contiguous run of the rows; a fixed order.
constexpr int kDwWaves = 8;
static __global__ void __launch_bounds__(kDwWaves * kWave) block_dw_kernel(BlockArgs A)
{
    __shared__ float lds[kDwWaves][kWave];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int64_t d = (int64_t)blockIdx.x * kWave + lane;
    const int per = (A.groups + kDwWaves - 1) / kDwWaves;
    float s = 0.0f;
    if (d < 2 * A.D)
#pragma unroll 8
        for (int g = wave * per; g < min(A.groups, (wave + 1) * per); ++g)
            s += A.part[(int64_t)g * 2 * A.D + d];
    lds[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || d >= 2 * A.D) return;
    for (int w = 1; w < kDwWaves; ++w) s += lds[w][lane];
    if (d >= A.D)
        A.dw_pre[d - A.D] = s;
    else if (A.dw_post)
        A.dw_post[d] = s;
}

}  // namespace pararnn
