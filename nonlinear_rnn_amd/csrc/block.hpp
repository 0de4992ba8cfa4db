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
// TT consecutive steps of one row: a lane owns a channel and holds its TT
// steps, so channel-major loads use a lane's contiguous steps and time-major
// ones the wave's contiguous channels, and no transpose goes through LDS.
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
// read once for each of the two norms and once more for the result.
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
// in the workgroup's own row, between one tile and the next.
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
// A lane owns pairs of channels (2 NP of them, the workgroup's pairs apart)
// and 4 steps: channel-major loads are 16 bytes (8 in bf16) along its steps,
// time-major ones two channels wide, a wave (or, TG = 2, either half of it)
// running along the channels.  Lanes of a half wave share steps, so a sum over
// the channels is a DPP reduction, then one across waves through LDS.
//
// Workgroups are dealt to the 8 XCDs in turn: each XCD takes a contiguous
// range of tiles, so that the tiles that share a channel's cache lines (4 or
// 8 of a line's 32 float32 steps each) run together on one L2.
constexpr int kTileSteps = 4;  // steps of a lane

struct Quad {  // 4 steps of a channel, as loaded
    uint32_t w[4];
};
__device__ __forceinline__ Quad load_quad(const void *p, int64_t off, int64_t st, int n, bool bf16)
{
    Quad q;
    if (st == 1 && n >= kTileSteps) {
        if (bf16) {
            const Words2 v = *reinterpret_cast<const Words2Any *>(static_cast<const uint16_t *>(p) + off);
            q.w[0] = v.x, q.w[1] = v.y, q.w[2] = q.w[3] = 0u;
        } else {
            const Words4 v = *reinterpret_cast<const Words4Any *>(static_cast<const float *>(p) + off);
            q.w[0] = v.x, q.w[1] = v.y, q.w[2] = v.z, q.w[3] = v.w;
        }
    } else {
        uint32_t e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            e[k] = k >= n ? 0u
                   : bf16 ? static_cast<const uint16_t *>(p)[off + k * st]
                          : static_cast<const uint32_t *>(p)[off + k * st];
#pragma unroll
        for (int k = 0; k < 4; ++k) q.w[k] = e[k];
        if (bf16) q.w[0] = e[0] | e[1] << 16, q.w[1] = e[2] | e[3] << 16;
    }
    return q;
}
__device__ __forceinline__ void quad_values(const Quad &q, bool bf16, float (&v)[4])
{
    v[0] = __uint_as_float(bf16 ? q.w[0] << 16 : q.w[0]);
    v[1] = __uint_as_float(bf16 ? q.w[0] & 0xffff0000u : q.w[1]);
    v[2] = __uint_as_float(bf16 ? q.w[1] << 16 : q.w[2]);
    v[3] = __uint_as_float(bf16 ? q.w[1] & 0xffff0000u : q.w[3]);
}
__device__ __forceinline__ void store_quad(void *p, int64_t off, int64_t st, int n, bool bf16,
                                           const float (&v)[4])
{
    if (st == 1 && n >= kTileSteps) {
        if (bf16) {
            const Words2 w = {bf16_bits(v[0]) | bf16_bits(v[1]) << 16,
                              bf16_bits(v[2]) | bf16_bits(v[3]) << 16};
            *reinterpret_cast<Words2Any *>(static_cast<uint16_t *>(p) + off) = w;
        } else {
            const Words4 w = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                              __float_as_uint(v[3])};
            *reinterpret_cast<Words4Any *>(static_cast<float *>(p) + off) = w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) store_any(p, off + k * st, v[k], bf16);
    }
}
// Two neighbouring channels of a step, the second only if `two`.
__device__ __forceinline__ Words2 load_pair(const void *p, int64_t off, bool two, bool bf16)
{
    Words2 r = {0u, 0u};
    if (bf16) {
        const uint16_t *a = static_cast<const uint16_t *>(p) + off;
        r.x = two ? *reinterpret_cast<const Word1Any *>(a) : *a;
    } else {
        const uint32_t *a = static_cast<const uint32_t *>(p) + off;
        if (two)
            r = *reinterpret_cast<const Words2Any *>(a);
        else
            r.x = *a;
    }
    return r;
}
__device__ __forceinline__ float pair_value(Words2 w, int i, bool bf16)
{
    if (bf16) return __uint_as_float(i ? w.x & 0xffff0000u : w.x << 16);
    return __uint_as_float(i ? w.y : w.x);
}
__device__ __forceinline__ void store_pair(void *p, int64_t off, bool two, bool bf16, float a,
                                           float b)
{
    if (!two) {
        store_any(p, off, a, bf16);
    } else if (bf16) {
        *reinterpret_cast<Word1Any *>(static_cast<uint16_t *>(p) + off) =
            bf16_bits(a) | bf16_bits(b) << 16;
    } else {
        const Words2 w = {__float_as_uint(a), __float_as_uint(b)};
        *reinterpret_cast<Words2Any *>(static_cast<float *>(p) + off) = w;
    }
}

// Sums of N values a lane over the lanes that share its steps: the whole
// workgroup (TG = 1) or the halves of every wave (TG = 2).
template <int N, int TG, int WAVES>
struct TileSums {
    float part[N * TG][16];
    float total[TG][(N + 3) / 4 * 4];
    __device__ __forceinline__ void sum(float (&v)[N])
    {
        const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
        const int group = TG == 2 ? lane / 32 : 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x = v[i];
            x += dppf<0x111>(0.0f, x);
            x += dppf<0x112>(0.0f, x);
            x += dppf<0x114>(0.0f, x);
            x += dppf<0x118>(0.0f, x);
            x += dppf<0x142, 0xA>(0.0f, x);
            if constexpr (TG == 1) x += dppf<0x143, 0xC>(0.0f, x);
            if (lane % (kWave / TG) == kWave / TG - 1) part[i * TG + group][wave] = x;
        }
        __syncthreads();
        for (int r = threadIdx.x / 16; r < N * TG; r += WAVES * kWave / 16) {
            const int w = threadIdx.x % 16;
            float x = w < WAVES ? part[r][w] : 0.0f;
            x += dppf<0x111>(0.0f, x);
            x += dppf<0x112>(0.0f, x);
            x += dppf<0x114>(0.0f, x);
            x += dppf<0x118>(0.0f, x);
            if (w == 15) total[r % TG][r / TG] = x;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = total[group][i];
    }
};

template <int TG>
struct TileAt {
    int64_t b, t;  // row and the lane's first step
    int n;         // its steps that exist
    __device__ __forceinline__ TileAt(const BlockArgs &A, int64_t tile)
    {
        b = tile / A.tiles_per_row;
        t = (tile - b * A.tiles_per_row) * (kTileSteps * TG);
        if (TG == 2) t += threadIdx.x % kWave / 32 * kTileSteps;
        n = (int)max((int64_t)0, min((int64_t)kTileSteps, A.T - t));
    }
};
// The lane's place among the workgroup's channel pairs.
template <int TG>
__device__ __forceinline__ int pair_of_lane()
{
    return TG == 2 ? (int)(threadIdx.x / kWave * 32 + threadIdx.x % 32) : (int)threadIdx.x;
}

template <int WAVES, int TG, int NP>
__global__ void __launch_bounds__(WAVES * kWave) block_tile_kernel(BlockArgs A)
{
    constexpr int kPairs = WAVES * kWave / TG;
    __shared__ TileSums<4, TG, WAVES> sums[2];
    const int64_t tile = tile_of(blockIdx.x, A.tiles);
    if (tile >= A.tiles) return;
    const TileAt<TG> at(A, tile);
    const bool gb = A.gate_bf16, xb = A.x_bf16, zb = A.z_bf16;
    const float over_d = 1.0f / (float)A.D;
    const int64_t ho = at.b * A.hsb + at.t * A.hst, go = at.b * A.gsb + at.t * A.gst;
    const int64_t xo = at.b * A.xsb + at.t * A.xst, zo = at.b * A.zsb + at.t * A.zst;

    Quad h[NP][2], g[NP][2];
    Words2 x[NP][4];
    float wp[NP][2], wn[NP][2];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int64_t d = 2 * (pair_of_lane<TG>() + p * kPairs);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = d + i < A.D ? at.n : 0;
            h[p][i] = g[p][i] = Quad{{0u, 0u, 0u, 0u}};
            if (A.h) h[p][i] = load_quad(A.h, ho + (d + i) * A.hsd, A.hst, n, false);
            if (A.gate) g[p][i] = load_quad(A.gate, go + (d + i) * A.gsd, A.gst, n, gb);
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int64_t d = 2 * (pair_of_lane<TG>() + p * kPairs);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[p][k] = Words2{0u, 0u};
            if (k < at.n && d < A.D) x[p][k] = load_pair(A.x, xo + d + k * A.xst, d + 1 < A.D, xb);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            wp[p][i] = A.h && d + i < A.D ? A.w_post[d + i] : 0.0f;
            wn[p][i] = d + i < A.D ? A.w_pre[d + i] : 0.0f;
        }
    }
    float v[NP][2][4], r1[4] = {0.0f, 0.0f, 0.0f, 0.0f}, r2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (A.h) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float hv[4], gv[4];
                quad_values(h[p][i], false, hv);
                quad_values(g[p][i], gb, gv);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[p][i][k] = gated_value(hv[k], gv[k], A.gate);
                    r1[k] = fmaf_(v[p][i][k], v[p][i][k], r1[k]);
                }
            }
        sums[0].sum(r1);
#pragma unroll
        for (int k = 0; k < 4; ++k) r1[k] = 1.0f / sqrtf(fmaf_(r1[k], over_d, A.eps));
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int64_t d = 2 * (pair_of_lane<TG>() + p * kPairs);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float y[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                y[i] = pair_value(x[p][k], i, xb);
                if (A.h) y[i] = fmaf_(v[p][i][k] * r1[k], A.scale * wp[p][i], y[i]);
                r2[k] = fmaf_(y[i], y[i], r2[k]);
                v[p][i][k] = y[i];
            }
            if (A.y && k < at.n && d < A.D)
                store_pair(A.y, xo + d + k * A.xst, d + 1 < A.D, xb, y[0], y[1]);
        }
    }
    sums[1].sum(r2);
#pragma unroll
    for (int k = 0; k < 4; ++k) r2[k] = 1.0f / sqrtf(fmaf_(r2[k], over_d, A.eps));
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int64_t d = 2 * (pair_of_lane<TG>() + p * kPairs);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < at.n && d < A.D)
                store_pair(A.z, zo + d + k * A.zst, d + 1 < A.D, zb, v[p][0][k] * r2[k] * wn[p][0],
                           v[p][1][k] * r2[k] * wn[p][1]);
    }
    if (A.rstd && pair_of_lane<TG>() == 0)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < at.n) {
                if (A.h) A.rstd[at.b * A.T + at.t + k] = r1[k];
                A.rstd[(A.B + at.b) * A.T + at.t + k] = r2[k];
            }
}

// Backward.  The means of both norms come from one round of sums: with
// e = gy + r2 q (dx without its mean),
//     mean(p n1) = scale (mean(w_post n1 e) - r2 mean(q n2) mean(w_post n1 n2)).
// The workgroup stays, takes every A.groups-th tile of its XCD's range, and
// keeps its channels' weight gradients in registers.
template <int WAVES, int TG, int NP>
__global__ void __launch_bounds__(WAVES * kWave) block_tile_adjoint_kernel(BlockArgs A)
{
    constexpr int kPairs = WAVES * kWave / TG;
    __shared__ TileSums<12, TG, WAVES> sums;
    const bool gb = A.gate_bf16, xb = A.x_bf16, zb = A.z_bf16;
    const float over_d = 1.0f / (float)A.D;
    const int64_t per = (A.tiles + 7) >> 3, first = (blockIdx.x & 7) * per;
    float wp[NP][2], wn[NP][2], s_post[NP][2], s_pre[NP][2];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int64_t d = 2 * (pair_of_lane<TG>() + p * kPairs);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            wp[p][i] = A.h && d + i < A.D ? A.scale * A.w_post[d + i] : 0.0f;
            wn[p][i] = d + i < A.D ? A.w_pre[d + i] : 0.0f;
            s_post[p][i] = s_pre[p][i] = 0.0f;
        }
    }
    for (int64_t tile = first + (blockIdx.x >> 3); tile < min(A.tiles, first + per);
         tile += A.groups >> 3) {
        const TileAt<TG> at(A, tile);
        const int64_t ho = at.b * A.hsb + at.t * A.hst, go = at.b * A.gsb + at.t * A.gst;
        const int64_t xo = at.b * A.xsb + at.t * A.xst, zo = at.b * A.zsb + at.t * A.zst;
        Quad h[NP][2], g[NP][2];
        Words2 x[NP][4], gy[NP][4], gz[NP][4];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int64_t d = 2 * (pair_of_lane<TG>() + p * kPairs);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = d + i < A.D ? at.n : 0;
                h[p][i] = g[p][i] = Quad{{0u, 0u, 0u, 0u}};
                if (A.h) h[p][i] = load_quad(A.h, ho + (d + i) * A.hsd, A.hst, n, false);
                if (A.gate) g[p][i] = load_quad(A.gate, go + (d + i) * A.gsd, A.gst, n, gb);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = k < at.n && d < A.D, two = d + 1 < A.D;
                x[p][k] = gy[p][k] = gz[p][k] = Words2{0u, 0u};
                if (in) x[p][k] = load_pair(A.x, xo + d + k * A.xst, two, xb);
                if (in && A.gy) gy[p][k] = load_pair(A.gy, xo + d + k * A.xst, two, xb);
                if (in && A.gz) gz[p][k] = load_pair(A.gz, zo + d + k * A.zst, two, zb);
            }
        }
        float r1[4], r2[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            r1[k] = A.h && k < at.n ? A.rstd_in[at.b * A.T + at.t + k] : 0.0f;
            r2[k] = k < at.n ? A.rstd_in[(A.B + at.b) * A.T + at.t + k] : 0.0f;
        }
        float e[NP][4][2], n2[NP][4][2], s[12];
#pragma unroll
        for (int i = 0; i < 12; ++i) s[i] = 0.0f;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float hv[4], gv[4];
                quad_values(h[p][i], false, hv);
                quad_values(g[p][i], gb, gv);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float wn1 = gated_value(hv[k], gv[k], A.gate) * r1[k] * wp[p][i];
                    const float b = (wn1 + pair_value(x[p][k], i, xb)) * r2[k];
                    const float z = pair_value(gz[p][k], i, zb), q = z * wn[p][i];
                    e[p][k][i] = fmaf_(r2[k], q, pair_value(gy[p][k], i, xb));
                    n2[p][k][i] = b;
                    s[k] = fmaf_(q, b, s[k]);
                    s[4 + k] = fmaf_(wn1, e[p][k][i], s[4 + k]);
                    s[8 + k] = fmaf_(wn1, b, s[8 + k]);
                    s_pre[p][i] = fmaf_(z, b, s_pre[p][i]);
                }
            }
        sums.sum(s);
        float m1[4], m2[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m2[k] = r2[k] * (s[k] * over_d);
            m1[k] = over_d * fmaf_(-m2[k], s[8 + k], s[4 + k]);
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int64_t d = 2 * (pair_of_lane<TG>() + p * kPairs);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int i = 0; i < 2; ++i) e[p][k][i] = fmaf_(-m2[k], n2[p][k][i], e[p][k][i]);
                if (k < at.n && d < A.D)
                    store_pair(A.dx, xo + d + k * A.xst, d + 1 < A.D, xb, e[p][k][0], e[p][k][1]);
            }
            if (!A.h) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float hv[4], gv[4], dh[4], dg[4];
                quad_values(h[p][i], false, hv);
                quad_values(g[p][i], gb, gv);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float sg = A.gate ? sigmoid_q(-kLog2e * gv[k]) : 1.0f;
                    const float act = A.gate ? gv[k] * sg : 1.0f;
                    const float n1 = hv[k] * act * r1[k], dx = e[p][k][i];
                    s_post[p][i] = fmaf_(dx, n1, s_post[p][i]);
                    const float dv = r1[k] * fmaf_(-n1, m1[k], dx * wp[p][i]);
                    dh[k] = dv * act;
                    dg[k] = dv * hv[k] * (sg * fmaf_(gv[k], 1.0f - sg, 1.0f));
                }
                const int n = d + i < A.D ? at.n : 0;
                store_quad(A.dh, ho + (d + i) * A.hsd, A.hst, n, false, dh);
                if (A.gate) store_quad(A.dgate, go + (d + i) * A.gsd, A.gst, n, gb, dg);
            }
        }
    }
    float *part = A.part + (int64_t)blockIdx.x * 2 * A.D;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int64_t d = 2 * (pair_of_lane<TG>() + p * kPairs);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float a = s_post[p][i], b = s_pre[p][i];
            if (TG == 2) {  // the halves hold the same channels
                a += __shfl_xor(a, 32);
                b += __shfl_xor(b, 32);
            }
            if ((TG == 1 || threadIdx.x % kWave < 32) && d + i < A.D) {
                part[d + i] = A.scale * a;
                part[A.D + d + i] = b;
            }
        }
    }
}

// dw_post and dw_pre: the workgroups' partial sums, 64 columns a workgroup,
// its waves each a contiguous run of the rows; a fixed order.
constexpr int kDwWaves = 8;
__global__ void __launch_bounds__(kDwWaves * kWave) block_dw_kernel(BlockArgs A)
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
