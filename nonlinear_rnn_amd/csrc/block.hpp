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

// dw_post and dw_pre: the workgroups' partial sums, in their order.
__global__ void block_dw_kernel(BlockArgs A)
{
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= 2 * A.D) return;
    float s = 0.0f;
    for (int32_t g = 0; g < A.groups; ++g) s += A.part[(int64_t)g * 2 * A.D + d];
    if (d >= A.D)
        A.dw_pre[d - A.D] = s;
    else if (A.dw_post)
        A.dw_post[d] = s;
}

}  // namespace pararnn
