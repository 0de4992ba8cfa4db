// Gated linear recurrence: host side of pararnn_gated_scan,
// pararnn_gated_scan_adjoint and pararnn_gated_step.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "gated.hpp"
#include "host.hpp"

using namespace pararnn;

namespace {

// Steps a lane holds in the kernels with lanes in time: one 16-byte load a
// plane.
constexpr int kStepsBf16 = 8, kStepsF32 = 4;

// Which kernel, and how the time axis is cut: spans per channel and their
// length.
struct GatedPlan {
    int64_t channels = 0, seg_len = 0;
    int32_t nseg = 1;
    int waves = 0;  // per channel, lanes in time; 0: a lane per channel
    size_t agg = 0, part = 0, total = 0;  // workspace: span maps, dlam partial sums
};

// The plan goes by the shape alone (not by the dtype), so that a workspace
// serves either.
pararnn_status_t gated_plan(const pararnn_shape_t *sh, bool adjoint, GatedPlan &pl)
{
    const pararnn_status_t st = check_shape(sh);
    if (st != PARARNN_OK) return st;
    if (sh->B > 0 && sh->D > ((int64_t(1) << 31) - 1) / sh->B) return PARARNN_ERR_UNSUPPORTED;
    pl.channels = sh->B * sh->D;
    const int64_t C = pl.channels, T = sh->T;
    constexpr int64_t kFull = 8 * kComputeUnits;  // waves that fill the device
    int64_t nseg = 1, unit = 1;
    // (a dispatch counts its work-items in 32 bits: 64 a channel)
    if (T > 2 && sh->u_stride_t == 1 && sh->s_stride_t == 1 && C < (int64_t(1) << 26)) {
        // one wave per channel where the channels fill the device, else the
        // channel's steps over 4 or 8 waves, and over workgroups where those
        // leave the device less than full (spans read their projections twice:
        // then as many as 32 waves a CU)
        pl.waves = C >= kFull || T <= 64 * kStepsBf16       ? 1
                   : C >= kFull / 4 || T <= 256 * kStepsBf16 ? 4
                                                             : 8;
        unit = (int64_t)pl.waves * kWave * kStepsBf16;
        if (C > 0 && C * pl.waves < kFull) nseg = (4 * kFull + C * pl.waves - 1) / (C * pl.waves);
        nseg = std::min(nseg, (T + 2 * unit - 1) / (2 * unit));
    } else {
        // a lane per channel: spans of at least 64 steps
        const int64_t waves = (C + kWave - 1) / kWave;
        nseg = waves > 0 ? 2 * kFull / waves : 1;
        nseg = std::min(nseg, (T + 63) / 64);
    }
    nseg = std::max<int64_t>(1, std::min<int64_t>(nseg, 4096));
    pl.seg_len = std::max<int64_t>(unit, ((T + nseg - 1) / nseg + unit - 1) / unit * unit);
    pl.nseg = (int32_t)std::max<int64_t>(1, (T + pl.seg_len - 1) / pl.seg_len);
    pl.agg = 0;
    size_t off = pl.nseg > 1 ? align_up((size_t)pl.nseg * C * sizeof(float2)) : 0;
    pl.part = off;
    if (adjoint) off = align_up(off + (size_t)sh->B * pl.nseg * sh->D * sizeof(float));
    pl.total = off;
    return PARARNN_OK;
}

void gated_args(GatedArgs &A, const pararnn_shape_t *sh, const GatedPlan &pl, const void *const *u,
                const float *lam, float power, const float *h0, const uint8_t *resets, void *ws)
{
    std::memset(&A, 0, sizeof(A));
    for (int g = 0; g < 3 && u; ++g) A.u[g] = u[g];
    A.lam = lam;
    A.power = power;
    A.h0 = h0;
    A.resets = resets;
    A.agg = reinterpret_cast<float2 *>(static_cast<char *>(ws) + pl.agg);
    A.seg_len = pl.seg_len;
    A.nseg = pl.nseg;
    A.B = sh->B;
    A.T = sh->T;
    A.D = sh->D;
    A.channels = pl.channels;
    A.usb = sh->u_stride_b;
    A.usd = sh->u_stride_d;
    A.ust = sh->u_stride_t;
    A.ssb = sh->s_stride_b;
    A.ssd = sh->s_stride_d;
    A.sst = sh->s_stride_t;
}

pararnn_status_t check_gated(const pararnn_shape_t *sh, const GatedPlan &pl, const void *const *u,
                             pararnn_dtype_t dt, const float *lam, float power, const void *ws,
                             size_t ws_bytes)
{
    if (dt != PARARNN_F32 && dt != PARARNN_BF16) return PARARNN_ERR_UNSUPPORTED;
    if (!(power > 0.0f) || std::isinf(power)) return PARARNN_ERR_INVALID;
    if (pl.channels > 0 && !lam) return PARARNN_ERR_INVALID;
    if (pl.channels > 0 && sh->T > 0) {
        if (!u) return PARARNN_ERR_INVALID;
        for (int g = 0; g < 3; ++g)
            if (!u[g]) return PARARNN_ERR_INVALID;
    }
    if (pl.total > 0 && pl.channels > 0 && (!ws || ws_bytes < pl.total || !aligned16(ws)))
        return PARARNN_ERR_WORKSPACE;
    return PARARNN_OK;
}

// One launch over (channels or groups of 64 of them) x spans.
template <bool ADJ, bool BF16, bool AGG>
hipError_t launch_gated(const GatedArgs &A, int waves, hipStream_t st)
{
    constexpr int K = BF16 ? kStepsBf16 : kStepsF32;
    const int64_t groups = waves ? A.channels : (A.channels + kWave - 1) / kWave;
    // (the last span's map, or backwards the first one's, is nobody's carry)
    const dim3 grid((unsigned)groups, (unsigned)(A.nseg - (AGG ? 1 : 0))),
        block((unsigned)(kWave * (waves ? waves : 1)));
#define PARARNN_GATED(NAME, ...)                                                                 \
    if constexpr (ADJ)                                                                           \
        hipLaunchKernelGGL((gated_##NAME##_adjoint_kernel<__VA_ARGS__>), grid, block, 0, st, A); \
    else                                                                                         \
        hipLaunchKernelGGL((gated_##NAME##_kernel<__VA_ARGS__>), grid, block, 0, st, A)
    if constexpr (!AGG)
        if (waves == 1 && A.nseg == 1 && A.T <= 16 * K) {
            const int lanes = A.T <= 4 * K ? 4 : 16;
            const dim3 few((unsigned)((A.channels * lanes + kShortThreads - 1) / kShortThreads)),
                wide(kShortThreads);
            if (lanes == 4 && ADJ)
                hipLaunchKernelGGL((gated_short_adjoint_kernel<BF16, K, 4>), few, wide, 0, st, A);
            else if (lanes == 4)
                hipLaunchKernelGGL((gated_short_kernel<BF16, K, 4>), few, wide, 0, st, A);
            else if (ADJ)
                hipLaunchKernelGGL((gated_short_adjoint_kernel<BF16, K, 16>), few, wide, 0, st, A);
            else
                hipLaunchKernelGGL((gated_short_kernel<BF16, K, 16>), few, wide, 0, st, A);
            return hipGetLastError();
        }
    switch (waves) {
    case 8: PARARNN_GATED(time, BF16, K, 8, AGG); break;
    case 4: PARARNN_GATED(time, BF16, K, 4, AGG); break;
    case 1: PARARNN_GATED(time, BF16, K, 1, AGG); break;
    default: PARARNN_GATED(channel, BF16, AGG); break;
    }
#undef PARARNN_GATED
    return hipGetLastError();
}

template <bool ADJ>
hipError_t run_gated(const GatedArgs &A, int waves, bool bf16, hipStream_t st)
{
    if (A.nseg > 1) {
        const hipError_t e = bf16 ? launch_gated<ADJ, true, true>(A, waves, st)
                                  : launch_gated<ADJ, false, true>(A, waves, st);
        if (e != hipSuccess) return e;
    }
    return bf16 ? launch_gated<ADJ, true, false>(A, waves, st)
                : launch_gated<ADJ, false, false>(A, waves, st);
}

}  // namespace

extern "C" {

size_t pararnn_gated_workspace_bytes(const pararnn_shape_t *shape, int adjoint)
{
    GatedPlan pl;
    return gated_plan(shape, adjoint != 0, pl) == PARARNN_OK ? pl.total : 0;
}

pararnn_status_t pararnn_gated_scan(const pararnn_shape_t *shape, const void *const u[3],
                                    pararnn_dtype_t u_dtype, const float *lam, float power,
                                    const float *h0, const uint8_t *resets, float *h,
                                    float *h_last, void *ws, size_t ws_bytes, void *stream)
{
    GatedPlan pl;
    pararnn_status_t st = gated_plan(shape, false, pl);
    if (st != PARARNN_OK) return st;
    st = check_gated(shape, pl, u, u_dtype, lam, power, ws, ws_bytes);
    if (st != PARARNN_OK) return st;
    if (pl.channels == 0 || (shape->T == 0 && !h_last)) return PARARNN_OK;
    if (shape->T > 0 && !h) return PARARNN_ERR_INVALID;
    GatedArgs A;
    gated_args(A, shape, pl, u, lam, power, h0, resets, ws);
    A.h = h;
    A.h_last = h_last;
    const hipError_t e =
        run_gated<false>(A, pl.waves, u_dtype == PARARNN_BF16, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

pararnn_status_t pararnn_gated_scan_adjoint(const pararnn_shape_t *shape, const void *const u[3],
                                            pararnn_dtype_t u_dtype, const float *lam, float power,
                                            const float *h0, const uint8_t *resets,
                                            const float *h, const float *gh, const float *gh_last,
                                            void *const du[3], float *dlam, float *dh0, void *ws,
                                            size_t ws_bytes, void *stream)
{
    GatedPlan pl;
    pararnn_status_t st = gated_plan(shape, true, pl);
    if (st != PARARNN_OK) return st;
    st = check_gated(shape, pl, u, u_dtype, lam, power, ws, ws_bytes);
    if (st != PARARNN_OK) return st;
    if (shape->D == 0) return PARARNN_OK;
    if (!dlam || !lam) return PARARNN_ERR_INVALID;
    if (pl.channels > 0 && shape->T > 0) {
        if (!h || !du) return PARARNN_ERR_INVALID;
        for (int g = 0; g < 3; ++g)
            if (!du[g]) return PARARNN_ERR_INVALID;
    }
    hipStream_t strm = static_cast<hipStream_t>(stream);
    GatedArgs A;
    gated_args(A, shape, pl, u, lam, power, h0, resets, ws);
    A.hs = h;
    A.gh = gh;
    A.gh_last = gh_last;
    for (int g = 0; g < 3 && du; ++g) A.du[g] = du[g];
    A.dlam = dlam;
    A.dh0 = dh0;
    A.dlam_part = reinterpret_cast<float *>(static_cast<char *>(ws) + pl.part);
    if (pl.channels > 0 && run_gated<true>(A, pl.waves, u_dtype == PARARNN_BF16, strm) != hipSuccess)
        return PARARNN_ERR_HIP;
    const int tpb = 256;  // no batch rows: a sum of no terms
    hipLaunchKernelGGL(gated_dlam_kernel, dim3((unsigned)((shape->D + tpb - 1) / tpb)), dim3(tpb),
                       0, strm, A);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

pararnn_status_t pararnn_gated_step(int64_t B, int64_t D, const void *const u[3],
                                    pararnn_dtype_t u_dtype, int64_t u_stride_b, const float *lam,
                                    float power, const int32_t *slots, float *states, int64_t pool,
                                    float *out, void *stream)
{
    if (B < 0 || D < 0 || pool < 0) return PARARNN_ERR_INVALID;
    if (B >= (int64_t(1) << 31) || D >= (int64_t(1) << 31) || pool >= (int64_t(1) << 31))
        return PARARNN_ERR_UNSUPPORTED;
    if (u_dtype != PARARNN_F32 && u_dtype != PARARNN_BF16) return PARARNN_ERR_UNSUPPORTED;
    if (!(power > 0.0f) || std::isinf(power)) return PARARNN_ERR_INVALID;
    if (B > 1 && u_stride_b < D) return PARARNN_ERR_INVALID;
    if (B == 0 || D == 0) return PARARNN_OK;
    if (!u || !lam || !out || (pool > 0 && !states)) return PARARNN_ERR_INVALID;
    for (int g = 0; g < 3; ++g)
        if (!u[g]) return PARARNN_ERR_INVALID;
    GatedStepArgs A;
    for (int g = 0; g < 3; ++g) A.u[g] = u[g];
    A.lam = lam;
    A.slots = slots;
    A.states = states;
    A.out = out;
    A.B = B;
    A.D = D;
    A.usb = u_stride_b;
    A.pool = pool;
    A.power = power;
    const dim3 grid((unsigned)((D + kGatedStepThreads - 1) / kGatedStepThreads),
                    (unsigned)std::min<int64_t>(B, 65535)),
        block(kGatedStepThreads);
    hipStream_t strm = static_cast<hipStream_t>(stream);
    if (u_dtype == PARARNN_BF16)
        hipLaunchKernelGGL((gated_step_kernel<true>), grid, block, 0, strm, A);
    else
        hipLaunchKernelGGL((gated_step_kernel<false>), grid, block, 0, strm, A);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

}  // extern "C"
