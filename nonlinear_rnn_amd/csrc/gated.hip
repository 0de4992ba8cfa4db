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
// Look back: what a chunk costs beside its bytes wants it long.  Float32,
// 1x262144x64 with part of its inputs still cached: 8 waves of 4 steps a lane
// 74.7 us, 4 of 8 64.4, 8 of 8 58.5 (from HBM 72).  16 waves of 8 take 65 us from
// HBM, but more than 8 elsewhere (bfloat16: backward 106 and 95, 2x16577x91 22
// and 18).
constexpr int kLookWaves = 8, kLookSteps = 8, kLookChunk = kLookWaves * kWave * kLookSteps;

// A dispatch's work-items in 32 bits, 512 a chunk.
constexpr int64_t kMostChunks = int64_t(1) << 23;

// Which kernel, and how the time axis is cut.
enum GatedKernel { kLanePerChannel, kLaneLookBack, kWavePerChannel, kGroupPerChannel, kLookBack };
struct GatedPlan {
    GatedKernel kernel = kLanePerChannel;
    int64_t channels = 0;
    int64_t chunks = 1;  // look back: places
    // workspace: tickets, the records' place, dlam partial sums
    size_t records = 0, part = 0, total = 0;
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
    size_t record = 0, lines = 0;
    // (a dispatch counts its work-items in 32 bits: 64 a channel)
    if (T > 6 && sh->u_stride_t == 1 && sh->s_stride_t == 1 && C < (int64_t(1) << 26)) {
        // Lanes in time; up to 6 steps a lane has all of its channel's (512
        // requests of 1024 channels: 6 steps bfloat16 47 us with lanes in time,
        // 13 with a lane per channel, 8 steps float32 25 and 31).
        // One wave a channel for sequences up to 512 steps, and up to 4095
        // where the channels fill the device (16 x 1024 channels of 600 steps
        // float32 35 us, with 4 waves 41; 8 x 1024 of 4096 steps, backward, 146
        // and 128), or longer if 4 waves' last chunk is mostly empty (4500 steps
        // bfloat16, backward, 178 and 219).  4 waves, and where they do not fill
        // the device, the channel's chunks side by side (2x65536x128 float32
        // 95 us with 4 waves, 58 looking back; 4x8192x256 bfloat16, 1024
        // channels, 19 and 24).
        const int64_t chunks = (T + kLookChunk - 1) / kLookChunk;
        constexpr int64_t four = 4 * kWave * kStepsBf16;
        const bool full = T >= 4096 && (T + four - 1) / four * four - T <= T / 8;
        pl.kernel = T <= kWave * kStepsBf16 || (C >= kFull && !full) ? kWavePerChannel
                    : C >= kFull / 4 || chunks <= 1                  ? kGroupPerChannel
                                                                     : kLookBack;
        if (pl.kernel == kLookBack && C * chunks >= kMostChunks) pl.kernel = kGroupPerChannel;
        if (pl.kernel == kLookBack) pl.chunks = chunks, record = sizeof(GatedRecord), lines = C;
    } else {
        // A lane per channel, one for the whole length of a short sequence
        // (64 x 1024 time-major channels float32, 16 steps, backward: 22 us, in
        // chunks 24; 32 steps 10.4 and 11.0) or where the channels fill the
        // device (time-major float32: 20x1000x4096 forward 293 us, in chunks 306,
        // backward 563 and 655, 16x1200x4096 backward 533 and 616; 10x2000x4096
        // 458 and 296, backward 722 and 646).
        const int64_t groups = (C + kWave - 1) / kWave, chunks = (T + kSpanChunk - 1) / kSpanChunk;
        if (T > 32 && groups < kFull / 2 && groups * chunks < kMostChunks) {
            pl.kernel = kLaneLookBack;
            pl.chunks = chunks;
            if (chunks > 1) record = 3 * sizeof(uint64_t), lines = groups;
        }
    }
    pl.records = align_up(lines * kTicketWords * sizeof(uint32_t));
    pl.part = align_up(pl.records + (size_t)(pl.chunks * C) * record);
    pl.total = adjoint ? align_up(pl.part + (size_t)(pl.chunks * C) * sizeof(float)) : pl.part;
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
    A.ticket = static_cast<uint32_t *>(ws);
    if (pl.part) A.words = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + pl.records);
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

#define PARARNN_GATED(NAME, GRID, BLOCK, ...)                                                    \
    if constexpr (ADJ)                                                                           \
        hipLaunchKernelGGL((gated_##NAME##_adjoint_kernel<__VA_ARGS__>), GRID, BLOCK, 0, st, A); \
    else                                                                                         \
        hipLaunchKernelGGL((gated_##NAME##_kernel<__VA_ARGS__>), GRID, BLOCK, 0, st, A)

template <bool ADJ, bool BF16, bool DOCS>
hipError_t run_gated(const GatedArgs &A, const GatedPlan &pl, hipStream_t st)
{
    constexpr int K = BF16 ? kStepsBf16 : kStepsF32;
    const unsigned groups = (unsigned)((A.channels + kWave - 1) / kWave);
    if (pl.part) {  // tickets and words
        const size_t words = pl.part / sizeof(uint64_t);
        hipLaunchKernelGGL(gated_clear_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0,
                           st, A, (int64_t)words);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    switch (pl.kernel) {
    case kLanePerChannel:
        PARARNN_GATED(channel, dim3(groups), dim3(kWave), BF16, DOCS);
        break;
    case kLaneLookBack:
        PARARNN_GATED(span, dim3((unsigned)(groups * pl.chunks)), dim3(kSpanWaves * kWave), BF16,
                      DOCS);
        break;
    case kWavePerChannel:
        if (A.T <= 16 * K) {  // several channels a wave
            const int lanes = A.T <= 4 * K ? 4 : 16;
            const dim3 grid((unsigned)((A.channels * lanes + kShortThreads - 1) / kShortThreads));
            if (lanes == 4) {
                PARARNN_GATED(short, grid, dim3(kShortThreads), BF16, DOCS, K, 4);
            } else {
                PARARNN_GATED(short, grid, dim3(kShortThreads), BF16, DOCS, K, 16);
            }
        } else {
            PARARNN_GATED(time, dim3((unsigned)A.channels), dim3(kWave), BF16, DOCS, K, 1);
        }
        break;
    case kGroupPerChannel:
        PARARNN_GATED(time, dim3((unsigned)A.channels), dim3(4 * kWave), BF16, DOCS, K, 4);
        break;
    case kLookBack:
        PARARNN_GATED(look, dim3((unsigned)(A.channels * pl.chunks)), dim3(kLookWaves * kWave), BF16,
                      DOCS, kLookSteps, kLookWaves);
        break;
    }
    return hipGetLastError();
}
#undef PARARNN_GATED

template <bool ADJ>
hipError_t run_gated(const GatedArgs &A, const GatedPlan &pl, bool bf16, hipStream_t st)
{
    if (A.resets) return bf16 ? run_gated<ADJ, true, true>(A, pl, st) : run_gated<ADJ, false, true>(A, pl, st);
    return bf16 ? run_gated<ADJ, true, false>(A, pl, st) : run_gated<ADJ, false, false>(A, pl, st);
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
    hipStream_t strm = static_cast<hipStream_t>(stream);
    const hipError_t e = run_gated<false>(A, pl, u_dtype == PARARNN_BF16, strm);
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
    if (pl.channels > 0) {
        if (run_gated<true>(A, pl, u_dtype == PARARNN_BF16, strm) != hipSuccess) return PARARNN_ERR_HIP;
    }
    hipLaunchKernelGGL(gated_dlam_kernel, dim3((unsigned)((shape->D + kWave - 1) / kWave)),
                       dim3(kDlamWaves * kWave), 0, strm, A, shape->B * pl.chunks);
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
