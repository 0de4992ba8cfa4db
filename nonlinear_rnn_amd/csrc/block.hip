// Block boundary: host side of pararnn_block_norm and its adjoint.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <iterator>

#include "block_launch.hpp"
#include "host.hpp"

using namespace pararnn;

namespace {

// Tilings of the register kernels: waves a workgroup, groups of 4 steps,
// channel pairs a lane; they hold waves 64 / groups * 2 pairs channels.
struct Tiling {
    int waves, groups, pairs;
    bool quads;
    int64_t channels() const { return (int64_t)waves * kWave / groups * 2 * pairs; }
};
#define PARARNN_TILING_ENTRY(W, G, P, Q) {W, G, P, Q},
constexpr Tiling kTilings[] = {PARARNN_BLOCK_TILINGS(PARARNN_TILING_ENTRY)};
constexpr Tiling kAdjointTilings[] = {PARARNN_BLOCK_ADJOINT_TILINGS(PARARNN_TILING_ENTRY)};
constexpr int64_t kStripSteps = 4, kStripGroups = 2 * kComputeUnits;

// The tiling that holds D channels with the most steps a tile that still
// makes two tiles a CU, and of those the narrowest; single steps where the
// planes' steps are not contiguous.  No waves: the strip kernels.
// (Two tiles a CU, not one or four: B=2 T=3000 D=1024 28 us, one 34, four 33;
// B=1 T=6000 D=512 15, 19 and 18.)  The backward pass keeps 8 waves a CU, what
// its registers allow.
struct BlockPlan {
    Tiling t = {0, 0, 0, false};
    int64_t tiles_per_row = 0, tiles = 0, groups = 0;  // groups: workgroups that stay (backward)
};
// The tensors that are there; the others' strides say nothing.  (Forward, z
// always is.)
struct BlockParts {
    bool h, gate, z;
};
BlockPlan block_plan(const pararnn_block_shape_t *sh, bool adjoint, BlockParts in)
{
    BlockPlan pl;
    const bool quads =
        (!in.h || sh->h_stride_t == 1) && (!in.gate || sh->g_stride_t == 1) && sh->T >= 4;
    // a lane's offset from the tile's base is 32 bits of bytes
    const int64_t reach = (int64_t(1) << 29) - 8;
    const bool near = sh->D >= 2 && (!in.h || sh->h_stride_d <= reach / sh->D) &&
                      (!in.gate || sh->g_stride_d <= reach / sh->D) &&
                      sh->x_stride_t <= reach / 16 && (!in.z || sh->z_stride_t <= reach / 16);
    const Tiling *list = adjoint ? kAdjointTilings : kTilings;
    const size_t count = adjoint ? std::size(kAdjointTilings) : std::size(kTilings);
    for (size_t i = 0; i < count; ++i) {
        const Tiling &t = list[i];
        const int64_t steps = 4 * t.groups;
        if (!near || t.channels() < sh->D || t.quads != quads) continue;
        if (t.groups > 1 && (sh->T < steps || sh->B * (sh->T / steps) < 2 * kComputeUnits)) continue;
        if (!pl.t.waves || t.groups > pl.t.groups ||
            (t.groups == pl.t.groups && t.channels() < pl.t.channels()))
            pl.t = t;
    }
    const auto cut = [&](int64_t steps) {
        pl.tiles_per_row = (sh->T + steps - 1) / steps;
        pl.tiles = sh->B * pl.tiles_per_row;
    };
    // the register kernels number their tiles, and forward a dispatch its
    // work-items, in 32 bits; the strip kernels' workgroups go on to the next tile
    constexpr int64_t k32 = int64_t(1) << 32;
    cut(pl.t.waves ? 4 * pl.t.groups : kStripSteps);
    if (pl.t.waves && (adjoint ? pl.tiles : (pl.tiles + 7) / 8 * 8 * pl.t.waves * kWave) >= k32) {
        pl.t = {0, 0, 0, false};
        cut(kStripSteps);
    }
    // resident workgroups, 8 waves a CU; a multiple of the 8 XCDs
    const int64_t fit = pl.t.waves ? 8 / std::min(8, pl.t.waves) * kComputeUnits : kStripGroups;
    // and as few as take the same number of tiles each
    const int64_t rounds = (pl.tiles + fit - 1) / fit;
    if (rounds > 0) pl.groups = std::min(((pl.tiles + rounds - 1) / rounds + 7) / 8 * 8, fit);
    return pl;
}

// Rows of D contiguous channels, (b, t) apart by the two strides.
bool rows_disjoint(int64_t B, int64_t T, int64_t D, int64_t sb, int64_t st)
{
    return planes_disjoint(B, T, D, sb, 1, st);
}

pararnn_status_t check_block(const pararnn_block_shape_t *sh)
{
    if (!sh) return PARARNN_ERR_INVALID;
    if (sh->B < 0 || sh->T < 0 || sh->D < 0) return PARARNN_ERR_INVALID;
    if (sh->B > (int64_t(1) << 31) || sh->D > (int64_t(1) << 24) || sh->T > (int64_t(1) << 31))
        return PARARNN_ERR_UNSUPPORTED;
    if (!planes_disjoint(sh->B, sh->T, sh->D, sh->h_stride_b, sh->h_stride_d, sh->h_stride_t) ||
        !planes_disjoint(sh->B, sh->T, sh->D, sh->g_stride_b, sh->g_stride_d, sh->g_stride_t) ||
        !rows_disjoint(sh->B, sh->T, sh->D, sh->x_stride_b, sh->x_stride_t) ||
        !rows_disjoint(sh->B, sh->T, sh->D, sh->z_stride_b, sh->z_stride_t))
        return PARARNN_ERR_INVALID;
    return PARARNN_OK;
}

bool known(pararnn_dtype_t d) { return d == PARARNN_F32 || d == PARARNN_BF16; }

void block_args(BlockArgs &A, const pararnn_block_shape_t *sh, const BlockPlan &pl)
{
    std::memset(&A, 0, sizeof(A));
    A.B = sh->B;
    A.T = sh->T;
    A.D = sh->D;
    A.hsb = sh->h_stride_b;
    A.hsd = sh->h_stride_d;
    A.hst = sh->h_stride_t;
    A.gsb = sh->g_stride_b;
    A.gsd = sh->g_stride_d;
    A.gst = sh->g_stride_t;
    A.xsb = sh->x_stride_b;
    A.xst = sh->x_stride_t;
    A.zsb = sh->z_stride_b;
    A.zst = sh->z_stride_t;
    A.tiles_per_row = pl.tiles_per_row;
    A.tiles = pl.tiles;
    A.groups = (int32_t)pl.groups;
}

// For the register kernels: a tensor that is not given is read from one that
// is (and dropped), so that their loads need no condition.
void stand_ins(BlockArgs &A, bool adjoint)
{
    A.has_gate = A.gate != nullptr;
    A.has_gy = A.gy != nullptr;
    A.has_gz = A.gz != nullptr;
    if (A.h && !A.gate) {
        A.gate = A.h;
        A.gate_bf16 = 0;
        A.gsb = A.hsb, A.gsd = A.hsd, A.gst = A.hst;
    }
    if (!adjoint) return;
    if (!A.gy) A.gy = A.x;
    if (!A.gz) {
        A.gz = A.x;
        A.z_bf16 = A.x_bf16;
        A.zsb = A.xsb, A.zst = A.xst;
    }
}

template <bool ADJ>
hipError_t launch_block(BlockArgs A, const BlockPlan &pl, hipStream_t st)
{
    const dim3 grid((unsigned)(ADJ ? pl.groups : (pl.tiles + 7) / 8 * 8)),
        block((unsigned)(pl.t.waves * kWave));
    if (!pl.t.waves) {
        const dim3 few((unsigned)pl.groups), strip(kBlockThreads);
        if constexpr (ADJ)
            hipLaunchKernelGGL((block_strip_adjoint_kernel<kStripSteps>), few, strip, 0, st, A);
        else
            hipLaunchKernelGGL((block_strip_kernel<kStripSteps>), few, strip, 0, st, A);
        return hipGetLastError();
    }
    stand_ins(A, ADJ);
    const int types = A.gate_bf16 * kGateBf16 | A.x_bf16 * kStreamBf16 | A.z_bf16 * kNormedBf16;
    const int tiling = tiling_code(pl.t.waves, pl.t.groups, pl.t.pairs, pl.t.quads);
    if (!A.h) return launch_block_norm(ADJ, tiling, grid, block, st, A);
    switch (types) {
    case kNormedBf16: return launch_block_f32(ADJ, tiling, grid, block, st, A);
    case kNormedBf16 | kGateBf16: return launch_block_gate(ADJ, tiling, grid, block, st, A);
    case kNormedBf16 | kStreamBf16: return launch_block_stream(ADJ, tiling, grid, block, st, A);
    case kNormedBf16 | kGateBf16 | kStreamBf16:
        return launch_block_bf16(ADJ, tiling, grid, block, st, A);
    default: return launch_block_args(ADJ, tiling, grid, block, st, A);
    }
}

}  // namespace

extern "C" {

pararnn_status_t pararnn_block_norm(const pararnn_block_shape_t *shape, const float *h,
                                    const void *gate, pararnn_dtype_t gate_dtype, const void *x,
                                    pararnn_dtype_t x_dtype, const float *w_post,
                                    const float *w_pre, float scale, float eps, void *y, void *z,
                                    pararnn_dtype_t z_dtype, float *rstd, void *stream)
{
    const pararnn_status_t st = check_block(shape);
    if (st != PARARNN_OK) return st;
    if (!known(x_dtype) || !known(z_dtype) || (gate && !known(gate_dtype)))
        return PARARNN_ERR_UNSUPPORTED;
    if (!std::isfinite(scale) || !(eps > 0.0f) || std::isinf(eps)) return PARARNN_ERR_INVALID;
    if (shape->B == 0 || shape->T == 0 || shape->D == 0) return PARARNN_OK;
    if (!x || !w_pre || !z || (h && (!w_post || !y)) || (!h && gate)) return PARARNN_ERR_INVALID;
    const BlockPlan pl = block_plan(shape, false, {h != nullptr, gate != nullptr, true});
    BlockArgs A;
    block_args(A, shape, pl);
    A.h = h;
    A.gate = gate;
    A.x = x;
    A.w_post = w_post;
    A.w_pre = w_pre;
    A.scale = scale;
    A.eps = eps;
    A.y = y;
    A.z = z;
    A.rstd = rstd;
    A.gate_bf16 = gate_dtype == PARARNN_BF16;
    A.x_bf16 = x_dtype == PARARNN_BF16;
    A.z_bf16 = z_dtype == PARARNN_BF16;
    const hipError_t e = launch_block<false>(A, pl, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

size_t pararnn_block_workspace_bytes(const pararnn_block_shape_t *shape)
{
    if (check_block(shape) != PARARNN_OK) return 0;
    int64_t groups = 0;  // enough for any of the tensors left out
    for (const bool z : {false, true})
        for (const BlockParts in : {BlockParts{false, false, z}, {true, false, z}, {true, true, z}})
            groups = std::max(groups, block_plan(shape, true, in).groups);
    return align_up((size_t)groups * 2 * shape->D * sizeof(float));
}

pararnn_status_t pararnn_block_norm_adjoint(const pararnn_block_shape_t *shape, const float *h,
                                            const void *gate, pararnn_dtype_t gate_dtype,
                                            const void *x, pararnn_dtype_t x_dtype,
                                            const float *w_post, const float *w_pre, float scale,
                                            const float *rstd, const void *gy, const void *gz,
                                            pararnn_dtype_t z_dtype, float *dh, void *dgate,
                                            void *dx, float *dw_post, float *dw_pre, void *ws,
                                            size_t ws_bytes, void *stream)
{
    const pararnn_status_t st = check_block(shape);
    if (st != PARARNN_OK) return st;
    if (!known(x_dtype) || !known(z_dtype) || (gate && !known(gate_dtype)))
        return PARARNN_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return PARARNN_ERR_INVALID;
    if (shape->D == 0) return PARARNN_OK;
    if (!dw_pre || (h && !dw_post) || (!h && gate)) return PARARNN_ERR_INVALID;
    const bool work = shape->B > 0 && shape->T > 0;
    if (work && (!x || !w_pre || !rstd || !dx || (h && (!w_post || !dh)) || (gate && !dgate)))
        return PARARNN_ERR_INVALID;
    const size_t need = pararnn_block_workspace_bytes(shape);
    if (work && (!ws || ws_bytes < need || !aligned16(ws))) return PARARNN_ERR_WORKSPACE;
    const BlockPlan pl = block_plan(shape, true, {h != nullptr, gate != nullptr, gz != nullptr});
    BlockArgs A;
    block_args(A, shape, pl);
    A.h = h;
    A.gate = gate;
    A.x = x;
    A.w_post = w_post;
    A.w_pre = w_pre;
    A.scale = scale;
    A.rstd_in = rstd;
    A.gy = gy;
    A.gz = gz;
    A.dh = dh;
    A.dgate = dgate;
    A.dx = dx;
    A.dw_post = dw_post;  // zero-sized planes have no address, their weights' gradient is zero
    A.dw_pre = dw_pre;
    A.part = static_cast<float *>(ws);
    A.gate_bf16 = gate_dtype == PARARNN_BF16;
    A.x_bf16 = x_dtype == PARARNN_BF16;
    A.z_bf16 = z_dtype == PARARNN_BF16;
    hipStream_t strm = static_cast<hipStream_t>(stream);
    if (work && launch_block<true>(A, pl, strm) != hipSuccess) return PARARNN_ERR_HIP;
    hipLaunchKernelGGL(block_dw_kernel, dim3((unsigned)((2 * shape->D + kWave - 1) / kWave)),
                       dim3(kDwWaves * kWave), 0, strm, A);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

}  // extern "C"
