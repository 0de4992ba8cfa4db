// Block boundary: host side of pararnn_block_norm and its adjoint.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "block.hpp"
#include "host.hpp"

using namespace pararnn;

namespace {

constexpr int64_t kBlockGroups = 8 * kComputeUnits;  // workgroups that stay resident

int block_steps(int64_t T) { return T >= 16 ? 16 : T >= 4 ? 4 : 1; }

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

int64_t block_tiles(const pararnn_block_shape_t *sh, int tt)
{
    return sh->B * ((sh->T + tt - 1) / tt);
}

void block_args(BlockArgs &A, const pararnn_block_shape_t *sh, int tt)
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
    A.tiles_per_row = (sh->T + tt - 1) / tt;
    A.tiles = block_tiles(sh, tt);
    A.groups = (int32_t)std::min<int64_t>(A.tiles, kBlockGroups);
}

#define PARARNN_BLOCK_LAUNCH(KERNEL)                                                             \
    switch (tt) {                                                                                \
    case 16: hipLaunchKernelGGL((KERNEL<16>), grid, block, 0, strm, A); break;                   \
    case 4: hipLaunchKernelGGL((KERNEL<4>), grid, block, 0, strm, A); break;                     \
    default: hipLaunchKernelGGL((KERNEL<1>), grid, block, 0, strm, A); break;                    \
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
    const int tt = block_steps(shape->T);
    BlockArgs A;
    block_args(A, shape, tt);
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
    hipStream_t strm = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)A.groups), block(kBlockThreads);
    PARARNN_BLOCK_LAUNCH(block_strip_kernel)
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

size_t pararnn_block_workspace_bytes(const pararnn_block_shape_t *shape)
{
    if (check_block(shape) != PARARNN_OK) return 0;
    const int64_t g = std::min<int64_t>(block_tiles(shape, block_steps(shape->T)), kBlockGroups);
    return align_up((size_t)g * 2 * shape->D * sizeof(float));
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
    const int tt = block_steps(shape->T);
    BlockArgs A;
    block_args(A, shape, tt);
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
    if (work) {
        const dim3 grid((unsigned)A.groups), block(kBlockThreads);
        PARARNN_BLOCK_LAUNCH(block_strip_adjoint_kernel)
        if (hipGetLastError() != hipSuccess) return PARARNN_ERR_HIP;
    }
    const int tpb = 256;
    hipLaunchKernelGGL(block_dw_kernel, dim3((unsigned)((2 * shape->D + tpb - 1) / tpb)), dim3(tpb),
                       0, strm, A);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

}  // extern "C"
