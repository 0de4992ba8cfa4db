// Distillation from top tokens: host side of pararnn_distill_top and its adjoint.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "distill.hpp"
#include "host.hpp"

using namespace pararnn;
using namespace pararnn::distill;

namespace {

pararnn_status_t check_distill(int64_t N, int64_t V, pararnn_dtype_t dtype, int64_t stride, int32_t count, float scale)
{
    if (N < 0 || V < 0 || count < 0) return PARARNN_ERR_INVALID;
    // a dispatch counts its work-items in 32 bits: 256 a row
    if (N >= (int64_t(1) << 24) || V >= (int64_t(1) << 31) || count > kMost) return PARARNN_ERR_UNSUPPORTED;
    if (dtype != PARARNN_F32 && dtype != PARARNN_BF16) return PARARNN_ERR_UNSUPPORTED;
    if (!(scale > 0.0f) || std::isinf(scale)) return PARARNN_ERR_INVALID;
    if (stride < 0 || (N > 1 && stride < V)) return PARARNN_ERR_INVALID;
    if (N > 0 && stride > INT64_MAX / N) return PARARNN_ERR_INVALID;
    return PARARNN_OK;
}

// Workgroups a row, by the rule of the token scores: one, unless there are too
// few rows to fill the device; then parts of at least 4096 logits.
int64_t parts_of(int64_t N, int64_t V)
{
    if (N <= 0) return 1;
    const int64_t want = std::min((4 * kComputeUnits + N - 1) / N, (V + 4095) / 4096);
    return std::max<int64_t>(1, std::min<int64_t>(want, kParts));
}

template <bool BF16>
pararnn_status_t run(const Args &A, hipStream_t s)
{
    const dim3 grid((unsigned)(A.N * A.parts)), block(kThreads);
    if (A.parts > 1) {
        hipLaunchKernelGGL((distill_kernel<BF16, true>), grid, block, 0, s, A);
        if (hipGetLastError() != hipSuccess) return PARARNN_ERR_HIP;
        hipLaunchKernelGGL((distill_join_kernel<BF16>), dim3((unsigned)A.N), block, 0, s, A);
    } else {
        hipLaunchKernelGGL((distill_kernel<BF16, false>), grid, block, 0, s, A);
    }
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

}  // namespace

extern "C" {

size_t pararnn_distill_workspace_bytes(int64_t N, int64_t V)
{
    if (N <= 0 || V <= 0 || N >= (int64_t(1) << 24) || V >= (int64_t(1) << 31)) return 0;
    const int64_t parts = parts_of(N, V);
    return parts == 1 ? 0 : align_up((size_t)N * parts * sizeof(float2));
}

pararnn_status_t pararnn_distill_top(int64_t N, int64_t V, const void *logits, pararnn_dtype_t dtype,
                                     int64_t row_stride, const int64_t *top_index, const float *top_logprob,
                                     int32_t top, int tail, float scale, float *loss, float *lse, float *log_rest,
                                     void *ws, size_t ws_bytes, void *stream)
{
    const pararnn_status_t st = check_distill(N, V, dtype, row_stride, top, scale);
    if (st != PARARNN_OK) return st;
    if (N == 0) return PARARNN_OK;
    if ((V > 0 && !logits) || (top > 0 && (!top_index || !top_logprob)) || !loss || !lse || !log_rest)
        return PARARNN_ERR_INVALID;
    const size_t need = pararnn_distill_workspace_bytes(N, V);
    if (need > 0 && (!ws || ws_bytes < need || !aligned16(ws))) return PARARNN_ERR_WORKSPACE;
    Args A;
    std::memset(&A, 0, sizeof(A));
    A.x = logits, A.index = top_index, A.logprob = top_logprob;
    A.N = N, A.V = V, A.stride = row_stride, A.count = top, A.tail = tail != 0, A.scale = scale;
    A.parts = (int32_t)parts_of(N, V);
    A.loss = loss, A.lse = lse, A.log_rest = log_rest;
    A.part_stats = static_cast<float2 *>(ws);
    hipStream_t strm = static_cast<hipStream_t>(stream);
    return dtype == PARARNN_BF16 ? run<true>(A, strm) : run<false>(A, strm);
}

pararnn_status_t pararnn_distill_top_adjoint(int64_t N, int64_t V, const void *logits, pararnn_dtype_t dtype,
                                             int64_t row_stride, const int64_t *top_index, const float *top_logprob,
                                             int32_t top, int tail, float scale, const float *lse,
                                             const float *log_rest, const float *g_loss, void *dlogits,
                                             int64_t d_stride, void *stream)
{
    pararnn_status_t st = check_distill(N, V, dtype, row_stride, top, scale);
    if (st == PARARNN_OK) st = check_distill(N, V, dtype, d_stride, top, scale);
    if (st != PARARNN_OK) return st;
    if (N == 0 || V == 0) return PARARNN_OK;
    if (logits == dlogits && row_stride != d_stride) return PARARNN_ERR_INVALID;
    if (!logits || (top > 0 && (!top_index || !top_logprob)) || !lse || !log_rest || !g_loss || !dlogits)
        return PARARNN_ERR_INVALID;
    Args A;
    std::memset(&A, 0, sizeof(A));
    A.x = logits, A.index = top_index, A.logprob = top_logprob;
    A.N = N, A.V = V, A.stride = row_stride, A.count = top, A.tail = tail != 0, A.scale = scale;
    A.lse_in = lse, A.log_rest_in = log_rest, A.g_loss = g_loss;
    A.dx = dlogits, A.dstride = d_stride;
    // a row's vectors, one more where it starts off their alignment
    const int64_t k = dtype == PARARNN_BF16 ? 8 : 4, per = kScoreUnroll * kThreads;
    A.parts = (int32_t)(((V + k - 1) / k + 1 + per - 1) / per);
    if (N * A.parts >= (int64_t(1) << 24)) return PARARNN_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)(N * A.parts)), block(kThreads);
    hipStream_t strm = static_cast<hipStream_t>(stream);
    if (dtype == PARARNN_BF16)
        hipLaunchKernelGGL((distill_adjoint_kernel<true>), grid, block, 0, strm, A);
    else
        hipLaunchKernelGGL((distill_adjoint_kernel<false>), grid, block, 0, strm, A);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

}  // extern "C"
