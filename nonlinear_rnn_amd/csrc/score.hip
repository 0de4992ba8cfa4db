// Token scores: host side of pararnn_token_logprobs and its adjoint.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "host.hpp"
#include "score.hpp"

using namespace pararnn;

namespace {

pararnn_status_t check_score(int64_t N, int64_t V, pararnn_dtype_t dtype, int64_t stride,
                             float scale)
{
    if (N < 0 || V < 0) return PARARNN_ERR_INVALID;
    if (N >= (int64_t(1) << 31) || V >= (int64_t(1) << 31)) return PARARNN_ERR_UNSUPPORTED;
    if (dtype != PARARNN_F32 && dtype != PARARNN_BF16) return PARARNN_ERR_UNSUPPORTED;
    if (!(scale > 0.0f) || std::isinf(scale)) return PARARNN_ERR_INVALID;
    if (stride < 0 || (N > 1 && stride < V)) return PARARNN_ERR_INVALID;
    if (N > 0 && stride > INT64_MAX / N) return PARARNN_ERR_INVALID;
    return PARARNN_OK;
}

}  // namespace

extern "C" {

size_t pararnn_logprobs_workspace_bytes(int64_t N, int64_t V, int32_t top)
{
    (void)N, (void)V, (void)top;
    return 0;
}

pararnn_status_t pararnn_token_logprobs(int64_t N, int64_t V, const void *logits,
                                        pararnn_dtype_t dtype, int64_t row_stride,
                                        const int64_t *tokens, int32_t top, float scale,
                                        float *logprob, float *entropy, float *lse,
                                        int64_t *top_index, float *top_logprob, void *ws,
                                        size_t ws_bytes, void *stream)
{
    const pararnn_status_t st = check_score(N, V, dtype, row_stride, scale);
    if (st != PARARNN_OK) return st;
    if (top < 0) return PARARNN_ERR_INVALID;
    if (top > PARARNN_TOP_MAX) return PARARNN_ERR_UNSUPPORTED;
    if (N == 0) return PARARNN_OK;
    if ((V > 0 && !logits) || !tokens || !logprob || (top > 0 && (!top_index || !top_logprob)))
        return PARARNN_ERR_INVALID;
    const size_t need = pararnn_logprobs_workspace_bytes(N, V, top);
    if (need > 0 && (!ws || ws_bytes < need || !aligned16(ws))) return PARARNN_ERR_WORKSPACE;
    ScoreArgs A;
    std::memset(&A, 0, sizeof(A));
    A.x = logits;
    A.tokens = tokens;
    A.logprob = logprob;
    A.entropy = entropy;
    A.lse = lse;
    A.top_index = top_index;
    A.top_logprob = top_logprob;
    A.N = N;
    A.V = V;
    A.stride = row_stride;
    A.top = top;
    A.scale = scale;
    hipStream_t strm = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)std::min<int64_t>(N, 1 << 20)), block(kScoreThreads);
    if (dtype == PARARNN_BF16)
        hipLaunchKernelGGL((score_row_kernel<true>), grid, block, 0, strm, A);
    else
        hipLaunchKernelGGL((score_row_kernel<false>), grid, block, 0, strm, A);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

pararnn_status_t pararnn_token_logprobs_adjoint(int64_t N, int64_t V, const void *logits,
                                                pararnn_dtype_t dtype, int64_t row_stride,
                                                const int64_t *tokens, float scale,
                                                const float *lse, const float *entropy,
                                                const float *g_logprob, const float *g_entropy,
                                                const float *g_lse, void *dlogits,
                                                int64_t d_stride, void *stream)
{
    pararnn_status_t st = check_score(N, V, dtype, row_stride, scale);
    if (st == PARARNN_OK) st = check_score(N, V, dtype, d_stride, scale);
    if (st != PARARNN_OK) return st;
    if (logits == dlogits && row_stride != d_stride) return PARARNN_ERR_INVALID;
    if (N == 0 || V == 0) return PARARNN_OK;
    if (!logits || !tokens || !lse || !dlogits || (g_entropy && !entropy))
        return PARARNN_ERR_INVALID;
    ScoreArgs A;
    std::memset(&A, 0, sizeof(A));
    A.x = logits;
    A.tokens = tokens;
    A.N = N;
    A.V = V;
    A.stride = row_stride;
    A.scale = scale;
    A.lse_in = lse;
    A.entropy_in = entropy;
    A.g_logprob = g_logprob;
    A.g_entropy = g_entropy;
    A.g_lse = g_lse;
    A.dx = dlogits;
    A.dstride = d_stride;
    hipStream_t strm = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)std::min<int64_t>(N, 1 << 20)), block(kScoreThreads);
    if (dtype == PARARNN_BF16)
        hipLaunchKernelGGL((score_adjoint_kernel<true>), grid, block, 0, strm, A);
    else
        hipLaunchKernelGGL((score_adjoint_kernel<false>), grid, block, 0, strm, A);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

}  // extern "C"
