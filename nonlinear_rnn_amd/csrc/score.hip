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
    // a dispatch counts its work-items in 32 bits: 256 a row
    if (N >= (int64_t(1) << 24) || V >= (int64_t(1) << 31)) return PARARNN_ERR_UNSUPPORTED;
    if (dtype != PARARNN_F32 && dtype != PARARNN_BF16) return PARARNN_ERR_UNSUPPORTED;
    if (!(scale > 0.0f) || std::isinf(scale)) return PARARNN_ERR_INVALID;
    if (stride < 0 || (N > 1 && stride < V)) return PARARNN_ERR_INVALID;
    if (N > 0 && stride > INT64_MAX / N) return PARARNN_ERR_INVALID;
    return PARARNN_OK;
}

// Workgroups a row: one, unless there are too few rows to fill the device (4
// workgroups a CU); then parts of at least 4096 logits (2048 and 16384 take the
// same time within 1 us for 16 rows of 65536 and 512 of 50003).
int64_t score_parts(int64_t N, int64_t V)
{
    if (N <= 0) return 1;
    const int64_t want = std::min((4 * kComputeUnits + N - 1) / N, (V + 4095) / 4096);
    return std::max<int64_t>(1, std::min<int64_t>(want, kScoreParts));
}

size_t score_stats_bytes(int64_t N, int64_t parts)
{
    return align_up((size_t)N * parts * sizeof(float4));
}

template <bool BF16, bool TOP>
hipError_t run_score(const ScoreArgs &A, hipStream_t st)
{
    const dim3 grid((unsigned)(A.N * A.parts)), wide(kScoreThreads), one(kWave);
    if (A.parts > 1) {
        hipLaunchKernelGGL((score_kernel<BF16, kScoreWaves, true, TOP>), grid, wide, 0, st, A);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((score_join_kernel<BF16>), dim3((unsigned)A.N), dim3(kJoinThreads), 0, st,
                           A);
    } else if (A.V <= 8192) {
        // up to a few dozen vectors a lane: no barriers between waves, no lists
        // to join (8192 rows with 8 alternatives, float32: 2000 logits 24 us,
        // with 4 waves 37; 8000 65 and 75; 4096 rows of 16000 64 and 67)
        hipLaunchKernelGGL((score_kernel<BF16, 1, false, TOP>), grid, one, 0, st, A);
    } else {
        hipLaunchKernelGGL((score_kernel<BF16, kScoreWaves, false, TOP>), grid, wide, 0, st, A);
    }
    return hipGetLastError();
}
template <bool BF16>
hipError_t run_score(const ScoreArgs &A, hipStream_t st)
{
    return A.top ? run_score<BF16, true>(A, st) : run_score<BF16, false>(A, st);
}

}  // namespace

extern "C" {

size_t pararnn_logprobs_workspace_bytes(int64_t N, int64_t V, int32_t top)
{
    if (N <= 0 || V <= 0 || top < 0 || top > PARARNN_TOP_MAX || N >= (int64_t(1) << 24) ||
        V >= (int64_t(1) << 31))
        return 0;
    const int64_t parts = score_parts(N, V);
    if (parts == 1) return 0;
    return score_stats_bytes(N, parts) + (size_t)N * parts * top * sizeof(uint64_t);
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
    A.parts = (int32_t)score_parts(N, V);
    if (need > 0) {
        A.part_stats = static_cast<float4 *>(ws);
        A.part_keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) +
                                                   score_stats_bytes(N, A.parts));
    }
    hipStream_t strm = static_cast<hipStream_t>(stream);
    const hipError_t e = dtype == PARARNN_BF16 ? run_score<true>(A, strm) : run_score<false>(A, strm);
    return e == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
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
    // a row's vectors, one more where it starts off their alignment
    const int64_t k = dtype == PARARNN_BF16 ? 8 : 4, per = kScoreUnroll * kScoreThreads;
    A.parts = (int32_t)(((V + k - 1) / k + 1 + per - 1) / per);
    if (N * A.parts >= (int64_t(1) << 24)) return PARARNN_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)(N * A.parts)), block(kScoreThreads);
    if (dtype == PARARNN_BF16)
        hipLaunchKernelGGL((score_adjoint_kernel<true>), grid, block, 0, strm, A);
    else
        hipLaunchKernelGGL((score_adjoint_kernel<false>), grid, block, 0, strm, A);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

}  // extern "C"
