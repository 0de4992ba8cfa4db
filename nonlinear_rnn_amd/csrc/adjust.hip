// Logits before sampling: host side of pararnn_adjust_logits.
#include <hip/hip_runtime.h>

#include <cstring>

#include "adjust.hpp"
#include "host.hpp"

using namespace pararnn;
using namespace pararnn::adjust;

extern "C" {

pararnn_status_t pararnn_adjust_logits(int64_t N, int64_t V, const void *logits, pararnn_dtype_t dtype,
                                       int64_t row_stride, const pararnn_adjust_t *how, void *out, int64_t out_stride,
                                       void *stream)
{
    const int64_t most = int64_t(1) << 31;
    if (N < 0 || V < 0 || !how || how->length < 0 || how->biases < 0 || how->allowed_count < 0)
        return PARARNN_ERR_INVALID;
    if (dtype != PARARNN_F32 && dtype != PARARNN_BF16) return PARARNN_ERR_UNSUPPORTED;
    if (N >= (int64_t(1) << 24) || V >= most || how->length >= most || how->biases >= most || how->allowed_count >= most)
        return PARARNN_ERR_UNSUPPORTED;
    for (const int64_t stride : {row_stride, out_stride}) {
        if (stride < 0 || (N > 1 && stride < V)) return PARARNN_ERR_INVALID;
        if (N > 0 && stride > INT64_MAX / 4 / N) return PARARNN_ERR_INVALID;
    }
    if (how->token_stride < 0 || (N > 0 && how->token_stride > INT64_MAX / 8 / N)) return PARARNN_ERR_INVALID;
    const bool history = how->length > 0;
    if (history && !how->tokens) return PARARNN_ERR_INVALID;
    if (how->biases > 0 && (!how->bias_index || !how->bias_value)) return PARARNN_ERR_INVALID;
    if (how->allowed) {
        const int64_t words = (V + 31) / 32;
        if (how->allowed_stride < words || how->allowed_stride >= most) return PARARNN_ERR_INVALID;
        if (!how->allowed_rows && how->allowed_count < N) return PARARNN_ERR_INVALID;
    }
    if (N == 0 || V == 0) return PARARNN_OK;
    if (!logits || !out || (logits == out && row_stride != out_stride)) return PARARNN_ERR_INVALID;
    Args A;
    std::memset(&A, 0, sizeof(A));
    A.x = logits, A.out = out, A.N = N, A.V = V, A.stride = row_stride, A.out_stride = out_stride;
    if (history) {
        A.tokens = how->tokens, A.token_stride = how->token_stride, A.length = how->length;
        A.lengths = how->lengths, A.prompt = how->prompt;
        A.repetition = how->repetition, A.presence = how->presence, A.frequency = how->frequency;
    }
    A.bias_index = how->bias_index, A.bias_value = how->bias_value, A.biases = how->biases;
    A.allowed = reinterpret_cast<const uint32_t *>(how->allowed), A.allowed_stride = how->allowed_stride;
    A.allowed_count = how->allowed_count, A.allowed_rows = how->allowed_rows;
    // a row's vectors, one more where it starts off their alignment
    const int64_t k = dtype == PARARNN_BF16 ? 8 : 4, per = kTokens / k;
    A.parts = (int32_t)(((V + k - 1) / k + 1 + per - 1) / per);
    if (N * A.parts >= (int64_t(1) << 24)) return PARARNN_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)(N * A.parts)), block(kThreads);
    const size_t lds = A.biases > 0 ? kTokens * sizeof(uint32_t) : 0;
    hipStream_t strm = static_cast<hipStream_t>(stream);
    if (dtype == PARARNN_BF16)
        hipLaunchKernelGGL((adjust_kernel<true>), grid, block, lds, strm, A);
    else
        hipLaunchKernelGGL((adjust_kernel<false>), grid, block, lds, strm, A);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

}  // extern "C"
