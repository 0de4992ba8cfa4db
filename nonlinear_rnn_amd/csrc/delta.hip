// Gated delta rule: host side of pararnn_delta_scan, its adjoint and its step.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "delta.hpp"
#include "delta_launch.hpp"
#include "host.hpp"

using namespace pararnn;
using namespace pararnn::delta;

namespace {

// Whether an index of these sizes and strides stays in 63 bits, its strides
// not negative; `apart`: and no two elements meet.
template <int N>
bool fits(const int64_t (&size)[N], const int64_t *stride, bool apart)
{
    int order[N];
    for (int i = 0; i < N; ++i) {
        if (stride[i] < 0) return false;
        order[i] = i;
        if (size[i] == 0) apart = false;
    }
    std::sort(order, order + N, [&](int a, int b) { return stride[a] < stride[b]; });
    __int128 reach = 0;  // the largest offset of the dimensions so far
    for (int i : order) {
        if (size[i] <= 1) continue;
        if (apart && (__int128)stride[i] <= reach) return false;
        reach += (__int128)stride[i] * (size[i] - 1);
        if (reach > (__int128)INT64_MAX / 4) return false;
    }
    return true;
}

int64_t chunk_of(pararnn_dtype_t dtype) { return dtype == PARARNN_BF16 ? Bf::kChunk : Fl::kChunk; }
int room_of(int64_t dk) { return dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }

// writes_o: the plane at o_stride is written, not the gradient that is read there.
pararnn_status_t check_delta(const pararnn_delta_shape_t *s, pararnn_dtype_t dtype, bool step, bool writes_o)
{
    if (!s) return PARARNN_ERR_INVALID;
    if (s->B < 0 || s->T < 0 || s->Hk < 0 || s->Hv < 0 || s->dk < 1 || s->dv < 1) return PARARNN_ERR_INVALID;
    if (s->Hk > 0 ? s->Hv < 1 || s->Hv % s->Hk : s->Hv > 0) return PARARNN_ERR_INVALID;
    if (step && s->T != 1) return PARARNN_ERR_INVALID;
    if (dtype != PARARNN_F32 && dtype != PARARNN_BF16) return PARARNN_ERR_UNSUPPORTED;
    if (s->dk > PARARNN_DELTA_KEY_MAX || s->dv > (1 << 20) || s->Hv > (1 << 20) || s->B > (int64_t(1) << 31) ||
        s->T > (int64_t(1) << 40))
        return PARARNN_ERR_UNSUPPORTED;
    const int64_t key[4] = {s->B, s->Hk, s->dk, s->T}, value[4] = {s->B, s->Hv, s->dv, s->T};
    const int64_t gate[3] = {s->B, s->Hv, s->T};
    if (!fits(key, s->q_stride, false) || !fits(key, s->k_stride, false) || !fits(value, s->v_stride, false) ||
        !fits(value, s->o_stride, writes_o) || !fits(gate, s->gate_stride, false))
        return PARARNN_ERR_INVALID;
    // a dispatch counts its work-items in 32 bits
    const int64_t most = int64_t(1) << 32, heads = s->B * s->Hv;
    if (step) {
        if (heads > most / kStepThreads - 1 ||
            heads * ((s->dv + kStepColumns - 1) / kStepColumns) > most / kStepThreads - 1)
            return PARARNN_ERR_UNSUPPORTED;
        return PARARNN_OK;
    }
    const int64_t chunks = (s->T + chunk_of(dtype) - 1) / chunk_of(dtype), blocks = (s->dv + 31) / 32 * 2;
    if (heads > most / kThreads - 1 || (heads > 0 && (blocks > most / kThreads / heads - 1 ||
                                                      chunks > most / kThreads / heads - 1)))
        return PARARNN_ERR_UNSUPPORTED;
    return PARARNN_OK;
}

// Wide workgroups where the chains are many (see kWide).
bool wide_chains(const pararnn_delta_shape_t *s)
{
    return room_of(s->dk) < 256 && s->dv > kNarrow && s->B * s->Hv * ((s->dv + kWide - 1) / kWide) >= kComputeUnits;
}
// Segments of a chain.  Two passes and a way along the segments instead of one way
// along the chunks: as many as fill the device twice, while a segment has 8 chunks,
// and so that the two ways are about as long.  4 heads of 64 x 64 float32, 65536
// steps: 437 us, in one way 7092.  18 heads of 80 x 100, 1531 steps, near the least
// that goes in segments: states 200 us instead of 218, their gradients 235 instead
// of 391.
int64_t segments_of(const pararnn_delta_shape_t *s, int64_t chunks)
{
    const int64_t chains = s->B * s->Hv * ((s->dv + kNarrow - 1) / kNarrow);
    if (chains == 0 || chunks < 32) return 1;
    const int64_t most = std::min<int64_t>({2 * kComputeUnits / chains, chunks / 8, (int64_t)std::sqrt(2.0 * chunks)});
    return most < 4 ? 1 : most;
}

struct Layout {
    size_t inverse, inverse_t, states, dstates, w, x, maps, marks, cuts, total;
    int64_t per, segments;  // chunks a segment
};
Layout layout(const pararnn_delta_shape_t *s, pararnn_dtype_t dtype, bool adjoint)
{
    const size_t C = (size_t)chunk_of(dtype), items = (size_t)(s->B * s->Hv) * ((s->T + C - 1) / C);
    const size_t pad = (size_t)(s->dv + 31) / 32 * 32, room = (size_t)room_of(s->dk);
    Layout l;
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t first = at;
        at += align_up(bytes);
        return first;
    };
    std::memset(&l, 0, sizeof(l));
    const size_t slots = C == 64 ? Slots<64>::kCount : Slots<32>::kCount;
    l.inverse = take(items * slots * sizeof(Fragment));
    if (adjoint) {
        l.inverse_t = take(items * slots * sizeof(Fragment));
        l.states = take(items * room * pad * 4);
        l.dstates = take(items * room * pad * 4);
        l.w = take(items * C * pad * 4);
        l.x = take(items * C * pad * 4);
    }
    const int64_t chunks = (s->T + C - 1) / C, want = segments_of(s, chunks);
    l.per = std::max<int64_t>(1, (chunks + want - 1) / want);
    l.segments = std::max<int64_t>(1, (chunks + l.per - 1) / l.per);
    if (l.segments > 1) {
        const size_t chains = (size_t)(s->B * s->Hv * l.segments), key_pad = (size_t)(s->dk + 15) / 16 * 16;
        l.maps = take(chains * room * (pad + key_pad) * 4);
        l.marks = take(chains * room * pad * 4);
        l.cuts = take(chains * 4);
    }
    l.total = at;
    return l;
}

Plane plane(const void *p, const int64_t *stride)
{
    return {const_cast<void *>(p), stride[0], stride[1], stride[2], stride[3]};
}

// The arguments that both directions share.
pararnn_status_t prepare(Args &A, const pararnn_delta_shape_t *s, pararnn_dtype_t dtype, const void *q, const void *k,
                         const void *v, const float *beta, const float *log_decay, const float *h0,
                         const uint8_t *resets, float scale, bool adjoint, void *ws, size_t ws_bytes)
{
    const pararnn_status_t st = check_delta(s, dtype, false, !adjoint);
    if (st != PARARNN_OK) return st;
    if (!std::isfinite(scale)) return PARARNN_ERR_INVALID;
    if (s->B > 0 && s->Hv > 0 && s->T > 0 && (!q || !k || !v || !beta)) return PARARNN_ERR_INVALID;
    const Layout l = layout(s, dtype, adjoint);
    if (l.total > 0 && (!ws || ws_bytes < l.total || !aligned16(ws))) return PARARNN_ERR_WORKSPACE;
    std::memset(&A, 0, sizeof(A));
    A.q = plane(q, s->q_stride);
    A.k = plane(k, s->k_stride);
    A.v = plane(v, s->v_stride);
    A.beta = beta;
    A.decay = log_decay;
    A.gate_b = s->gate_stride[0], A.gate_h = s->gate_stride[1], A.gate_t = s->gate_stride[2];
    A.resets = resets;
    A.h0 = h0;
    A.B = s->B, A.T = s->T, A.Hk = (int32_t)s->Hk, A.Hv = (int32_t)s->Hv;
    A.key = (int32_t)s->dk, A.value = (int32_t)s->dv;
    A.chunks = (s->T + chunk_of(dtype) - 1) / chunk_of(dtype);
    A.value_pad = (int32_t)((s->dv + 31) / 32 * 32);
    const int columns = wide_chains(s) ? kWide : kNarrow;
    A.blocks = (A.value_pad + columns - 1) / columns;
    A.scale = scale;
    char *const base = static_cast<char *>(ws);
    A.key_pad = (A.key + 15) / 16 * 16;
    A.per = (int32_t)l.per, A.segments = (int32_t)l.segments;
    if (l.segments > 1) {
        A.maps = reinterpret_cast<float *>(base + l.maps);
        A.marks = reinterpret_cast<float *>(base + l.marks);
        A.cuts = reinterpret_cast<int32_t *>(base + l.cuts);
    }
    A.inverse = reinterpret_cast<Fragment *>(base + l.inverse);
    if (adjoint) {
        A.inverse_t = reinterpret_cast<Fragment *>(base + l.inverse_t);
        A.states = reinterpret_cast<float *>(base + l.states);
        A.dstates = reinterpret_cast<float *>(base + l.dstates);
        A.w = reinterpret_cast<float *>(base + l.w);
        A.x = reinterpret_cast<float *>(base + l.x);
    }
    return PARARNN_OK;
}

// Queries and keys go to LDS as they lie in memory, the steps side by side or
// the channels; other strides are gathered.
bool time_first(const pararnn_delta_shape_t *s) { return s->k_stride[3] == 1 || s->k_stride[2] != 1; }

template <bool ADJOINT, bool HALF>
pararnn_status_t run(const Args &A, const pararnn_delta_shape_t *s, void *stream)
{
    const bool tf = time_first(s), w = wide_chains(s);
    switch (room_of(s->dk)) {
    case 64: return ADJOINT ? run_adjoint<HALF, 64>(A, tf, w, stream) : run_scan<HALF, 64>(A, tf, w, stream);
    case 128: return ADJOINT ? run_adjoint<HALF, 128>(A, tf, w, stream) : run_scan<HALF, 128>(A, tf, w, stream);
    default: return ADJOINT ? run_adjoint<HALF, 256>(A, tf, w, stream) : run_scan<HALF, 256>(A, tf, w, stream);
    }
}

template <bool HALF>
void launch_step(const StepArgs &A, hipStream_t st)
{
    const dim3 grid((unsigned)(A.B * A.Hv * A.blocks)), block(kStepThreads);
    if (A.key <= 64)
        hipLaunchKernelGGL((delta_step_kernel<HALF, 4>), grid, block, 0, st, A);
    else if (A.key <= 128)
        hipLaunchKernelGGL((delta_step_kernel<HALF, 8>), grid, block, 0, st, A);
    else
        hipLaunchKernelGGL((delta_step_kernel<HALF, 16>), grid, block, 0, st, A);
}

}  // namespace

extern "C" {

size_t pararnn_delta_workspace_bytes(const pararnn_delta_shape_t *shape, pararnn_dtype_t dtype, int adjoint)
{
    if (check_delta(shape, dtype, false, !adjoint) != PARARNN_OK) return 0;
    return layout(shape, dtype, adjoint != 0).total;
}

pararnn_status_t pararnn_delta_scan(const pararnn_delta_shape_t *shape, const void *q, const void *k, const void *v,
                                    pararnn_dtype_t dtype, const float *beta, const float *log_decay, const float *h0,
                                    const uint8_t *resets, float scale, float *o, float *last, void *ws,
                                    size_t ws_bytes, void *stream)
{
    Args A;
    const pararnn_status_t st = prepare(A, shape, dtype, q, k, v, beta, log_decay, h0, resets, scale, false, ws, ws_bytes);
    if (st != PARARNN_OK) return st;
    if (A.B == 0 || A.Hv == 0) return PARARNN_OK;
    if (A.T > 0 && !o) return PARARNN_ERR_INVALID;
    A.o = plane(o, shape->o_stride);
    A.last = last;
    return dtype == PARARNN_BF16 ? run<false, true>(A, shape, stream) : run<false, false>(A, shape, stream);
}

pararnn_status_t pararnn_delta_scan_adjoint(const pararnn_delta_shape_t *shape, const void *q, const void *k,
                                            const void *v, pararnn_dtype_t dtype, const float *beta,
                                            const float *log_decay, const float *h0, const uint8_t *resets,
                                            float scale, const float *go, const float *g_last,
                                            const pararnn_delta_grads_t *g, void *ws, size_t ws_bytes, void *stream)
{
    Args A;
    const pararnn_status_t st = prepare(A, shape, dtype, q, k, v, beta, log_decay, h0, resets, scale, true, ws, ws_bytes);
    if (st != PARARNN_OK) return st;
    if (!g) return PARARNN_ERR_INVALID;
    const int64_t key[4] = {A.B, A.Hk, A.key, A.T}, value[4] = {A.B, A.Hv, A.value, A.T};
    if (!fits(key, g->dq_stride, true) || !fits(key, g->dk_stride, true) || !fits(value, g->dv_stride, true))
        return PARARNN_ERR_INVALID;
    if (A.B == 0 || A.Hv == 0) return PARARNN_OK;
    if (A.T > 0 && (!g->dq || !g->dk || !g->dv || !g->dbeta || (log_decay && !g->dlog_decay)))
        return PARARNN_ERR_INVALID;
    A.o = plane(go, shape->o_stride);
    A.g_last = g_last;
    A.dq = plane(g->dq, g->dq_stride);
    A.dk = plane(g->dk, g->dk_stride);
    A.dv = plane(g->dv, g->dv_stride);
    A.dbeta = g->dbeta;
    A.ddecay = log_decay ? g->dlog_decay : nullptr;
    A.dh0 = g->dh0;
    return dtype == PARARNN_BF16 ? run<true, true>(A, shape, stream) : run<true, false>(A, shape, stream);
}

pararnn_status_t pararnn_delta_step(const pararnn_delta_shape_t *shape, const void *q, const void *k, const void *v,
                                    pararnn_dtype_t dtype, const float *beta, const float *log_decay,
                                    const int32_t *slots, float *states, int64_t pool, float scale, float *o,
                                    void *stream)
{
    const pararnn_status_t st = check_delta(shape, dtype, true, true);
    if (st != PARARNN_OK) return st;
    if (pool < 0 || !std::isfinite(scale)) return PARARNN_ERR_INVALID;
    if (shape->B == 0 || shape->Hv == 0) return PARARNN_OK;
    if (!q || !k || !v || !beta || !o || (pool > 0 && !states)) return PARARNN_ERR_INVALID;
    if (pool > INT64_MAX / 8 / shape->dk / shape->dv / shape->Hv) return PARARNN_ERR_INVALID;
    StepArgs A;
    std::memset(&A, 0, sizeof(A));
    A.q = q, A.k = k, A.v = v, A.beta = beta, A.decay = log_decay, A.slots = slots, A.states = states, A.o = o;
    A.q_b = shape->q_stride[0], A.q_h = shape->q_stride[1], A.q_d = shape->q_stride[2];
    A.k_b = shape->k_stride[0], A.k_h = shape->k_stride[1], A.k_d = shape->k_stride[2];
    A.v_b = shape->v_stride[0], A.v_h = shape->v_stride[1], A.v_d = shape->v_stride[2];
    A.o_b = shape->o_stride[0], A.o_h = shape->o_stride[1], A.o_d = shape->o_stride[2];
    A.gate_b = shape->gate_stride[0], A.gate_h = shape->gate_stride[1];
    A.B = shape->B, A.pool = pool, A.scale = scale;
    A.Hk = (int32_t)shape->Hk, A.Hv = (int32_t)shape->Hv, A.key = (int32_t)shape->dk, A.value = (int32_t)shape->dv;
    A.blocks = (A.value + kStepColumns - 1) / kStepColumns;
    hipStream_t strm = static_cast<hipStream_t>(stream);
    if (dtype == PARARNN_BF16)
        launch_step<true>(A, strm);
    else
        launch_step<false>(A, strm);
    return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP;
}

}  // extern "C"
