// Gated linear recurrence, forward, backward and for one step:
//     l_t = -power softplus(lam) sig(u_r),  a_t = exp(l_t),
//     h_t = k_t a_t h_{t-1} + sqrt(1 - a_t^2) sig(u_i) u_x,
// k_t = 0 at the first step of a document, else 1.  The affine maps
// (k_t a_t, b_t) compose associatively, so a channel's steps may be split
// anywhere: a span's maps compose to one map, and the state before a span is
// the earlier spans' maps applied to h_0 ("Параллельность RNN?", forpes.ru,
// §1.3, level 2, is the same scan with the Newton system's maps).
//
// Numbers.  Slow channels have a_t close to 1, where exp(l) in float32 has
// lost l.  So the decay is computed as m = 1 - exp(l) from
//     exp(l) - 1 = 2 exp(l/2) sinh(l/2),
// with sinh's odd polynomial below |l| = 1 (first term left out: 1e-8 of the
// sum) and 1 - exp(l/2)^2 above, where nothing cancels.  Then
// 1 - a^2 = m (2 - m) holds full relative precision too.  Everything is
// float32; only bf16 gradients are rounded, once, when they are stored.
#pragma once

#include "elements.hpp"

namespace pararnn {

struct GatedArgs {
    const void *u[3];       // r, i, x
    const float *lam;       // [D]
    const float *h0;        // [B][D] or null
    const uint8_t *resets;  // [B][T] or null
    float *h;               // forward: out
    float *h_last;          // [B][D] or null
    // backward
    const float *hs;        // the forward's states
    const float *gh;        // or null
    const float *gh_last;   // or null
    void *du[3];
    float *dlam, *dh0;
    float *dlam_part;       // [B][nseg][D]
    // spans of the time axis
    float2 *agg;            // [nseg][channels]
    int64_t seg_len;
    int32_t nseg;
    float power;
    int64_t B, T, D, channels;
    int64_t usb, usd, ust, ssb, ssd, sst;
};

// log2 of the decay at sig(u_r) = 1: -power softplus(lam) log2(e).
__device__ __forceinline__ float decay_rate(float lam, float power)
{
    const float sp = fmaxf(lam, 0.0f) + log1pf(expf(-fabsf(lam)));
    // fmaxf drops a NaN lam: put it back
    return lam != lam ? lam : -power * sp * kLog2e;
}

struct Decay {
    float q;   // sig(u_r)
    float l2;  // log2 a
    float m;   // 1 - a
    float y;   // 1 - a^2
};
__device__ __forceinline__ Decay decay(float rate, float r)
{
    Decay v;
    v.q = sigmoid_q(-kLog2e * r);
    v.l2 = rate * v.q;
    const float x = v.l2 * 0.34657359027997264f;  // l / 2
    const float t = ex2(0.5f * v.l2);             // exp(l / 2)
    const float s = x * x;
    const float p = fmaf_(s, fmaf_(s, fmaf_(s, 1.9841270e-4f, 8.3333333e-3f), 0.16666667f), 1.0f);
    v.m = x > -0.5f ? -2.0f * t * (x * p) : fmaf_(-t, t, 1.0f);
    v.y = fmaf_(-v.m, v.m, 2.0f * v.m);
    return v;
}

// The step map of h: (k a, b).
__device__ __forceinline__ Map1 gated_map(float rate, float r, float i, float x, bool reset)
{
    const Decay v = decay(rate, r);
    return {reset ? 0.0f : 1.0f - v.m,
            __builtin_amdgcn_sqrtf(v.y) * sigmoid_q(-kLog2e * i) * x};
}

// Gradients of one step from G = dL/dh_t (total) and h_{t-1}.  With
// a' = k a: dL/dl = G (a' h_{t-1} - a^2 / sqrt(1 - a^2) sig(u_i) u_x).  Where
// l has underflowed to 0 the second term's own factor (l, or sig(u_r)) makes
// the product 0; the division is left out there.
struct GatedGrad {
    float r, i, x;
    float lam;  // dL/dl sig(u_r), to be summed
};
__device__ __forceinline__ GatedGrad gated_grad(const Decay &v, float ui, float ux, bool reset,
                                                float G, float hp)
{
    const float inv = v.y > 1e-30f ? __builtin_amdgcn_rsqf(v.y) : 0.0f;
    const float gain = v.y * inv;
    const float si = sigmoid_q(-kLog2e * ui);
    const float a = 1.0f - v.m;
    GatedGrad g;
    g.x = G * gain * si;
    g.i = g.x * ux * (1.0f - si);
    const float carried = reset ? 0.0f : a * hp;
    const float dl = G * (carried - fmaf_(-v.y, inv, inv) * (si * ux));
    g.lam = dl * v.q;
    g.r = dl * (v.l2 * 0.6931471805599453f) * (1.0f - v.q);
    return g;
}

// ------------------------------------------------------ lane per channel ---
// Any layout: lane = channel, so time-major planes load coalesced, and a
// single token of many requests is one step of every lane.  kSteps steps are
// loaded before the first is used.  With few channels the time axis is cut
// into spans: one launch composes every span's map (AGG), the next applies
// the maps of the spans before it and runs the span again.
constexpr int kGatedSteps = 8;

template <bool BF16, bool AGG>
__global__ void __launch_bounds__(kWave) gated_channel_kernel(GatedArgs A)
{
    const int64_t ch = (int64_t)blockIdx.x * kWave + threadIdx.x;
    if (ch >= A.channels) return;
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const int32_t seg = blockIdx.y;
    const int64_t t0 = seg * A.seg_len, t1 = min(A.T, t0 + A.seg_len);
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const uint8_t *rs = A.resets ? A.resets + b * A.T : nullptr;

    Map1 span = {1.0f, 0.0f};
    float h = A.h0 ? A.h0[ch] : 0.0f;
    if constexpr (!AGG)
        for (int32_t j = 0; j < seg; ++j) {
            const float2 m = A.agg[(int64_t)j * A.channels + ch];
            h = fmaf_(m.x, h, m.y);
        }
    for (int64_t t = t0; t < t1; t += kGatedSteps) {
        float u[3][kGatedSteps];
        bool cut[kGatedSteps];
#pragma unroll
        for (int k = 0; k < kGatedSteps; ++k) {
            const bool in = t + k < t1;
            const int64_t o = uo + (in ? t + k : t) * A.ust;
#pragma unroll
            for (int g = 0; g < 3; ++g) u[g][k] = load_gate<BF16>(A.u[g], o);
            cut[k] = rs && rs[in ? t + k : t] != 0;
        }
#pragma unroll
        for (int k = 0; k < kGatedSteps; ++k) {
            if (t + k >= t1) break;
            const Map1 m = gated_map(rate, u[0][k], u[1][k], u[2][k], cut[k]);
            if constexpr (AGG) {
                span = compose(m, span);
            } else {
                h = fmaf_(m.a, h, m.b);
                A.h[so + (t + k) * A.sst] = h;
            }
        }
    }
    if constexpr (AGG)
        A.agg[(int64_t)seg * A.channels + ch] = make_float2(span.a, span.b);
    else if (A.h_last && seg == A.nseg - 1)
        A.h_last[ch] = h;
}

// Backward: with w_t = dL/dh_{t-1} through step t alone,
//     w_t = k_t a_t (gh_t + w_{t+1}),  w_{T+1} = gh_last,  dL/dh_0 = w_1,
// again affine maps, composed from the last span to the first.
template <bool BF16, bool AGG>
__global__ void __launch_bounds__(kWave) gated_channel_adjoint_kernel(GatedArgs A)
{
    const int64_t ch = (int64_t)blockIdx.x * kWave + threadIdx.x;
    if (ch >= A.channels) return;
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const int32_t seg = blockIdx.y + (AGG ? 1 : 0);
    const int64_t t0 = seg * A.seg_len, t1 = min(A.T, t0 + A.seg_len);
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const uint8_t *rs = A.resets ? A.resets + b * A.T : nullptr;

    Map1 span = {1.0f, 0.0f};
    float w = A.gh_last ? A.gh_last[ch] : 0.0f;
    if constexpr (!AGG)
        for (int32_t j = A.nseg - 1; j > seg; --j) {
            const float2 m = A.agg[(int64_t)j * A.channels + ch];
            w = fmaf_(m.x, w, m.y);
        }
    const float h0 = A.h0 ? A.h0[ch] : 0.0f;
    float dlam = 0.0f;
    for (int64_t t = t1 - 1; t >= t0; t -= kGatedSteps) {
        float u[3][kGatedSteps], hp[kGatedSteps], gh[kGatedSteps];
        bool cut[kGatedSteps];
#pragma unroll
        for (int k = 0; k < kGatedSteps; ++k) {
            const int64_t tk = t - k >= t0 ? t - k : t;
            const int64_t o = uo + tk * A.ust;
            u[0][k] = load_gate<BF16>(A.u[0], o);
            cut[k] = rs && rs[tk] != 0;
            gh[k] = A.gh ? A.gh[so + tk * A.sst] : 0.0f;
            if constexpr (!AGG) {
                u[1][k] = load_gate<BF16>(A.u[1], o);
                u[2][k] = load_gate<BF16>(A.u[2], o);
                hp[k] = tk > 0 ? A.hs[so + (tk - 1) * A.sst] : h0;
            }
        }
#pragma unroll
        for (int k = 0; k < kGatedSteps; ++k) {
            if (t - k < t0) break;
            const Decay v = decay(rate, u[0][k]);
            const float ka = cut[k] ? 0.0f : 1.0f - v.m;
            if constexpr (AGG) {
                span = compose({ka, ka * gh[k]}, span);
            } else {
                const float G = gh[k] + w;
                w = ka * G;
                const GatedGrad g = gated_grad(v, u[1][k], u[2][k], cut[k], G, hp[k]);
                const int64_t o = uo + (t - k) * A.ust;
                store_gate<BF16>(A.du[0], o, g.r);
                store_gate<BF16>(A.du[1], o, g.i);
                store_gate<BF16>(A.du[2], o, g.x);
                dlam += g.lam;
            }
        }
    }
    if constexpr (AGG) {
        A.agg[(int64_t)seg * A.channels + ch] = make_float2(span.a, span.b);
    } else {
        A.dlam_part[(b * A.nseg + seg) * A.D + d] = dlam;
        if (A.dh0 && seg == 0) A.dh0[ch] = w;
    }
}

// ---------------------------------------------------------- lanes in time ---
// Time-contiguous planes: a channel's steps side by side in the lanes of W
// waves, K steps a lane, so that every load and store of a wave is one
// contiguous run.  Per chunk of 64 K W steps a lane composes its own steps,
// the wave scans the lanes' maps (DPP), W > 1 waves exchange their totals
// through LDS (one barrier a chunk, two buffers), and every lane runs its
// steps again from the state in front of them.  The chunk's last state starts
// the next one; the next chunk's loads are issued before this one's scan.
template <int K, bool BF16>
struct GatedChunk {
    Raw<BF16, K> u[3];
    uint32_t cut;
};
template <int K, bool BF16>
__device__ __forceinline__ GatedChunk<K, BF16> load_chunk(const GatedArgs &A, int64_t uo,
                                                          const uint8_t *rs, int64_t t, int64_t t1)
{
    GatedChunk<K, BF16> c;
#pragma unroll
    for (int g = 0; g < 3; ++g) c.u[g] = load_raw<BF16, K>(A.u[g], uo, t, t1);
    c.cut = rs ? load_flags<K>(rs, t, t1) : 0u;
    return c;
}

// The state before wave `wave`'s part of the chunk, from the one before the
// chunk and the waves' maps in order; `carry` moves on to the next chunk.
template <int W>
__device__ __forceinline__ float through_waves(const Map1 *maps, int wave, float &carry)
{
    float mine = carry;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w == wave) mine = carry;
        carry = fmaf_(maps[w].a, carry, maps[w].b);
    }
    return mine;
}

template <bool BF16, int K, int W, bool AGG>
__global__ void __launch_bounds__(W * kWave) gated_time_kernel(GatedArgs A)
{
    __shared__ Map1 maps[2][W];
    const int64_t ch = blockIdx.x;
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const int32_t seg = blockIdx.y;
    const int64_t t0 = seg * A.seg_len, t1 = min(A.T, t0 + A.seg_len);
    const int wave = threadIdx.x / kWave;
    constexpr int P = K * W * kWave;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const uint8_t *rs = A.resets ? A.resets + b * A.T : nullptr;

    Map1 span = {1.0f, 0.0f};
    float carry = A.h0 ? A.h0[ch] : 0.0f;
    if constexpr (!AGG)
        for (int32_t j = 0; j < seg; ++j) {
            const float2 m = A.agg[(int64_t)j * A.channels + ch];
            carry = fmaf_(m.x, carry, m.y);
        }
    int64_t t = t0 + (int64_t)threadIdx.x * K;
    GatedChunk<K, BF16> now = load_chunk<K, BF16>(A, uo, rs, t, t1);
    int parity = 0;
    for (int64_t c = t0; c < t1; c += P, t += P, parity ^= 1) {
        GatedChunk<K, BF16> next;
        if (c + P < t1) next = load_chunk<K, BF16>(A, uo, rs, t + P, t1);
        Map1 m[K], own = {1.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            m[k] = gated_map(rate, now.u[0].get(k), now.u[1].get(k), now.u[2].get(k),
                             now.cut >> k & 1u);
            m[k] = keep_or_identity(m[k], t + k < t1);
            own = compose(m[k], own);
        }
        const Map1 upto = wave_scan_inclusive(own);
        float before = carry;
        if constexpr (W > 1) {
            if (threadIdx.x % kWave == kWave - 1) maps[parity][wave] = upto;
            __syncthreads();
            if constexpr (AGG) {
#pragma unroll
                for (int w = 0; w < W; ++w) span = compose(maps[parity][w], span);
            } else {
                before = through_waves<W>(maps[parity], wave, carry);
            }
        } else if constexpr (AGG) {
            span = compose(upto, span);  // in the last lane
        }
        if constexpr (!AGG) {
            const Map1 prior = wave_shift_up(upto);
            float h = fmaf_(prior.a, before, prior.b);
            float out[K];
#pragma unroll
            for (int k = 0; k < K; ++k) out[k] = h = fmaf_(m[k].a, h, m[k].b);
            store_raw<false, K>(A.h, so, t, t1, out);
            if constexpr (W == 1) carry = __shfl(h, kWave - 1);
            if (A.h_last && t < A.T && t + K >= A.T)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (t + k == A.T - 1) A.h_last[ch] = out[k];
        }
        now = next;
    }
    if constexpr (AGG)
        if (threadIdx.x == W * kWave - 1)
            A.agg[(int64_t)seg * A.channels + ch] = make_float2(span.a, span.b);
}

// Backward: lanes run backwards in time (lane 0 holds a chunk's last steps),
// so that the same scan composes the maps of w from the end.
template <int K, bool BF16>
struct GatedBackChunk {
    Raw<BF16, K> u[3];
    Raw<false, K> h, gh;
    float before;  // the state in front of the wave's steps
    uint32_t cut;
};
template <int K, bool BF16, bool AGG>
__device__ __forceinline__ GatedBackChunk<K, BF16> load_back(const GatedArgs &A, int64_t uo,
                                                             int64_t so, const uint8_t *rs,
                                                             int64_t t, int64_t first, int64_t t1,
                                                             float h0)
{
    GatedBackChunk<K, BF16> c;
    c.u[0] = load_raw<BF16, K>(A.u[0], uo, t, t1);
    if constexpr (!AGG) {
        c.u[1] = load_raw<BF16, K>(A.u[1], uo, t, t1);
        c.u[2] = load_raw<BF16, K>(A.u[2], uo, t, t1);
        c.h = load_raw<false, K>(A.hs, so, t, t1);
        c.before = first > 0 && first <= A.T ? A.hs[so + first - 1] : h0;
    }
    if (A.gh) {
        c.gh = load_raw<false, K>(A.gh, so, t, t1);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) c.gh.w[k] = 0u;
    }
    c.cut = rs ? load_flags<K>(rs, t, t1) : 0u;
    return c;
}

template <bool BF16, int K, int W, bool AGG>
__global__ void __launch_bounds__(W * kWave) gated_time_adjoint_kernel(GatedArgs A)
{
    __shared__ Map1 maps[2][W];
    __shared__ float sums[W];
    const int64_t ch = blockIdx.x;
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const int32_t seg = blockIdx.y + (AGG ? 1 : 0);
    const int64_t t0 = seg * A.seg_len, t1 = min(A.T, t0 + A.seg_len);
    const int wave = threadIdx.x / kWave;
    constexpr int P = K * W * kWave;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const uint8_t *rs = A.resets ? A.resets + b * A.T : nullptr;

    Map1 span = {1.0f, 0.0f};
    float carry = A.gh_last ? A.gh_last[ch] : 0.0f, dlam = 0.0f;
    const float h0 = A.h0 ? A.h0[ch] : 0.0f;
    if constexpr (!AGG)
        for (int32_t j = A.nseg - 1; j > seg; --j) {
            const float2 m = A.agg[(int64_t)j * A.channels + ch];
            carry = fmaf_(m.x, carry, m.y);
        }
    int64_t c = t0 + (t1 - t0 - 1) / P * P;  // the last chunk of the span
    const int at = W * kWave - 1 - (int)threadIdx.x, wave_at = (W - 1 - wave) * kWave;
    GatedBackChunk<K, BF16> now =
        load_back<K, BF16, AGG>(A, uo, so, rs, c + at * K, c + wave_at * K, t1, h0);
    int parity = 0;
    for (; c >= t0; c -= P, parity ^= 1) {
        const int64_t t = c + at * K;
        GatedBackChunk<K, BF16> next;
        if (c > t0)
            next = load_back<K, BF16, AGG>(A, uo, so, rs, t - P, c - P + wave_at * K, t1, h0);
        Decay v[K];
        Map1 own = {1.0f, 0.0f};
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            v[k] = decay(rate, now.u[0].get(k));
            const float ka = now.cut >> k & 1u ? 0.0f : 1.0f - v[k].m;
            own = compose(keep_or_identity(Map1{ka, ka * now.gh.get(k)}, t + k < t1), own);
        }
        const Map1 upto = wave_scan_inclusive(own);
        float after = carry;
        if constexpr (W > 1) {
            if (threadIdx.x % kWave == kWave - 1) maps[parity][wave] = upto;
            __syncthreads();
            if constexpr (AGG) {
#pragma unroll
                for (int w = 0; w < W; ++w) span = compose(maps[parity][w], span);
            } else {
                after = through_waves<W>(maps[parity], wave, carry);
            }
        } else if constexpr (AGG) {
            span = compose(upto, span);
        }
        if constexpr (!AGG) {
            const Map1 prior = wave_shift_up(upto);
            float w = fmaf_(prior.a, after, prior.b);
            // the state before the lane's first step: the next lane's last one
            float hp0 = __shfl_down(now.h.get(K - 1), 1);
            if (threadIdx.x % kWave == kWave - 1) hp0 = now.before;
            float gr[K], gi[K], gx[K];
#pragma unroll
            for (int k = K - 1; k >= 0; --k) {
                const bool cut = now.cut >> k & 1u, in = t + k < t1;
                const float G = now.gh.get(k) + w;
                const GatedGrad g = gated_grad(v[k], now.u[1].get(k), now.u[2].get(k), cut, G,
                                               k ? now.h.get(k ? k - 1 : 0) : hp0);
                gr[k] = g.r, gi[k] = g.i, gx[k] = g.x;
                dlam += in ? g.lam : 0.0f;
                w = in ? (cut ? 0.0f : (1.0f - v[k].m) * G) : w;
            }
            store_raw<BF16, K>(A.du[0], uo, t, t1, gr);
            store_raw<BF16, K>(A.du[1], uo, t, t1, gi);
            store_raw<BF16, K>(A.du[2], uo, t, t1, gx);
            if constexpr (W == 1) carry = __shfl(w, kWave - 1);
            if (A.dh0 && c == 0 && threadIdx.x == W * kWave - 1) A.dh0[ch] = w;
        }
        now = next;
    }
    if constexpr (AGG) {
        if (threadIdx.x == W * kWave - 1)
            A.agg[(int64_t)seg * A.channels + ch] = make_float2(span.a, span.b);
    } else {
        float s = wave_sum_to_last(dlam);
        if constexpr (W > 1) {
            if (threadIdx.x % kWave == kWave - 1) sums[wave] = s;
            __syncthreads();
            s = 0.0f;
            for (int w = 0; w < W; ++w) s += sums[w];
        }
        if (threadIdx.x == W * kWave - 1) A.dlam_part[(b * A.nseg + seg) * A.D + d] = s;
    }
}

// --------------------------------------------------- lanes in time, short ---
// At most G K steps: G lanes a channel and 64 / G channels a wave, each lane's
// K steps in one access as above.  (With a wave a channel, T = 100 of 64000
// channels left 7 of 8 lanes idle.)
constexpr int kShortThreads = 256;

// Inclusive scan of the maps over groups of G neighbouring lanes, each group's
// first lane first (its last, REVERSE); then the map in front of the lane's own.
template <int G, bool REVERSE>
__device__ __forceinline__ Map1 group_scan_exclusive(Map1 x)
{
    const int lane = threadIdx.x % G, at = REVERSE ? G - 1 - lane : lane;
#pragma unroll
    for (int o = 1; o < G; o *= 2) {
        const Map1 y = REVERSE ? Map1{__shfl_down(x.a, o), __shfl_down(x.b, o)}
                               : Map1{__shfl_up(x.a, o), __shfl_up(x.b, o)};
        if (at >= o) x = compose(x, y);
    }
    const Map1 y = REVERSE ? Map1{__shfl_down(x.a, 1), __shfl_down(x.b, 1)}
                           : Map1{__shfl_up(x.a, 1), __shfl_up(x.b, 1)};
    return at > 0 ? y : Map1{1.0f, 0.0f};
}

template <bool BF16, int K, int G>
__global__ void __launch_bounds__(kShortThreads) gated_short_kernel(GatedArgs A)
{
    const int64_t ch = ((int64_t)blockIdx.x * kShortThreads + threadIdx.x) / G;
    const bool here = ch < A.channels;  // the others follow along for the shuffles
    const int64_t b = here ? ch / A.D : 0, d = here ? ch - b * A.D : 0;
    const int64_t t = (int64_t)(threadIdx.x % G) * K, end = here ? A.T : 0;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const uint8_t *rs = A.resets ? A.resets + b * A.T : nullptr;
    const GatedChunk<K, BF16> c = load_chunk<K, BF16>(A, uo, rs, t, end);
    const float h0 = A.h0 && here ? A.h0[ch] : 0.0f;
    Map1 m[K], own = {1.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
        m[k] = gated_map(rate, c.u[0].get(k), c.u[1].get(k), c.u[2].get(k), c.cut >> k & 1u);
        m[k] = keep_or_identity(m[k], t + k < end);
        own = compose(m[k], own);
    }
    const Map1 prior = group_scan_exclusive<G, false>(own);
    float h = fmaf_(prior.a, h0, prior.b), out[K];
#pragma unroll
    for (int k = 0; k < K; ++k) out[k] = h = fmaf_(m[k].a, h, m[k].b);
    if (t >= end) return;
    store_raw<false, K>(A.h, so, t, end, out);
    if (A.h_last)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t + k == A.T - 1) A.h_last[ch] = out[k];
}

template <bool BF16, int K, int G>
__global__ void __launch_bounds__(kShortThreads) gated_short_adjoint_kernel(GatedArgs A)
{
    const int64_t ch = ((int64_t)blockIdx.x * kShortThreads + threadIdx.x) / G;
    const bool here = ch < A.channels;
    const int64_t b = here ? ch / A.D : 0, d = here ? ch - b * A.D : 0;
    const int64_t t = (int64_t)(threadIdx.x % G) * K, end = here ? A.T : 0;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const uint8_t *rs = A.resets ? A.resets + b * A.T : nullptr;
    const float h0 = A.h0 && here ? A.h0[ch] : 0.0f;
    const GatedBackChunk<K, BF16> c = load_back<K, BF16, false>(A, uo, so, rs, t, 0, end, h0);
    const float after = A.gh_last && here ? A.gh_last[ch] : 0.0f;
    Decay v[K];
    Map1 own = {1.0f, 0.0f};
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        v[k] = decay(rate, c.u[0].get(k));
        const float ka = c.cut >> k & 1u ? 0.0f : 1.0f - v[k].m;
        own = compose(keep_or_identity(Map1{ka, ka * c.gh.get(k)}, t + k < end), own);
    }
    const Map1 prior = group_scan_exclusive<G, true>(own);
    float w = fmaf_(prior.a, after, prior.b);
    float hp = __shfl_up(c.h.get(K - 1), 1);
    if (threadIdx.x % G == 0) hp = h0;
    float gr[K], gi[K], gx[K], dlam = 0.0f;
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        const bool cut = c.cut >> k & 1u, in = t + k < end;
        const float g_total = c.gh.get(k) + w;
        const GatedGrad g = gated_grad(v[k], c.u[1].get(k), c.u[2].get(k), cut, g_total,
                                       k ? c.h.get(k ? k - 1 : 0) : hp);
        gr[k] = g.r, gi[k] = g.i, gx[k] = g.x;
        dlam += in ? g.lam : 0.0f;
        w = in ? (cut ? 0.0f : (1.0f - v[k].m) * g_total) : w;
    }
#pragma unroll
    for (int o = 1; o < G; o *= 2) dlam += __shfl_xor(dlam, o);
    if (t >= end) return;
    store_raw<BF16, K>(A.du[0], uo, t, end, gr);
    store_raw<BF16, K>(A.du[1], uo, t, end, gi);
    store_raw<BF16, K>(A.du[2], uo, t, end, gx);
    if (t > 0) return;
    if (A.dh0) A.dh0[ch] = w;
    A.dlam_part[b * A.D + d] = dlam;  // one span
}

// dL/dlam = -power sig(lam) sum (dL/dl sig(u_r)), the partial sums of the
// batch rows and spans added in a fixed order.
__global__ void gated_dlam_kernel(GatedArgs A)
{
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= A.D) return;
    float s = 0.0f;
    const int64_t n = A.B * A.nseg;
    for (int64_t j = 0; j < n; ++j) s += A.dlam_part[j * A.D + d];
    A.dlam[d] = -A.power * sigmoid_q(-kLog2e * A.lam[d]) * s;
}

// ----------------------------------------------------------- one step ---
struct GatedStepArgs {
    const void *u[3];
    const float *lam;
    const int32_t *slots;
    float *states, *out;
    int64_t B, D, usb, pool;
    float power;
};
constexpr int kGatedStepThreads = 256;

template <bool BF16>
__global__ void __launch_bounds__(kGatedStepThreads) gated_step_kernel(GatedStepArgs A)
{
    const int64_t d = (int64_t)blockIdx.x * kGatedStepThreads + threadIdx.x;
    if (d >= A.D) return;
    for (int64_t b = blockIdx.y; b < A.B; b += gridDim.y) {
        const int64_t slot = A.slots ? A.slots[b] : b;
        if (slot < 0 || slot >= A.pool) {
            A.out[b * A.D + d] = 0.0f;
            continue;
        }
        const int64_t o = b * A.usb + d;
        const Map1 m = gated_map(decay_rate(A.lam[d], A.power), load_gate<BF16>(A.u[0], o),
                                 load_gate<BF16>(A.u[1], o), load_gate<BF16>(A.u[2], o), false);
        float *s = A.states + slot * A.D + d;
        const float h = fmaf_(m.a, *s, m.b);
        *s = h;
        A.out[b * A.D + d] = h;
    }
}

}  // namespace pararnn
