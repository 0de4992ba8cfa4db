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
// lost l.  So m = 1 - exp(l) is computed from
//     exp(l) - 1 = 2 exp(l/2) sinh(l/2),
// with sinh's odd polynomial below |l| = 1 (first term left out: 1e-8 of the
// sum) and 1 - exp(l/2)^2 above, where nothing cancels.  Then
// 1 - a^2 = m (2 - m) holds full relative precision too.  The decay itself is
// 1 - m below |l| = 1 and exp(l/2)^2 above, where 1 - m would have lost it: the
// states of fast channels keep their relative precision.  Everything is
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
    float *dlam_part;       // [place][B][D]
    // look back
    uint32_t *ticket;       // a line a channel, or a group of 64
    union {
        struct GatedRecord *records;  // [place][channels]
        uint64_t *words;              // [place][3][channels]; null: one place
    };
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
    float a;
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
    const bool slow = x > -0.5f;
    const float m = slow ? -2.0f * t * (x * p) : fmaf_(-t, t, 1.0f);
    v.a = slow ? 1.0f - m : t * t;
    v.y = fmaf_(-m, m, 2.0f * m);
    return v;
}

// A step, or a span of steps: x -> a x + b, with l = log2 a.  Near a = 1 a
// product of decays loses at every step what its factors have lost; their
// logarithms add up in full.  So a span's a is 2^l, l the sum of its steps'.
// (A steady gate at -8 over 262144 steps: what is left of h_0 was off by 0.8%
// with products, with sums by 1e-5, in chunks of 64 steps by 1.5e-4.)
//
// A reset cuts: what is before it is not multiplied by 0, which would keep a
// NaN or an infinity, but left out.  A cut span has a = -0 (decays are not
// negative, and +0 where they underflow) and l = -inf.  Where every number is
// finite the product with -0 does the same: forward with lanes in time, and in
// the lanes' scan, it is done that way first, and once more, CAREFUL, where a
// lane of the wave ends with a number that is not finite, as any does that met
// one.  (Careful at once, 16x600x1024 float32 takes 42 us instead of 38.  With a
// lane a channel a first pass does not pay: 512x1x4096 bfloat16 28 us with it, 18
// without.)  Kernels without resets (DOCS false) do not look for cuts.
struct Span {
    float a, b, l;
};
constexpr float kCut = -0.0f, kNoMemory = -__builtin_inff();
template <bool DOCS>
__device__ __forceinline__ bool is_cut(float a)
{
    return DOCS && __float_as_uint(a) == 0x80000000u;
}
__device__ __forceinline__ bool any_not_finite(float x)
{
    return __ballot(!(fabsf(x) < __builtin_inff())) != 0;
}
template <bool CAREFUL, class M>
__device__ __forceinline__ float through(const M &m, float x)
{
    return is_cut<CAREFUL>(m.a) ? m.b : fmaf_(m.a, x, m.b);
}
template <bool DOCS>
__device__ __forceinline__ Span span_of(float l, float b)
{
    return {DOCS && l == kNoMemory ? kCut : ex2(l), b, l};
}
// L behind E, by the product of their decays; that of a cut E is -0 as well.
template <bool CAREFUL>
__device__ __forceinline__ Map1 joined(const Map1 &L, const Map1 &E)
{
    return {is_cut<CAREFUL>(L.a) ? L.a : L.a * E.a, through<CAREFUL>(L, E.b)};
}

// The span of the steps, or spans, added so far.
template <bool DOCS, bool CAREFUL>
struct Running {
    float l = 0.0f, b = 0.0f;
    __device__ __forceinline__ void add(const Span &m)
    {
        b = through<CAREFUL>(m, b);
        l = is_cut<DOCS>(m.a) ? kNoMemory : l + m.l;
    }
};
// `add_all` adds the steps in order; TWICE: without care first.
template <bool DOCS, bool TWICE, class F>
__device__ __forceinline__ Span sum_of(const F &add_all)
{
    Running<DOCS, DOCS && !TWICE> r;
    add_all(r);
    if constexpr (DOCS && TWICE) {
        if (any_not_finite(r.b)) {
            Running<DOCS, true> c;
            add_all(c);
            return span_of<DOCS>(c.l, c.b);
        }
    }
    return span_of<DOCS>(r.l, r.b);
}

template <bool DOCS>
__device__ __forceinline__ Span forward_step(float rate, float r, float i, float x, bool reset)
{
    const Decay v = decay(rate, r);
    return {DOCS && reset ? kCut : v.a, __builtin_amdgcn_sqrtf(v.y) * sigmoid_q(-kLog2e * i) * x,
            v.l2};
}
// Backwards, of w: w -> a (gh + w), from a span's last step to its first.  A step
// past the end (not `in`, gh = 0) comes before all others and leaves w, which is
// 0 in a span so far, as it is.  (Forward, steps past the end come last, and no
// one asks for what is behind them.)
template <bool DOCS>
struct RunningBack {
    float l = 0.0f, b = 0.0f;
    __device__ __forceinline__ void add(const Decay &v, float gh, bool reset, bool in)
    {
        const bool cut = DOCS && reset && in;
        b = cut ? 0.0f : v.a * (gh + b);
        l = cut ? kNoMemory : l + (in ? v.l2 : 0.0f);
    }
    __device__ __forceinline__ Span span() const { return span_of<DOCS>(l, b); }
};

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
    GatedGrad g;
    g.x = G * gain * si;
    g.i = g.x * ux * (1.0f - si);
    const float carried = reset ? 0.0f : v.a * hp;
    const float dl = G * (carried - v.a * v.a * inv * (si * ux));
    g.lam = dl * v.q;
    g.r = dl * (v.l2 * 0.6931471805599453f) * (1.0f - v.q);
    return g;
}

// -------------------------------------------------------------- look back ---
// Where there are too few channels to fill the device, the time axis is cut
// into chunks that run side by side, and the projections are still read once.
// A workgroup publishes its chunk's composed map, then looks back over a window
// of predecessors until one has published the state behind it and all nearer
// ones their maps, and applies these maps in order.  It publishes its own
// state, and runs its steps.  A state is always the one before it under the
// chunk's map, rounded once: the results do not depend on how far a workgroup
// had to look.  A channel's chunks are handed out by its ticket in the order of
// their places, so every predecessor is already running and the wait ends.
// (One ticket for all channels: 8192 chunks took 113 us, most of it in line for
// that word.)
//
// A published word is 64 bits, the value and a tag that is zero before, stored
// and loaded in one device-coherent access: no word is seen half written, and
// none needs the others' order.  Tickets and words are cleared by
// gated_clear_kernel.
__device__ __forceinline__ void publish(uint64_t *word, float v)
{
    __hip_atomic_store(word, (1ull << 32) | __float_as_uint(v), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t published(const uint64_t *word)
{
    return __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float read_lane(float v, int lane)
{
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
__device__ __forceinline__ float word_value(uint64_t w) { return __uint_as_float((uint32_t)w); }

__global__ void gated_clear_kernel(GatedArgs A, int64_t words)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < words) reinterpret_cast<uint64_t *>(A.ticket)[i] = 0;
}

// This workgroup's place in its channel.  A ticket has a line of its own.
constexpr int kTicketWords = 32;
__device__ __forceinline__ uint32_t take_ticket(const GatedArgs &A, int64_t ch, uint32_t *lds)
{
    if (threadIdx.x == 0) *lds = atomicAdd(A.ticket + ch * kTicketWords, 1u);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*lds);
}
// ------------------------------------------------------ lane per channel ---
// Any layout: lane = channel, so time-major planes load coalesced, and a
// single token of many requests is one step of every lane.  kGatedSteps steps
// are loaded before the first is used.
constexpr int kGatedSteps = 8;

template <int K>
struct LaneSteps {
    float u[3][K];
    bool cut[K];
};
// Steps t .. t + K - 1; those from T on repeat the last.
template <bool BF16, bool DOCS, int K>
__device__ __forceinline__ LaneSteps<K> lane_steps(const GatedArgs &A, int64_t uo, int64_t b,
                                                   int64_t t)
{
    LaneSteps<K> c;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t tk = min(t + k, A.T - 1);
#pragma unroll
        for (int g = 0; g < 3; ++g) c.u[g][k] = load_gate<BF16>(A.u[g], uo + tk * A.ust);
        c.cut[k] = DOCS && A.resets[b * A.T + tk] != 0;
    }
    return c;
}
// The states of steps t .. t + K - 1 from the one before them.
template <bool DOCS, int K>
__device__ __forceinline__ void lane_states(const GatedArgs &A, int64_t so, int64_t ch, int64_t t,
                                            const Span (&m)[K], float h)
{
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (t + k >= A.T) continue;
        h = through<DOCS>(m[k], h);
        A.h[so + (t + k) * A.sst] = h;
        if (A.h_last && t + k == A.T - 1) A.h_last[ch] = h;
    }
}
template <int K>
struct LaneBack {
    float hp[K], gh[K];  // the state before each step, its gradient
};
template <int K>
__device__ __forceinline__ LaneBack<K> lane_back(const GatedArgs &A, int64_t so, int64_t t, float h0)
{
    LaneBack<K> c;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t tk = min(t + k, A.T - 1);
        c.gh[k] = A.gh ? A.gh[so + tk * A.sst] : 0.0f;
        if (t + k >= A.T) c.gh[k] = 0.0f;
        c.hp[k] = tk > 0 ? A.hs[so + (tk - 1) * A.sst] : h0;
    }
    return c;
}
// The gradients of steps t + K - 1 .. t from w behind them: with w_t =
// dL/dh_{t-1} through step t alone,
//     w_t = k_t a_t (gh_t + w_{t+1}),  w_{T+1} = gh_last,  dL/dh_0 = w_1,
// again affine maps, composed from the last step to the first.
template <bool BF16, int K>
__device__ __forceinline__ float lane_gradients(const GatedArgs &A, int64_t uo, int64_t t,
                                                const LaneSteps<K> &c, const LaneBack<K> &e,
                                                const Decay (&v)[K], float w, float &dlam)
{
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        if (t + k >= A.T) continue;
        const float G = e.gh[k] + w;
        w = c.cut[k] ? 0.0f : v[k].a * G;
        const GatedGrad g = gated_grad(v[k], c.u[1][k], c.u[2][k], c.cut[k], G, e.hp[k]);
        const int64_t o = uo + (t + k) * A.ust;
        store_gate<BF16>(A.du[0], o, g.r);
        store_gate<BF16>(A.du[1], o, g.i);
        store_gate<BF16>(A.du[2], o, g.x);
        dlam += g.lam;
    }
    return w;
}

// Single tokens and short runs, or channels that fill the device: one lane runs
// its channel from end to end.  512x1x4096 time-major bfloat16 17 us; bound by
// the launch, and by the bytes where there are many channels (20x1000x4096
// float32 293 us, 4.5 TB/s).  The state goes on by 8 steps at a time: what a
// steady gate near no decay leaves of it after T steps is within 2^-22 T / 8 of
// itself.
template <bool BF16, bool DOCS>
__global__ void __launch_bounds__(kWave) gated_channel_kernel(GatedArgs A)
{
    const int64_t ch = (int64_t)blockIdx.x * kWave + threadIdx.x;
    if (ch >= A.channels) return;
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    float h = A.h0 ? A.h0[ch] : 0.0f;
    if (A.T == 0 && A.h_last) A.h_last[ch] = h;
    Span m[kGatedSteps];
    const auto load = [&](int64_t t) {
        const auto c = lane_steps<BF16, DOCS, kGatedSteps>(A, uo, b, t);
#pragma unroll
        for (int k = 0; k < kGatedSteps; ++k)
            m[k] = forward_step<DOCS>(rate, c.u[0][k], c.u[1][k], c.u[2][k], c.cut[k]);
    };
    int64_t t = 0;
    for (; t + kGatedSteps < A.T; t += kGatedSteps) {
        load(t);
        lane_states<DOCS, kGatedSteps>(A, so, ch, t, m, h);
        const Span own = sum_of<DOCS, false>([&](auto &sum) {
#pragma unroll
            for (int k = 0; k < kGatedSteps; ++k) sum.add(m[k]);
        });
        h = through<DOCS>(own, h);
    }
    if (t < A.T) {
        load(t);
        lane_states<DOCS, kGatedSteps>(A, so, ch, t, m, h);
    }
}
template <bool BF16, bool DOCS>
__global__ void __launch_bounds__(kWave) gated_channel_adjoint_kernel(GatedArgs A)
{
    const int64_t ch = (int64_t)blockIdx.x * kWave + threadIdx.x;
    if (ch >= A.channels) return;
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const float h0 = A.h0 ? A.h0[ch] : 0.0f;
    float w = A.gh_last ? A.gh_last[ch] : 0.0f, dlam = 0.0f;
    for (int64_t t = (A.T - 1) / kGatedSteps * kGatedSteps; t >= 0 && A.T > 0; t -= kGatedSteps) {
        const auto c = lane_steps<BF16, DOCS, kGatedSteps>(A, uo, b, t);
        const auto e = lane_back<kGatedSteps>(A, so, t, h0);
        Decay v[kGatedSteps];
#pragma unroll
        for (int k = 0; k < kGatedSteps; ++k) v[k] = decay(rate, c.u[0][k]);
        const float first = lane_gradients<BF16, kGatedSteps>(A, uo, t, c, e, v, w, dlam);
        if (t == 0) {
            w = first;
            break;
        }
        RunningBack<DOCS> own;
#pragma unroll
        for (int k = kGatedSteps - 1; k >= 0; --k) own.add(v[k], e.gh[k], c.cut[k], t + k < A.T);
        w = through<DOCS>(own.span(), w);
    }
    A.dlam_part[ch] = dlam;
    if (A.dh0) A.dh0[ch] = w;
}

// Else: a chunk of 64 steps of 64 channels a workgroup, 8 steps of each a wave.
// Every step is in registers once; the waves' maps meet in shared memory.
// 11x153600x64 time-major float32 468 us (3.7 TB/s), with documents 519;
// 8x4096x1024 bfloat16 115 us (2.9 TB/s), backward 254.  Bound by the registers
// that its single-element loads and their addresses take (2 workgroups a CU,
// backward 1), and with few channels by the steps of looking back: when these
// took 500 and 264 us, chunks of 128 steps took 447 of the first, but 313 of the
// backward pass; capped at 3 and 2 workgroups' registers it spilled and took 611
// and 261.
constexpr int kSpanWaves = 8, kSpanChunk = kSpanWaves * kGatedSteps;

// A lane: the state behind place - 1 > -1 of channel ch, from the words of the
// nearest kLookAhead predecessors, which are loaded together.
constexpr int kLookAhead = 6;
template <bool DOCS>
__device__ __forceinline__ float lane_look_back(const uint64_t *words, int64_t channels, int64_t ch,
                                                int64_t place)
{
    for (;;) {
        uint64_t h[kLookAhead], l[kLookAhead], b[kLookAhead];
#pragma unroll
        for (int j = 0; j < kLookAhead; ++j) {
            const uint64_t *r = words + max(place - 1 - j, int64_t(0)) * 3 * channels + ch;
            h[j] = published(r);
            if (j + 1 < kLookAhead) l[j] = published(r + channels), b[j] = published(r + 2 * channels);
        }
        bool found = false;
        float state = 0.0f;
#pragma unroll
        for (int j = kLookAhead - 1; j >= 0; --j) {
            if (place - 1 - j < 0) continue;
            if (h[j]) {
                found = true, state = word_value(h[j]);
            } else if (j + 1 < kLookAhead) {
                found = found && l[j] && b[j];
                state = through<DOCS>(span_of<DOCS>(word_value(l[j]), word_value(b[j])), state);
            }
        }
        if (found) return state;
        __builtin_amdgcn_s_sleep(1);
    }
}

// The chunk's place, the workgroup's channels, and after carry() the state
// before this wave's steps.
struct SpanPlace {
    int64_t place, ch;
    bool here;
    int wave, lane;
};
__device__ __forceinline__ SpanPlace span_place(const GatedArgs &A, uint32_t *ticket)
{
    const uint32_t groups = (uint32_t)((A.channels + kWave - 1) / kWave);
    const int64_t group = blockIdx.x % groups;
    SpanPlace s;
    s.place = A.words ? take_ticket(A, group, ticket) : 0;
    s.wave = threadIdx.x / kWave, s.lane = threadIdx.x % kWave;
    s.ch = group * kWave + s.lane;
    s.here = s.ch < A.channels;
    s.ch = min(s.ch, A.channels - 1);
    return s;
}
template <bool DOCS>
__device__ __forceinline__ float span_carry(const GatedArgs &A, const SpanPlace &s, const Span &own,
                                            float start, Span (*maps)[kWave], float *carry)
{
    maps[s.wave][s.lane] = own;
    __syncthreads();
    if (s.wave == 0 && A.words) {
        if (s.here) {
            const Span all = sum_of<DOCS, false>([&](auto &sum) {
#pragma unroll
                for (int w = 0; w < kSpanWaves; ++w) sum.add(maps[w][s.lane]);
            });
            uint64_t *r = A.words + s.place * 3 * A.channels + s.ch;
            if (s.place > 0) {
                publish(r + A.channels, all.l);
                publish(r + 2 * A.channels, all.b);
            }
            const float before =
                s.place > 0 ? lane_look_back<DOCS>(A.words, A.channels, s.ch, s.place) : start;
            publish(r, through<DOCS>(all, before));
            carry[s.lane] = before;
        }
    }
    __syncthreads();
    float h = A.words ? carry[s.lane] : start;
    for (int w = 0; w < s.wave; ++w) h = through<DOCS>(maps[w][s.lane], h);
    return h;
}

template <bool BF16, bool DOCS>
__global__ void __launch_bounds__(kSpanWaves * kWave) gated_span_kernel(GatedArgs A)
{
    __shared__ Span maps[kSpanWaves][kWave];
    __shared__ float carry[kWave];
    __shared__ uint32_t ticket;
    const SpanPlace s = span_place(A, &ticket);
    const int64_t b = s.ch / A.D, d = s.ch - b * A.D;
    const int64_t t = s.place * kSpanChunk + s.wave * kGatedSteps;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const auto c = lane_steps<BF16, DOCS, kGatedSteps>(A, uo, b, t);
    Span m[kGatedSteps];
#pragma unroll
    for (int k = 0; k < kGatedSteps; ++k)
        m[k] = forward_step<DOCS>(rate, c.u[0][k], c.u[1][k], c.u[2][k], c.cut[k]);
    const Span own = sum_of<DOCS, false>([&](auto &sum) {
#pragma unroll
        for (int k = 0; k < kGatedSteps; ++k) sum.add(m[k]);
    });
    const float h = span_carry<DOCS>(A, s, own, A.h0 ? A.h0[s.ch] : 0.0f, maps, carry);
    if (s.here) lane_states<DOCS, kGatedSteps>(A, so, s.ch, t, m, h);
}

// Backward: places and waves count from the end.
template <bool BF16, bool DOCS>
__global__ void __launch_bounds__(kSpanWaves * kWave) gated_span_adjoint_kernel(GatedArgs A)
{
    __shared__ Span maps[kSpanWaves][kWave];
    __shared__ float carry[kWave], sums[kSpanWaves][kWave];
    __shared__ uint32_t ticket;
    const SpanPlace s = span_place(A, &ticket);
    const int64_t b = s.ch / A.D, d = s.ch - b * A.D;
    const int64_t chunk = (A.T + kSpanChunk - 1) / kSpanChunk - 1 - s.place;
    const int64_t t = chunk * kSpanChunk + (kSpanWaves - 1 - s.wave) * kGatedSteps;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const auto c = lane_steps<BF16, DOCS, kGatedSteps>(A, uo, b, t);
    const auto e = lane_back<kGatedSteps>(A, so, t, A.h0 ? A.h0[s.ch] : 0.0f);
    Decay v[kGatedSteps];
    RunningBack<DOCS> own;
#pragma unroll
    for (int k = kGatedSteps - 1; k >= 0; --k) {
        v[k] = decay(rate, c.u[0][k]);
        own.add(v[k], e.gh[k], c.cut[k], t + k < A.T);
    }
    float w = span_carry<DOCS>(A, s, own.span(), A.gh_last ? A.gh_last[s.ch] : 0.0f, maps, carry), dlam = 0.0f;
    if (s.here) w = lane_gradients<BF16, kGatedSteps>(A, uo, t, c, e, v, w, dlam);
    sums[s.wave][s.lane] = dlam;
    __syncthreads();
    if (!s.here) return;
    if (A.dh0 && t == 0) A.dh0[s.ch] = w;
    if (s.wave != 0) return;
    for (int j = 1; j < kSpanWaves; ++j) dlam += sums[j][s.lane];
    A.dlam_part[s.place * A.channels + s.ch] = dlam;
}

// ---------------------------------------------------------- lanes in time ---
// Time-contiguous planes: a channel's steps side by side in the lanes of W
// waves, K steps a lane, so that every load and store of a wave is one
// contiguous run.  Per chunk of 64 K W steps a lane composes its own steps,
// the wave scans the lanes' maps (DPP), W > 1 waves exchange their totals
// through LDS (one barrier a chunk, two buffers), and every lane runs its
// steps again from the state in front of them.  The chunk's last state starts
// the next one; the next chunk's loads are issued before this one's scan.
// Bound by HBM: every plane goes once, 4x16384x4096 bfloat16 510 us (5.3 TB/s,
// a large copy's rate), backward 8x4096x1024 bfloat16 129 us (5.2 TB/s), with
// documents 138 (the steps take more operations, and registers allow 3 waves a
// SIMD); a lane per channel took 19.8 ms and 5.0 ms of these.
template <int K, bool BF16>
struct GatedChunk {
    Raw<BF16, K> u[3];
    uint32_t cut;
};
template <int K, bool BF16, bool DOCS>
__device__ __forceinline__ GatedChunk<K, BF16> load_chunk(const GatedArgs &A, int64_t uo, int64_t b,
                                                          int64_t t, int64_t t1)
{
    GatedChunk<K, BF16> c;
#pragma unroll
    for (int g = 0; g < 3; ++g) c.u[g] = load_raw<BF16, K>(A.u[g], uo, t, t1);
    c.cut = DOCS ? load_flags<K>(A.resets + b * A.T, t, t1) : 0u;
    return c;
}

// The state before wave `wave`'s part of the chunk, from the one before the
// chunk and the waves' maps in order; `carry` moves on to the next chunk.
template <bool DOCS, int W>
__device__ __forceinline__ float through_waves(const Span *maps, int wave, float &carry)
{
    float mine = carry;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w == wave) mine = carry;
        carry = through<DOCS>(maps[w], carry);
    }
    return mine;
}
template <bool DOCS, int W>
__device__ __forceinline__ Span all_waves(const Span *maps)
{
    return sum_of<DOCS, true>([&](auto &sum) {
#pragma unroll
        for (int w = 0; w < W; ++w) sum.add(maps[w]);
    });
}

// A lane's steps, and the span they make.
template <int K, bool BF16, bool DOCS>
__device__ __forceinline__ Span chunk_maps(const GatedChunk<K, BF16> &c, float rate, Span (&m)[K])
{
#pragma unroll
    for (int k = 0; k < K; ++k)
        m[k] = forward_step<DOCS>(rate, c.u[0].get(k), c.u[1].get(k), c.u[2].get(k), c.cut >> k & 1u);
    return sum_of<DOCS, true>([&](auto &sum) {
#pragma unroll
        for (int k = 0; k < K; ++k) sum.add(m[k]);
    });
}
// The wave's lanes up to each one, from its lanes' spans: products of at most 64
// decays, good for the states within the wave.  And its whole span (in the last
// lane), which goes on to the steps behind it.
__device__ __forceinline__ Map1 careful_scan(Map1 x)
{
    x = joined<true>(x, dpp_map<0x111>(x));
    x = joined<true>(x, dpp_map<0x112>(x));
    x = joined<true>(x, dpp_map<0x114>(x));
    x = joined<true>(x, dpp_map<0x118>(x));
    x = joined<true>(x, dpp_map<0x142, 0xA>(x));
    return joined<true>(x, dpp_map<0x143, 0xC>(x));
}
template <bool DOCS>
struct WaveSpans {
    Map1 upto;
    Span all;
    uint64_t cuts = 0;  // the cut lanes (a product of two -0 is +0)
    __device__ __forceinline__ explicit WaveSpans(const Span &own)
    {
        const Map1 x = {own.a, own.b};
        if constexpr (DOCS) cuts = __ballot(is_cut<DOCS>(own.a));
        upto = wave_scan_inclusive(x);
        if (DOCS && any_not_finite(upto.b)) upto = careful_scan(x);
        // (a NaN in front of a cut is in the sum)
        const float l = wave_sum_to_last(own.l);
        all = span_of<DOCS>(cuts ? kNoMemory : l, upto.b);
    }
    // the state, or w, before the lane's steps
    __device__ __forceinline__ float before_lane(float before_wave) const
    {
        const Map1 x = wave_shift_up(upto);
        if (DOCS && any_not_finite(before_wave) &&
            __builtin_amdgcn_mbcnt_hi((uint32_t)(cuts >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)cuts, 0u)))
            return x.b;
        return through<false>(x, before_wave);
    }
    // behind the wave's
    __device__ __forceinline__ float behind(float before_wave) const
    {
        return through<DOCS>(Map1{read_lane(all.a, kWave - 1), read_lane(all.b, kWave - 1)},
                             before_wave);
    }
};

// A lane's states from the one before them.
template <bool DOCS, int K>
__device__ __forceinline__ void chunk_states(const GatedArgs &A, int64_t so, int64_t ch, int64_t t,
                                             const Span (&m)[K], float h)
{
    float out[K], last = h;
#pragma unroll
    for (int k = 0; k < K; ++k) out[k] = last = through<false>(m[k], last);
    if constexpr (DOCS) {
        if (any_not_finite(last)) {
            last = h;
#pragma unroll
            for (int k = 0; k < K; ++k) out[k] = last = through<true>(m[k], last);
        }
    }
    if (t >= A.T) return;
    store_raw<false, K>(A.h, so, t, A.T, out);
    if (A.h_last && t + K >= A.T)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t + k == A.T - 1) A.h_last[ch] = out[k];
}

// Every channel's steps one chunk after the other, in one workgroup.
template <bool BF16, bool DOCS, int K, int W>
__global__ void __launch_bounds__(W * kWave) gated_time_kernel(GatedArgs A)
{
    __shared__ Span maps[2][W];
    const int64_t ch = blockIdx.x;
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const int wave = threadIdx.x / kWave;
    constexpr int P = K * W * kWave;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    float carry = A.h0 ? A.h0[ch] : 0.0f;
    int64_t t = (int64_t)threadIdx.x * K;
    GatedChunk<K, BF16> now = load_chunk<K, BF16, DOCS>(A, uo, b, t, A.T);
    int parity = 0;
    for (int64_t c = 0; c < A.T; c += P, t += P, parity ^= 1) {
        GatedChunk<K, BF16> next;
        if (c + P < A.T) next = load_chunk<K, BF16, DOCS>(A, uo, b, t + P, A.T);
        Span m[K];
        const WaveSpans<DOCS> spans(chunk_maps<K, BF16, DOCS>(now, rate, m));
        float before = carry;
        if constexpr (W > 1) {
            if (threadIdx.x % kWave == kWave - 1) maps[parity][wave] = spans.all;
            __syncthreads();
            before = through_waves<DOCS, W>(maps[parity], wave, carry);
        }
        chunk_states<DOCS, K>(A, so, ch, t, m, spans.before_lane(before));
        if constexpr (W == 1) carry = spans.behind(carry);
        now = next;
    }
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
template <int K, bool BF16, bool DOCS>
__device__ __forceinline__ GatedBackChunk<K, BF16> load_back(const GatedArgs &A, int64_t uo,
                                                             int64_t so, int64_t b,
                                                             int64_t t, int64_t first, int64_t end,
                                                             float h0)
{
    GatedBackChunk<K, BF16> c;
#pragma unroll
    for (int g = 0; g < 3; ++g) c.u[g] = load_raw<BF16, K>(A.u[g], uo, t, end);
    c.h = load_raw<false, K>(A.hs, so, t, end);
    c.before = first > 0 && first <= A.T ? A.hs[so + first - 1] : h0;
    if (A.gh) {
        c.gh = load_raw<false, K>(A.gh, so, t, end);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) c.gh.w[k] = 0u;
    }
    c.cut = DOCS ? load_flags<K>(A.resets + b * A.T, t, end) : 0u;
    return c;
}
template <int K, bool BF16, bool DOCS>
__device__ __forceinline__ Span back_maps(const GatedBackChunk<K, BF16> &c, float rate, int64_t t,
                                          int64_t end, Decay (&v)[K])
{
    RunningBack<DOCS> own;
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        v[k] = decay(rate, c.u[0].get(k));
        own.add(v[k], c.gh.get(k), c.cut >> k & 1u, t + k < end);
    }
    return own.span();
}
// A lane's gradients from the w behind them and the state before its first
// step; returns its own w, and adds to dlam.
template <int K, bool BF16>
__device__ __forceinline__ float chunk_gradients(const GatedArgs &A, int64_t uo, int64_t t,
                                                 int64_t end, const GatedBackChunk<K, BF16> &c,
                                                 const Decay (&v)[K], float w, float hp,
                                                 float &dlam)
{
    float gr[K], gi[K], gx[K];
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
        const bool cut = c.cut >> k & 1u, in = t + k < end;
        const float G = c.gh.get(k) + w;
        const GatedGrad g = gated_grad(v[k], c.u[1].get(k), c.u[2].get(k), cut, G,
                                       k ? c.h.get(k ? k - 1 : 0) : hp);
        gr[k] = g.r, gi[k] = g.i, gx[k] = g.x;
        dlam += in ? g.lam : 0.0f;
        w = in ? (cut ? 0.0f : v[k].a * G) : w;
    }
    if (t >= end) return w;
    store_raw<BF16, K>(A.du[0], uo, t, end, gr);
    store_raw<BF16, K>(A.du[1], uo, t, end, gi);
    store_raw<BF16, K>(A.du[2], uo, t, end, gx);
    return w;
}
// The workgroup's sum of dlam, in its last thread.
template <int W>
__device__ __forceinline__ float dlam_sum(float dlam, float *lds)
{
    float s = wave_sum_to_last(dlam);
    if constexpr (W > 1) {
        if (threadIdx.x % kWave == kWave - 1) lds[threadIdx.x / kWave] = s;
        __syncthreads();
        s = 0.0f;
        for (int w = 0; w < W; ++w) s += lds[w];
    }
    return s;
}

template <bool BF16, bool DOCS, int K, int W>
__global__ void __launch_bounds__(W * kWave) gated_time_adjoint_kernel(GatedArgs A)
{
    __shared__ Span maps[2][W];
    __shared__ float sums[W];
    const int64_t ch = blockIdx.x;
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const int wave = threadIdx.x / kWave;
    constexpr int P = K * W * kWave;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    float carry = A.gh_last ? A.gh_last[ch] : 0.0f, dlam = 0.0f;
    const float h0 = A.h0 ? A.h0[ch] : 0.0f;
    int64_t c = (A.T - 1) / P * P;  // the last chunk
    const int at = W * kWave - 1 - (int)threadIdx.x, wave_at = (W - 1 - wave) * kWave;
    GatedBackChunk<K, BF16> now =
        load_back<K, BF16, DOCS>(A, uo, so, b, c + at * K, c + wave_at * K, A.T, h0);
    int parity = 0;
    for (; c >= 0; c -= P, parity ^= 1) {
        const int64_t t = c + at * K;
        GatedBackChunk<K, BF16> next;
        if (c > 0) next = load_back<K, BF16, DOCS>(A, uo, so, b, t - P, c - P + wave_at * K, A.T, h0);
        Decay v[K];
        const WaveSpans<DOCS> spans(back_maps<K, BF16, DOCS>(now, rate, t, A.T, v));
        float after = carry;
        if constexpr (W > 1) {
            if (threadIdx.x % kWave == kWave - 1) maps[parity][wave] = spans.all;
            __syncthreads();
            after = through_waves<DOCS, W>(maps[parity], wave, carry);
        }
        // the state before the lane's first step: the next lane's last one
        float hp = __shfl_down(now.h.get(K - 1), 1);
        if (threadIdx.x % kWave == kWave - 1) hp = now.before;
        const float w = chunk_gradients<K, BF16>(A, uo, t, A.T, now, v,
                                                 spans.before_lane(after), hp, dlam);
        if constexpr (W == 1) carry = spans.behind(carry);
        if (A.dh0 && t == 0) A.dh0[ch] = w;
        now = next;
    }
    const float s = dlam_sum<W>(dlam, sums);
    if (threadIdx.x == W * kWave - 1) A.dlam_part[ch] = s;
}

// ------------------------------------------------ lanes in time, look back ---
// Few channels: a channel's chunks run side by side, each in a workgroup of its
// own.  A wave looks back over 64 predecessors, a lane each.  1x262144x64
// float32 72 us from HBM (3.7 TB/s; 60 where part of it is still cached),
// backward 124.  Bound by the time a chunk waits for its loads and then for its
// predecessor, with 4 chunks a CU.
struct GatedRecord {
    uint64_t l, b;  // the chunk's map
    uint64_t h;     // the state behind the chunk
    uint64_t unused;
};
// A wave: the state behind place - 1 > -1 of channel ch.
template <bool DOCS>
__device__ __forceinline__ float look_back(const GatedRecord *records, int64_t channels, int64_t ch,
                                           int64_t place)
{
    const int64_t at = place - 1 - threadIdx.x % kWave;
    const GatedRecord *r = records + max(at, int64_t(0)) * channels + ch;
    for (;;) {
        const uint64_t h = published(&r->h), l = published(&r->l), b = published(&r->b);
        // up to the nearest state, every lane has to be ready
        const uint64_t states = __ballot(h != 0), ready = __ballot(l != 0 && b != 0);
        const uint64_t nearer = (states & -states) - 1;
        if (states && (ready & nearer) == nearer) {
            int lane = __ffsll((unsigned long long)states) - 1;
            float state = read_lane(word_value(h), lane);
            const Span m = span_of<DOCS>(word_value(l), word_value(b));
            while (--lane >= 0)
                state = through<DOCS>(Map1{read_lane(m.a, lane), read_lane(m.b, lane)}, state);
            return state;
        }
        __builtin_amdgcn_s_sleep(1);
    }
}

// Publishes the chunk's map and state and returns the state before the chunk,
// in every thread.
template <bool DOCS, int W>
__device__ __forceinline__ float chunk_carry(const GatedArgs &A, const Span *maps, int64_t ch,
                                             int64_t place, float start, float *lds)
{
    if (threadIdx.x < kWave) {
        GatedRecord *r = A.records + place * A.channels + ch;
        const Span all = all_waves<DOCS, W>(maps);
        if (place > 0 && threadIdx.x == 0) {
            publish(&r->l, all.l);
            publish(&r->b, all.b);
        }
        const float before = place > 0 ? look_back<DOCS>(A.records, A.channels, ch, place) : start;
        if (threadIdx.x == 0) {
            publish(&r->h, through<DOCS>(all, before));
            *lds = before;
        }
    }
    __syncthreads();
    return *lds;
}

template <bool BF16, bool DOCS, int K, int W>
__global__ void __launch_bounds__(W * kWave) gated_look_kernel(GatedArgs A)
{
    __shared__ Span maps[W];
    __shared__ uint32_t ticket;
    __shared__ float carry_lds;
    const int64_t ch = blockIdx.x % (uint32_t)A.channels;
    const int64_t place = take_ticket(A, ch, &ticket);
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const int wave = threadIdx.x / kWave;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const int64_t t = place * (K * W * kWave) + (int64_t)threadIdx.x * K;
    const GatedChunk<K, BF16> c = load_chunk<K, BF16, DOCS>(A, uo, b, t, A.T);
    Span m[K];
    const WaveSpans<DOCS> spans(chunk_maps<K, BF16, DOCS>(c, rate, m));
    if (threadIdx.x % kWave == kWave - 1) maps[wave] = spans.all;
    __syncthreads();
    float carry = chunk_carry<DOCS, W>(A, maps, ch, place, A.h0 ? A.h0[ch] : 0.0f, &carry_lds);
    const float before = through_waves<DOCS, W>(maps, wave, carry);
    chunk_states<DOCS, K>(A, so, ch, t, m, spans.before_lane(before));
}

template <bool BF16, bool DOCS, int K, int W>
__global__ void __launch_bounds__(W * kWave) gated_look_adjoint_kernel(GatedArgs A)
{
    __shared__ Span maps[W];
    __shared__ float sums[W];
    __shared__ uint32_t ticket;
    __shared__ float carry_lds;
    const int64_t ch = blockIdx.x % (uint32_t)A.channels;
    const int64_t place = take_ticket(A, ch, &ticket);
    const int64_t b = ch / A.D, d = ch - b * A.D;
    const int wave = threadIdx.x / kWave;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const float h0 = A.h0 ? A.h0[ch] : 0.0f;
    constexpr int P = K * W * kWave;
    const int64_t c0 = ((A.T + P - 1) / P - 1 - place) * P;  // places count from the end
    const int at = W * kWave - 1 - (int)threadIdx.x;
    const int64_t t = c0 + at * K;
    const GatedBackChunk<K, BF16> c =
        load_back<K, BF16, DOCS>(A, uo, so, b, t, c0 + (W - 1 - wave) * (kWave * K), A.T, h0);
    Decay v[K];
    const WaveSpans<DOCS> spans(back_maps<K, BF16, DOCS>(c, rate, t, A.T, v));
    if (threadIdx.x % kWave == kWave - 1) maps[wave] = spans.all;
    __syncthreads();
    float carry = chunk_carry<DOCS, W>(A, maps, ch, place, A.gh_last ? A.gh_last[ch] : 0.0f, &carry_lds);
    const float after = through_waves<DOCS, W>(maps, wave, carry);
    float hp = __shfl_down(c.h.get(K - 1), 1), dlam = 0.0f;
    if (threadIdx.x % kWave == kWave - 1) hp = c.before;
    const float w = chunk_gradients<K, BF16>(A, uo, t, A.T, c, v, spans.before_lane(after), hp,
                                             dlam);
    if (A.dh0 && t == 0) A.dh0[ch] = w;
    const float s = dlam_sum<W>(dlam, sums);
    if (threadIdx.x == W * kWave - 1) A.dlam_part[place * A.channels + ch] = s;
}

// --------------------------------------------------- lanes in time, short ---
// At most G K steps: G lanes a channel and 64 / G channels a wave, each lane's
// K steps in one access as above.  (With a wave a channel, T = 100 of 64000
// channels left 7 of 8 lanes idle: 64x100x1000 bfloat16 100 us, here 27;
// 64x32x1024 float32 43 and 14.)  Bound by partial lines of odd lengths and by
// the launch.
constexpr int kShortThreads = 256;

// Inclusive scan of the maps over groups of G neighbouring lanes, each group's
// first lane first (its last, REVERSE); then the map in front of the lane's own.
template <bool CAREFUL, int G, bool REVERSE>
__device__ __forceinline__ Map1 group_scan(Map1 x)
{
    const int lane = threadIdx.x % G, at = REVERSE ? G - 1 - lane : lane;
#pragma unroll
    for (int o = 1; o < G; o *= 2) {
        const Map1 y = REVERSE ? Map1{__shfl_down(x.a, o), __shfl_down(x.b, o)}
                               : Map1{__shfl_up(x.a, o), __shfl_up(x.b, o)};
        if (at >= o) x = joined<CAREFUL>(x, y);
    }
    return x;
}
// `start` through the group's spans in front of the lane's own.
template <bool DOCS, int G, bool REVERSE>
__device__ __forceinline__ float before_lane(const Span &own, float start)
{
    const int lane = threadIdx.x % G, at = REVERSE ? G - 1 - lane : lane;
    Map1 x = group_scan<false, G, REVERSE>(Map1{own.a, own.b});
    if (DOCS && any_not_finite(x.b)) x = group_scan<true, G, REVERSE>(Map1{own.a, own.b});
    const uint64_t wave_cuts = DOCS ? __ballot(is_cut<DOCS>(own.a)) : 0;
    const Map1 y = REVERSE ? Map1{__shfl_down(x.a, 1), __shfl_down(x.b, 1)}
                           : Map1{__shfl_up(x.a, 1), __shfl_up(x.b, 1)};
    if (at == 0) return start;
    if constexpr (DOCS) {
        // the group's cut lanes, and those in front of this one
        const uint32_t cuts = (uint32_t)(wave_cuts >> (threadIdx.x % kWave - lane)) & ((1u << G) - 1);
        if (REVERSE ? cuts >> (lane + 1) : cuts & ((1u << lane) - 1))
            if (!(fabsf(start) < __builtin_inff())) return y.b;
    }
    return through<false>(y, start);
}

template <bool BF16, bool DOCS, int K, int G>
__global__ void __launch_bounds__(kShortThreads) gated_short_kernel(GatedArgs A)
{
    const int64_t ch = ((int64_t)blockIdx.x * kShortThreads + threadIdx.x) / G;
    const bool here = ch < A.channels;  // the others follow along for the shuffles
    const int64_t b = here ? ch / A.D : 0, d = here ? ch - b * A.D : 0;
    const int64_t t = (int64_t)(threadIdx.x % G) * K, end = here ? A.T : 0;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const GatedChunk<K, BF16> c = load_chunk<K, BF16, DOCS>(A, uo, b, t, end);
    const float h0 = A.h0 && here ? A.h0[ch] : 0.0f;
    Span m[K];
    const float h = before_lane<DOCS, G, false>(chunk_maps<K, BF16, DOCS>(c, rate, m), h0);
    if (here) chunk_states<DOCS, K>(A, so, ch, t, m, h);
}

template <bool BF16, bool DOCS, int K, int G>
__global__ void __launch_bounds__(kShortThreads) gated_short_adjoint_kernel(GatedArgs A)
{
    const int64_t ch = ((int64_t)blockIdx.x * kShortThreads + threadIdx.x) / G;
    const bool here = ch < A.channels;
    const int64_t b = here ? ch / A.D : 0, d = here ? ch - b * A.D : 0;
    const int64_t t = (int64_t)(threadIdx.x % G) * K, end = here ? A.T : 0;
    const float rate = decay_rate(A.lam[d], A.power);
    const int64_t uo = b * A.usb + d * A.usd, so = b * A.ssb + d * A.ssd;
    const float h0 = A.h0 && here ? A.h0[ch] : 0.0f;
    const GatedBackChunk<K, BF16> c = load_back<K, BF16, DOCS>(A, uo, so, b, t, 0, end, h0);
    const float after = A.gh_last && here ? A.gh_last[ch] : 0.0f;
    Decay v[K];
    const float behind = before_lane<DOCS, G, true>(back_maps<K, BF16, DOCS>(c, rate, t, end, v), after);
    float hp = __shfl_up(c.h.get(K - 1), 1), dlam = 0.0f;
    if (threadIdx.x % G == 0) hp = h0;
    const float w = chunk_gradients<K, BF16>(A, uo, t, end, c, v, behind, hp,
                                             dlam);
#pragma unroll
    for (int o = 1; o < G; o *= 2) dlam += __shfl_xor(dlam, o);
    if (t > 0 || !here) return;
    if (A.dh0) A.dh0[ch] = w;
    A.dlam_part[b * A.D + d] = dlam;  // one span
}

// dL/dlam = -power sig(lam) sum (dL/dl sig(u_r)): 64 channels a workgroup, its
// waves each a contiguous run of the partial sums' rows; a fixed order.  Bound
// by latency: a wave has 4 rows of loads in flight.
constexpr int kDlamWaves = 8;
__global__ void __launch_bounds__(kDlamWaves * kWave) gated_dlam_kernel(GatedArgs A, int64_t rows)
{
    __shared__ float lds[kDlamWaves][kWave];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int64_t d = (int64_t)blockIdx.x * kWave + lane;
    const int64_t per = (rows + kDlamWaves - 1) / kDlamWaves;
    float s = 0.0f;
    if (d < A.D)
#pragma unroll 4
        for (int64_t j = wave * per; j < min(rows, (wave + 1) * per); ++j)
            s += A.dlam_part[j * A.D + d];
    lds[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || d >= A.D) return;
    for (int w = 1; w < kDlamWaves; ++w) s += lds[w][lane];
    A.dlam[d] = -A.power * sigmoid_q(-kLog2e * A.lam[d]) * s;
}

// ----------------------------------------------------------- one step ---
// A lane per channel of a request, its state read and written in its slot of
// the pool; no scan.  64 requests x 1024 channels: 3 us on the device, the
// launch's own time; the call itself takes 9.
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
        const Span m = forward_step<false>(decay_rate(A.lam[d], A.power), load_gate<BF16>(A.u[0], o),
                                 load_gate<BF16>(A.u[1], o), load_gate<BF16>(A.u[2], o), false);
        float *s = A.states + slot * A.D + d;
        const float h = through<false>(m, *s);
        *s = h;
        A.out[b * A.D + d] = h;
    }
}

}  // namespace pararnn
