"""Bounds for every element of the operators' results, from the oracle's formulas
with the roundings carried along.  u = 2^-24, half an ulp of 1 in float32.

Gated recurrence.  A log decay is a product of two numbers of under 8 roundings,
so a decay a = exp(l) is within (8 |l| + 4) u of itself; 1 - a^2 holds relative
precision, and with its root, two sigmoids and the products an input term b is
within 24 u |b|.  With S the same recurrence of the magnitudes, one step brings
the state's error from E to
    a (E + (8 |l| + 8) u S) + 24 u |b| + 2 u S,
and the levels at which spans are joined (under 32, two roundings each) add
64 u S once.  Backwards the same holds for G; the local factors of the
gradients, their differences term by term, follow.  A sum has a rounding of the
sum of its magnitudes for each addition on the longest path.

Scores.  The sum of exponentials is within (V / 256 + 32) u of itself, lse has
roundings of its own size besides; p = exp(x - lse) carries lse's error and
(4 |log p| + 16) u; the gradient is p times coefficients, the token's own
besides."""
import numpy as np

from oracle import language as ref

U = 2.0 ** -24
BF16_HALF_ULP = 2.0 ** -8 * 1.01  # of the value: 8 significant bits
TINY = 1e-36  # float32 has no numbers of full precision below


def bf16(x):
    """float64 values rounded to bfloat16, nearest even."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def scan_inputs(B, T, D, half, docs, with_h0, seed=0, power=8.0):
    """Inputs that their types hold, as float64."""
    r = np.random.default_rng(seed + 1000 * T + D)
    kind = bf16 if half else lambda x: np.float32(x).astype(np.float64)

    def f32(x):
        return np.float32(x).astype(np.float64)
    decay = 0.9 + 0.099 * r.random(D)
    return dict(u=[kind(r.standard_normal((B, D, T))) for _ in range(3)],
                lam=f32(np.log(np.expm1(-np.log(decay) / power))), power=power,
                h0=f32(r.standard_normal((B, D))) if with_h0 else None,
                resets=r.random((B, T)) < docs if docs else None,
                gh=f32(r.standard_normal((B, D, T))), gl=f32(r.standard_normal((B, D))))


def _local(c):
    """l, a, gain, sig(u_i), sig(u_r), kept decays."""
    l, q = ref._log_decay(c["u"][0], c["lam"], c["power"])
    a, gain, si = np.exp(l), np.sqrt(-np.expm1(2 * l)), ref._sig(c["u"][1])
    kept = a if c["resets"] is None else np.where(c["resets"][:, None, :], 0.0, a)
    return l, q, a, gain, si, kept


def _recur(kept, l, add, start):
    """Magnitudes S and errors E of x_t = kept_t x_{t-1} + add_t, add_t within 24 u."""
    S, E = np.empty_like(kept), np.empty_like(kept)
    s, e = np.abs(start), np.zeros_like(start)
    for t in range(kept.shape[-1]):
        k, b = kept[..., t], np.abs(add[..., t])
        e = k * (e + U * (8 * np.abs(l[..., t]) + 8) * s) + 24 * U * b
        s = k * s + b
        e = e + 2 * U * s
        S[..., t], E[..., t] = s, e
    return S, E + 64 * U * S


def scan(c):
    """(h, its bound)."""
    l, _, _, gain, si, kept = _local(c)
    h = ref.gated_scan(c["u"], c["lam"], c["h0"], c["power"], c["resets"])
    h0 = np.zeros(kept.shape[:2]) if c["h0"] is None else c["h0"]
    return h, _recur(kept, l, gain * si * c["u"][2], h0)[1] + TINY


def additions(B, T, D, layout):
    """Additions on the longest path of a sum over a channel's steps and the batch."""
    lanes = T if layout != "channel" and (T <= 64 or B * D >= 65536) else T // 32
    return 64 + lanes + B * (1 + T // 512)


def scan_adjoint(c, h, layout="channel", half=False):
    """(results, their bounds) for the states h that the kernel is given."""
    want = ref.gated_scan_adjoint(c["u"], c["lam"], c["h0"], h, c["gh"], c["power"], c["resets"], c["gl"])
    l, q, a, gain, si, kept = _local(c)
    B, D, T = kept.shape
    x = c["u"][2]
    # G_t = gh_t + kept_{t+1} G_{t+1}, G_T = gh_T + gl: the last factor is that of step t + 1
    after, l_after = np.zeros_like(kept), np.zeros_like(kept)
    after[..., :-1], l_after[..., :-1] = kept[..., 1:], l[..., 1:]
    add = c["gh"].copy()
    add[..., -1] += c["gl"]
    G = np.empty_like(kept)
    g = np.zeros((B, D))
    for t in range(T - 1, -1, -1):
        g = G[..., t] = add[..., t] + after[..., t] * g
    SG, EG = (v[..., ::-1] for v in _recur(after[..., ::-1], l_after[..., ::-1], add[..., ::-1], np.zeros((B, D))))
    before = np.empty_like(h)
    before[..., 0], before[..., 1:] = 0.0 if c["h0"] is None else c["h0"], h[..., :-1]
    one = kept * before
    two = np.divide(a * a, gain, out=np.zeros_like(gain), where=gain > 1e-15) * si * x
    al, G_, one_, two_ = np.abs(l), np.abs(G), np.abs(one), np.abs(two)
    dl = G * (one - two)
    tol_dl = EG * np.abs(one - two) + G_ * U * ((8 * al + 8) * one_ + (16 * al + 40) * two_)
    ux = G * gain * si
    tol_x = EG * gain * si + 40 * U * np.abs(ux)
    tol_i = tol_x * np.abs(x) * (1 - si) + np.abs(ux * x) * U * (16 * (1 - si) + 4)
    tol_r = tol_dl * al * (1 - q) + np.abs(dl) * al * U * (24 * (1 - q) + 4)
    tol = dict(du=[tol_r, tol_i, tol_x])
    if half:
        tol["du"] = [t + BF16_HALF_ULP * (np.abs(v) + t) for t, v in zip(tol["du"], want["du"])]
    tol["du"] = [t + TINY for t in tol["du"]]
    tol["dh0"] = kept[..., 0] * (EG[..., 0] + U * (8 * al[..., 0] + 8) * SG[..., 0]) + TINY
    factor = c["power"] * ref._sig(c["lam"])
    terms = np.abs(dl * q)
    errors = (tol_dl * q + 16 * U * terms).sum((0, 2))
    tol["dlam"] = factor * (errors + U * additions(B, T, D, layout) * terms.sum((0, 2))) + 16 * U * np.abs(want["dlam"])
    return want, tol


def score_inputs(N, V, half, masked=0.0, seed=0):
    r = np.random.default_rng(seed + 31 * N + V)
    x = 3 * r.standard_normal((N, V)) + 2 * r.standard_normal((N, 1))
    x = bf16(x) if half else np.float32(x).astype(np.float64)
    x[r.random((N, V)) < masked] = -np.inf
    tokens = r.integers(0, V, N)
    if N > 2:
        tokens[1] = -1
    g = [np.float32(r.standard_normal(N)).astype(np.float64) for _ in range(3)]
    return dict(x=x, tokens=tokens, g=g)


def score_adjoint(c, scale=1.0, half=False):
    """(gradient, its bound); g: of logprob, entropy and lse.  The lse and the
    entropy are the forward pass's, with its errors."""
    x, tokens, (g_lp, g_h, g_lse) = c["x"], c["tokens"], c["g"]
    N, V = x.shape
    s = ref.token_logprobs(x, tokens, 0, scale)
    want = ref.token_logprobs_adjoint(x, tokens, g_lp, g_h, g_lse, scale)
    live = np.isfinite(s["lse"])
    lse = np.where(live, s["lse"], 0.0)[:, None]
    lp = np.where(np.isfinite(x) & live[:, None], scale * np.where(np.isfinite(x), x, 0.0) - lse, -np.inf)
    p = np.exp(lp)
    lp = np.where(p > 0, lp, 0.0)
    base = U * (V / 256 + 32)
    error_lse = base + 4 * U * (np.abs(lse) + 64)
    error_lp = error_lse + 4 * U * np.abs(lp)
    error_h = 2 * base + 4 * U * 64
    glp, gh, gl = (np.abs(v)[:, None] for v in (np.where(tokens >= 0, g_lp, 0.0), g_h, g_lse))
    H = s["entropy"][:, None]
    tol = scale * p * ((glp + gl + gh * np.abs(lp + H)) * (error_lp + 20 * U) + gh * (error_lp + error_h))
    scored = (tokens >= 0) & live
    tol[scored, tokens[scored]] += scale * np.abs(g_lp[scored]) * 4 * U
    tol = tol + TINY * (1 + scale * (glp + gl + gh * 128))
    return want, tol + (BF16_HALF_ULP * (np.abs(want) + tol) if half else 0.0)


def outside(got, want, tol):
    """Elements that are out of their bound."""
    return ~(np.abs(np.asarray(got, np.float64) - want) <= tol)
