"""The bounds of language_bounds.py hold and can fail, on the CPU: at every size
the GPU tests use them at, a float32 evaluation is inside, and results of zeros, results with
a piece missing and gradients without one of their terms are outside."""
import numpy as np
import pytest

from oracle import language as ref
from tests import language_bounds as lb
from tests.language_bounds import outside

SCANS = [(1, 1, 1, "channel"), (2, 1, 130, "time"), (1, 2, 3, "channel"), (3, 7, 65, "channel"), (2, 17, 33, "time"),
         (2, 64, 64, "channel"), (1, 65, 2, "channel"), (2, 128, 21, "channel"), (2, 300, 33, "channel"),
         (5, 129, 200, "channel"), (1, 513, 9, "channel"), (2, 1025, 3, "time"), (1, 4100, 2, "channel"),
         (3, 12289, 5, "channel"), (1, 4097, 300, "channel"), (1, 30000, 70, "time"), (3, 65, 130, "time"),
         (1, 600, 2100, "channel"), (1, 4200, 2049, "channel"), (1, 20011, 1, "channel")]
SCORES = [(1, 1, 0.0), (3, 2, 0.0), (5, 64, 0.3), (4, 257, 0.0), (2, 4097, 0.9), (3, 1000, 0.0), (2, 70001, 0.0),
          (2, 131072, 0.3), (300, 129, 0.0)]


# (both types at sizes that take little; the largest in float32)
TYPED_SCANS = [c + (half,) for c in SCANS for half in (False, True) if not half or c[0] * c[1] * c[2] <= 500_000]


def scan_case(B, T, D, half=False):
    return lb.scan_inputs(B, T, D, half, 0.02 if D % 2 else None, D != 5)


def scan_f32(c):
    """The recurrence step by step in float32."""
    f = np.float32
    ur, ui, ux = (p.astype(f) for p in c["u"])
    lam = c["lam"].astype(f)
    soft = np.log1p(np.exp(lam))
    l = -f(c["power"]) * soft[None, :, None] / (1 + np.exp(-ur))
    a, b = np.exp(l), np.sqrt(-np.expm1(2 * l)) / (1 + np.exp(-ui)) * ux
    if c["resets"] is not None:
        a = np.where(c["resets"][:, None, :], f(0), a)
    h = np.zeros(a.shape[:2], f) if c["h0"] is None else c["h0"].astype(f)
    out = np.empty_like(a)
    for t in range(a.shape[-1]):
        h = out[..., t] = a[..., t] * h + b[..., t]
    return out


@pytest.mark.parametrize("B,T,D,layout,half", TYPED_SCANS)
def test_scan_bounds(B, T, D, layout, half):
    c = scan_case(B, T, D, half)
    h, tol = lb.scan(c)
    got = scan_f32(c)
    assert not outside(got, h, tol).any()
    assert outside(0 * h, h, tol).mean() > 0.95
    span = max(1, min(T, 64))  # the last chunk of one channel, and a state carried over it lost
    for piece in (slice(T - 1, T), slice(T - span, T)):
        bad = got.copy()
        bad[-1, -1, piece] = 0
        assert outside(bad, h, tol).any()
    if T > 1 and c["resets"] is None:  # the state before the last half does not reach it
        half_way = dict(c, u=[p[..., T // 2:] for p in c["u"]], h0=None)
        bad = got.copy()
        bad[..., T // 2:] = ref.gated_scan(half_way["u"], c["lam"], None, c["power"])
        assert outside(bad, h, tol).any()


@pytest.mark.parametrize("B,T,D,layout,half", TYPED_SCANS)
def test_scan_adjoint_bounds(B, T, D, layout, half):
    c = scan_case(B, T, D, half)
    h = scan_f32(c).astype(np.float64)
    want, tol = lb.scan_adjoint(c, h, layout, half)
    flat = [(want["du"][g], tol["du"][g]) for g in range(3)] + [(want[k], tol[k]) for k in ("dh0", "dlam")]
    for i, (w, t) in enumerate(flat):
        assert np.isfinite(t).all() and (t >= 0).all()
        live = np.abs(w) > 1e-30  # dh0 of a channel whose first step is a reset is 0
        if live.any():
            assert outside(0 * w, w, t)[live].mean() > (0.8 if i < 4 else 0.5), i
    # without the input's part of the decay's gradient, and without the state's
    l, q, a, gain, si, kept = lb._local(c)
    before = np.concatenate([np.zeros((B, D, 1)) if c["h0"] is None else c["h0"][..., None], h[..., :-1]], -1)
    G = want["du"][2] / (gain * si)
    state, value = G * kept * before, G * a * a / gain * si * c["u"][2]
    for term, part in (("input", state), ("state", -value)):
        if term == "state" and not np.abs(state).any():
            continue
        assert outside(part * l * (1 - q), want["du"][0], tol["du"][0]).mean() > 0.5, term
        assert outside(-c["power"] * ref._sig(c["lam"]) * (part * q).sum((0, 2)), want["dlam"], tol["dlam"]).any(), term
    # G without what comes from behind
    if T > 1:
        alone = dict(c, gl=0 * c["gl"])
        lost = lb.ref.gated_scan_adjoint(c["u"], c["lam"], c["h0"], h, c["gh"], c["power"], c["resets"], 0 * c["gl"])
        assert outside(lost["du"][2], want["du"][2], tol["du"][2]).any() and alone is not c
    bad = want["du"][0].copy()
    bad[-1, -1, T - 1:] = 0
    assert outside(bad, want["du"][0], tol["du"][0]).any()


@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("N,V,masked", SCORES)
def test_score_adjoint_bounds(N, V, masked, half, scale):
    c = lb.score_inputs(N, V, half, masked)
    want, tol = lb.score_adjoint(c, scale, half)
    s = ref.token_logprobs(c["x"], c["tokens"], 0, scale)
    f = np.float32
    lse, H = s["lse"].astype(f)[:, None], s["entropy"].astype(f)[:, None]
    with np.errstate(invalid="ignore"):
        lp = f(scale) * c["x"].astype(f) - lse
        p = np.where(np.isfinite(lse), np.exp(lp), f(0))
    glp, gh, gl = (v.astype(f)[:, None] for v in (np.where(c["tokens"] >= 0, c["g"][0], 0.0), c["g"][1], c["g"][2]))
    terms = [-glp * p, gl * p, np.where(p > 0, -gh * p * (np.where(p > 0, lp, 0) + H), 0)]
    own = np.zeros_like(p)
    rows = np.flatnonzero((c["tokens"] >= 0) & np.isfinite(s["lse"]))
    own[rows, c["tokens"][rows]] = c["g"][0][rows]
    whole = sum(terms) + own

    def stored(x):
        return lb.bf16(f(scale) * x) if half else f(scale) * x
    assert not outside(stored(whole), want, tol).any()
    live = np.abs(want) > 1e-30
    if live.any() and V > 1:
        assert outside(0 * want, want, tol)[live].mean() > 0.95
        for k in range(3):
            if np.abs(terms[k]).any():
                assert outside(stored(whole - terms[k]), want, tol)[live].mean() > 0.3, k
        assert outside(stored(whole - own), want, tol).any()
