"""A bound for every element of the distillation's results, from the oracle's
formulas with the roundings carried along (u = 2^-24).

Sums of exponentials are within (V / 256 + 32) u of themselves (a thread's
share, then a tree), so a log probability is within that, 4 u of its own size
and 4 u of the row's largest distance from the maximum.  A teacher's
probability is within 4 u of itself, r = 1 - P therefore within 4 u P + u.
The loss is a sum of products of these; the gradient takes q from lse, a float32
with a rounding of its own size, and r / q_rest from log_rest."""
import numpy as np

from oracle import logits as ref

U = 2.0 ** -24
BF16_HALF_ULP = 2.0 ** -8 * 1.01
TINY = 1e-36


def _parts(c, tail, scale):
    x, index, lp = c["x"], c["index"], c["logprob"]
    N, V = x.shape
    out = ref.distill_top(x, index, lp, tail, scale)
    used = index >= 0
    p = np.where(used, np.exp(np.where(used, lp, -np.inf)), 0.0)
    r = 1.0 - p.sum(1)
    r = np.where((r >= ref.REST) & tail, r, 0.0)
    return out, used, p, r, U * (V / 256 + 32)


def loss(c, tail, scale=1.0):
    """(results, their bounds)."""
    out, used, p, r, base = _parts(c, tail, scale)
    x, index = c["x"], c["index"]
    lse = np.where(np.isfinite(out["lse"]), out["lse"], 0.0)
    lq = np.where(used, scale * np.take_along_axis(x, np.clip(index, 0, x.shape[1] - 1), 1) - lse[:, None], 0.0)
    lq = np.where(p > 0, lq, 0.0)
    with np.errstate(invalid="ignore"):
        spread = np.abs(scale * np.where(np.isfinite(x), x, 0.0)).max(1) + np.abs(lse)
    err = base + 4 * U * (np.abs(lq) + spread[:, None] + 1)
    lp = np.where(p > 0, c["logprob"], 0.0)
    tol = (p * (err + 8 * U * (np.abs(lp) + np.abs(lq)))).sum(1)
    rest = np.where(np.isfinite(out["log_rest"]), out["log_rest"], 0.0)
    log_r = np.log(np.where(r > 0, r, 1.0))
    err_rest = 2 * base + 4 * U * (np.abs(rest) + spread + 1)
    dr = 4 * U * p.sum(1) + U
    tol += np.where(r > 0, r * (err_rest + 8 * U * np.abs(log_r)) + dr * (np.abs(log_r - rest) + 1), 0.0)
    return out, dict(loss=tol + 4 * U * np.abs(np.where(np.isfinite(out["loss"]), out["loss"], 0)) + TINY,
                     lse=base + 4 * U * (np.abs(lse) + spread), log_rest=err_rest)


def gradient(c, g, tail, scale=1.0, half=False):
    """(gradient, its bound)."""
    out, used, p, r, base = _parts(c, tail, scale)
    x, index = c["x"], c["index"]
    N, V = x.shape
    want = ref.distill_top_adjoint(x, index, c["logprob"], g, tail, scale)
    live = np.isfinite(out["lse"]) & used.any(1)
    lse = np.where(live, out["lse"], 0.0)[:, None]
    lq = np.where(np.isfinite(x) & live[:, None], scale * np.where(np.isfinite(x), x, 0.0) - lse, -np.inf)
    q = np.exp(lq)
    lq = np.where(q > 0, lq, 0.0)
    rest = np.where(np.isfinite(out["log_rest"]), out["log_rest"], 0.0)[:, None]
    err = base + 4 * U * (2 * np.abs(lse) + 64 + np.abs(lq))
    err_rest = 2 * base + 4 * U * (np.abs(rest) + np.abs(lse) + 64)
    P, dr, share = p.sum(1)[:, None], 4 * U * p.sum(1)[:, None] + U, r[:, None] * np.exp(-rest)
    share = np.where(r[:, None] > 0, share, 0.0)
    tol = q * ((P + r[:, None] + share) * (err + err_rest + 32 * U) + dr * (1 + np.exp(-rest)))
    at = np.zeros((N, V + 1))
    for n in range(N):
        np.add.at(at[n], np.where(used[n], index[n], V), p[n] * 16 * U)
    tol = np.abs(g)[:, None] * scale * (tol + at[:, :V]) + 4 * U * np.abs(want) + TINY
    return want, tol + (BF16_HALF_ULP * (np.abs(want) + tol) if half else 0.0)
