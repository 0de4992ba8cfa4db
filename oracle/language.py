"""Float64 oracle of the language-model operators: the gated linear
recurrence, the block boundary and the token scores, forward and backward,
written out from their definitions in numpy, one step at a time."""
import numpy as np


def _sig(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def _log_decay(ur, lam, power):
    """l [B][D][T], sig(u_r)."""
    soft = np.maximum(lam, 0) + np.log1p(np.exp(-np.abs(lam)))
    q = _sig(ur)
    return -power * soft[None, :, None] * q, q


def gated_scan(u, lam, h0, power, resets=None):
    """h [B][D][T] from planes u = (r, i, x) [B][D][T]."""
    ur, ui, ux = (np.asarray(p, np.float64) for p in u)
    lam = np.asarray(lam, np.float64)
    B, D, T = ur.shape
    l, _ = _log_decay(ur, lam, power)
    a, gain = np.exp(l), np.sqrt(-np.expm1(2 * l))
    h = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64).copy()
    out = np.empty((B, D, T))
    for t in range(T):
        if resets is not None:  # nothing of the state is kept, also where it is not finite
            h = np.where(np.asarray(resets[:, t], bool)[:, None], 0.0, h)
        h = a[..., t] * h + gain[..., t] * _sig(ui[..., t]) * ux[..., t]
        out[..., t] = h
    return out


def gated_scan_adjoint(u, lam, h0, h, gh, power, resets=None, gh_last=None):
    """dict(du, dlam, dh0), and dlam_terms: the sum of the terms' magnitudes,
    by which the rounding of the sum is judged."""
    ur, ui, ux = (np.asarray(p, np.float64) for p in u)
    lam, h = np.asarray(lam, np.float64), np.asarray(h, np.float64)
    B, D, T = ur.shape
    l, q = _log_decay(ur, lam, power)
    a, y = np.exp(l), -np.expm1(2 * l)
    gain, si = np.sqrt(y), _sig(ui)
    du = [np.zeros((B, D, T)) for _ in range(3)]
    carry = np.zeros((B, D)) if gh_last is None else np.asarray(gh_last, np.float64).copy()
    dl_q, dl_q_abs, G_max = np.zeros((B, D)), np.zeros((B, D)), 0.0
    for t in range(T - 1, -1, -1):
        cut = np.zeros((B, 1), bool) if resets is None else np.asarray(resets[:, t], bool)[:, None]
        G = carry + (0.0 if gh is None else np.asarray(gh[..., t], np.float64))
        G_max = max(G_max, float(np.abs(G).max(initial=0.0)))
        before = h[..., t - 1] if t else (np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64))
        before = np.where(cut, 0.0, before)
        at, gt, st, xt = a[..., t], gain[..., t], si[..., t], ux[..., t]
        # d sqrt(1 - e^{2l}) / dl = -e^{2l} / sqrt(1 - e^{2l}); its product with l -> 0 as l -> 0
        slope = np.divide(at * at, gt, out=np.zeros_like(gt), where=gt > 1e-15)
        dl = G * (at * before - slope * st * xt)
        du[0][..., t] = dl * l[..., t] * (1 - q[..., t])
        du[1][..., t] = G * gt * xt * st * (1 - st)
        du[2][..., t] = G * gt * st
        dl_q += dl * q[..., t]
        dl_q_abs += np.abs(G * at * before * q[..., t]) + np.abs(G * slope * st * xt * q[..., t])
        carry = np.where(cut, 0.0, at * G)
    factor = -power * _sig(lam)
    return dict(du=du, dlam=factor * dl_q.sum(0), dh0=carry, G_max=G_max,
                dlam_terms=np.abs(factor) * dl_q_abs.sum(0))


def block_norm(h, x, w_post, w_pre, gate=None, scale=1.0, eps=1e-6):
    """(y, z, rstd [2][B][T]); h, gate [B][D][T], x [B][T][D]."""
    y = np.asarray(x, np.float64)
    r1 = np.zeros(y.shape[:2])
    if h is not None:
        v = np.asarray(h, np.float64).transpose(0, 2, 1)
        if gate is not None:
            g = np.asarray(gate, np.float64).transpose(0, 2, 1)
            v = v * g * _sig(g)
        r1 = 1 / np.sqrt((v * v).mean(-1) + eps)
        y = y + scale * v * r1[..., None] * w_post
    r2 = 1 / np.sqrt((y * y).mean(-1) + eps)
    return y, y * r2[..., None] * w_pre, np.stack([r1, r2])


def block_norm_adjoint(h, x, w_post, w_pre, gy, gz, gate=None, scale=1.0, eps=1e-6):
    """dict(dh, dgate, dx, dw_post, dw_pre)."""
    y, _, (r1, r2) = block_norm(h, x, w_post, w_pre, gate, scale, eps)
    zero = np.zeros_like(y)
    gy = zero if gy is None else np.asarray(gy, np.float64)
    gz = zero if gz is None else np.asarray(gz, np.float64)
    n2 = y * r2[..., None]
    q = gz * w_pre
    dx = gy + r2[..., None] * (q - n2 * (q * n2).mean(-1, keepdims=True))
    out = dict(dx=dx, dw_pre=(gz * n2).sum((0, 1)), dh=None, dgate=None, dw_post=None,
               dw_terms=np.abs(gz * n2).sum((0, 1)))
    if h is None:
        return out
    hh = np.asarray(h, np.float64).transpose(0, 2, 1)
    g = np.ones_like(hh) if gate is None else np.asarray(gate, np.float64).transpose(0, 2, 1)
    act = g if gate is None else g * _sig(g)
    n1 = hh * act * r1[..., None]
    p = scale * dx * w_post
    dv = r1[..., None] * (p - n1 * (p * n1).mean(-1, keepdims=True))
    out["dw_post"] = (scale * dx * n1).sum((0, 1))
    out["dw_terms"] = out["dw_terms"] + np.abs(scale * dx * n1).sum((0, 1))
    out["dh"] = (dv * act).transpose(0, 2, 1)
    if gate is not None:
        out["dgate"] = (dv * hh * (_sig(g) * (1 + g * (1 - _sig(g))))).transpose(0, 2, 1)
    return out


def token_logprobs(logits, tokens, top=0, scale=1.0):
    """dict(logprob, entropy, lse, top_index, top_logprob), row by row."""
    x = np.asarray(logits, np.float64)
    N, V = x.shape
    out = dict(logprob=np.zeros(N), entropy=np.zeros(N), lse=np.full(N, -np.inf),
               top_index=np.full((N, top), -1, np.int64), top_logprob=np.full((N, top), -np.inf))
    for n in range(N):
        row, t = scale * x[n], int(tokens[n])
        bad = np.isnan(row).any() or np.isposinf(row).any()
        live = np.flatnonzero(~np.isneginf(row) & ~np.isnan(row))
        if bad:
            out["lse"][n] = out["entropy"][n] = np.nan
        elif live.size:
            m = row[live].max()
            out["lse"][n] = m + np.log(np.exp(row[live] - m).sum())
            logp = row[live] - out["lse"][n]
            out["entropy"][n] = -(np.exp(logp) * logp).sum()
        if t >= V:
            out["logprob"][n] = np.nan
        elif t >= 0:
            out["logprob"][n] = -np.inf if not live.size and not bad else row[t] - out["lse"][n]
        best = live[np.lexsort((live, -x[n][live]))][:top]
        out["top_index"][n, :best.size] = best
        out["top_logprob"][n, :best.size] = row[best] - out["lse"][n]
    return out


def token_logprobs_adjoint(logits, tokens, g_logprob=None, g_entropy=None, g_lse=None, scale=1.0):
    """dL/dlogits."""
    x = np.asarray(logits, np.float64)
    s = token_logprobs(x, tokens, 0, scale)
    out = np.zeros_like(x)
    N, V = x.shape
    for n in range(N):
        if np.isneginf(s["lse"][n]):
            continue
        logp = scale * x[n] - s["lse"][n]
        p = np.exp(logp)
        plogp = np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0)
        glp = g_logprob[n] if g_logprob is not None and tokens[n] >= 0 else 0.0
        out[n] = -glp * p
        if g_lse is not None:
            out[n] += g_lse[n] * p
        if g_entropy is not None:
            out[n] -= g_entropy[n] * (plogp + p * s["entropy"][n])
        if 0 <= tokens[n] < V:
            out[n, tokens[n]] += glp
    return scale * out
