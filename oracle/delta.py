"""Float64 oracle of the gated delta rule, forward, backward and a step, written
out from the definition in numpy, one step at a time."""
import numpy as np

FORGET = -104.0  # a log decay below keeps nothing: its exponential is 0 in float32


def _by_heads(x, heads):
    """[B][H][d][T] float64 with key heads repeated for the value heads that share them."""
    x = np.asarray(x, np.float64)
    return np.repeat(x, heads // x.shape[1], axis=1)


def _decay(log_decay, resets, shape):
    """(a [B][H][T], cut [B][H][T]): a step that is cut keeps nothing."""
    g = np.zeros(shape) if log_decay is None else np.asarray(log_decay, np.float64)
    cut = g < FORGET
    if resets is not None:
        cut = cut | np.asarray(resets, bool)[:, None]
    return np.exp(np.where(cut, 0.0, g)), cut


def _step(S, a, cut, k, v, b):
    """(decayed state, what is missing, what is written, new state); S [B][H][dk][dv]."""
    S = np.where(cut[..., None, None], 0.0, a[..., None, None] * S)
    miss = v - np.einsum("bhd,bhdv->bhv", k, S)
    w = b[..., None] * miss
    return S, miss, w, S + k[..., None] * w[:, :, None]


def delta_scan(q, k, v, beta, log_decay=None, h0=None, scale=1.0, resets=None):
    """(o [B][Hv][dv][T], last [B][Hv][dk][dv])."""
    v, b = np.asarray(v, np.float64), np.asarray(beta, np.float64)
    B, H, dv, T = v.shape
    q, k = _by_heads(q, H), _by_heads(k, H)
    a, cut = _decay(log_decay, resets, b.shape)
    S = np.zeros((B, H, k.shape[2], dv)) if h0 is None else np.asarray(h0, np.float64).copy()
    o = np.zeros(v.shape)
    for t in range(T):
        S = _step(S, a[..., t], cut[..., t], k[..., t], v[..., t], b[..., t])[3]
        o[..., t] = scale * np.einsum("bhd,bhdv->bhv", q[..., t], S)
    return o, S


def delta_scan_adjoint(q, k, v, beta, log_decay=None, h0=None, go=None, g_last=None, scale=1.0, resets=None):
    """dict(dq, dk, dv, dbeta, dlog_decay, dh0)."""
    v, b = np.asarray(v, np.float64), np.asarray(beta, np.float64)
    B, H, dv, T = v.shape
    Hk = np.shape(q)[1]
    q, k = _by_heads(q, H), _by_heads(k, H)
    dk = k.shape[2]
    a, cut = _decay(log_decay, resets, b.shape)
    states = [np.zeros((B, H, dk, dv)) if h0 is None else np.asarray(h0, np.float64)]
    for t in range(T):
        states.append(_step(states[-1], a[..., t], cut[..., t], k[..., t], v[..., t], b[..., t])[3])
    g = np.zeros((B, H, dk, dv)) if g_last is None else np.asarray(g_last, np.float64).copy()
    go = np.zeros(v.shape) if go is None else np.asarray(go, np.float64)
    out = dict(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape), dbeta=np.zeros(b.shape),
               dlog_decay=np.zeros(b.shape))
    for t in range(T - 1, -1, -1):
        S, miss, w, after = _step(states[t], a[..., t], cut[..., t], k[..., t], v[..., t], b[..., t])
        out["dq"][..., t] = scale * np.einsum("bhdv,bhv->bhd", after, go[..., t])
        g = g + scale * q[..., t][..., None] * go[..., t][:, :, None]
        gw = np.einsum("bhd,bhdv->bhv", k[..., t], g)
        out["dbeta"][..., t] = (gw * miss).sum(-1)
        out["dv"][..., t] = gm = b[..., t][..., None] * gw
        out["dk"][..., t] = np.einsum("bhdv,bhv->bhd", g, w) - np.einsum("bhdv,bhv->bhd", S, gm)
        g = g - k[..., t][..., None] * gm[:, :, None]
        out["dlog_decay"][..., t] = np.where(cut[..., t], 0.0, (g * S).sum((2, 3)))
        g = np.where(cut[..., t][..., None, None], 0.0, a[..., t][..., None, None] * g)
    for n in ("dq", "dk"):
        out[n] = out[n].reshape(B, Hk, H // Hk, dk, T).sum(2)
    return out | dict(dh0=g)


def delta_step(q, k, v, beta, log_decay, states, slots=None, scale=1.0):
    """(o [B][Hv][dv], the pool's states)."""
    states = np.asarray(states, np.float64).copy()
    B = np.shape(v)[0]
    o = np.zeros(np.shape(v))
    for b in range(B):
        slot = b if slots is None else int(slots[b])
        if not 0 <= slot < states.shape[0]:
            continue
        one = [np.asarray(x[b:b + 1])[..., None] for x in (q, k, v, beta)]
        g = None if log_decay is None else np.asarray(log_decay[b:b + 1])[..., None]
        r, S = delta_scan(*one, g, states[slot:slot + 1], scale)
        o[b], states[slot] = r[0, ..., 0], S[0]
    return o, states
