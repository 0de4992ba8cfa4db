"""Inputs and tolerances for the tests of the gated delta rule.

Tolerances are of norms.  The state goes from step to step by maps of norm at
most 1 (unit keys, beta in [0, 1], decays at most 1), so a rounding is not
amplified on its way; what a step writes is a difference of two numbers of its
inputs' size, once again as much.  On the way from the state before a chunk to
the output eight operands are rounded or products of two remainders left out
(the state, R, the inverse, W twice, P; two products of two such operands), each
with bfloat16 inputs within 2^-17 of itself, with float32 inputs a sum of 64 to
256 products of 2^-24.  With the factor of two, and as much again for the sums
of the gates' factors, relative to the norm of the result:
    8 * 2 * 2 * 2^-17 = 2^-12 at most, the roundings independent: 2^-14;
    float32: sums of 256 terms as random walks, 16 * 2^-24 * 32 = 2^-15.
The largest error of one element may be 16 times as large against the root mean
square.  A gradient passes through the chain twice: twice as much.  Rounding to
bfloat16 adds at most 2^-8 of an element (half a step of 8 bits), so of the norm."""
import numpy as np
import torch

from oracle import delta as ref

FORWARD = {True: 2.0 ** -14, False: 2.0 ** -15}


def inputs(B, T, Hk, Hv, dk, dv, half, layout="channel", decay="mild", docs=0.0, h0=True, seed=0):
    """float64 arrays that their types hold, by name."""
    r = np.random.default_rng(seed + 7919 * T + 31 * dk + dv)

    def kept(x, as_half):
        t = torch.from_numpy(np.asarray(x, np.float32))
        return (t.bfloat16() if as_half else t).double().numpy()

    def unit(x):
        return x / np.maximum(np.linalg.norm(x, axis=2, keepdims=True), 1e-30)
    c = dict(q=kept(unit(r.standard_normal((B, Hk, dk, T))), half), k=kept(unit(r.standard_normal((B, Hk, dk, T))), half),
             v=kept(r.standard_normal((B, Hv, dv, T)), half), beta=kept(r.random((B, Hv, T)), False),
             h0=kept(r.standard_normal((B, Hv, dk, dv)), False) if h0 else None,
             resets=r.random((B, T)) < docs if docs else None)
    if decay == "none":
        c["log_decay"] = None
    else:
        g = -0.2 * r.random((B, Hv, T))
        if decay == "strong":
            g = -30.0 * r.random((B, Hv, T))
        if decay == "forget":  # steps that keep nothing, by the type's lowest value and by infinity
            g[r.random(g.shape) < 0.05] = -np.inf
            g[r.random(g.shape) < 0.05] = np.finfo(np.float32).min
            g[r.random(g.shape) < 0.05] = -104.5
        c["log_decay"] = kept(g, False)
    c["go"], c["g_last"] = kept(r.standard_normal((B, Hv, dv, T)), False), kept(r.standard_normal((B, Hv, dk, dv)), False)
    return c


def place(x, layout, dtype, dev):
    """A tensor [B][H][d][T] in a layout."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(dev)
    B, H, d, T = t.shape
    if layout == "channel":
        return t
    if layout == "time":
        return t.permute(0, 3, 1, 2).contiguous().permute(0, 2, 3, 1)
    if layout == "slices":  # heads in the middle of a wider projection, an odd number of elements apart
        wide = torch.zeros((B, H * d + 5, T + 3), dtype=dtype, device=dev)
        wide[:, 2:2 + H * d, 1:1 + T] = t.reshape(B, H * d, T)
        return wide[:, 2:2 + H * d, 1:1 + T].unflatten(1, (H, d))
    assert layout == "apart"  # neither steps nor channels side by side
    wide = torch.zeros((T, 2, B, 2, d, 3, H), dtype=dtype, device=dev)
    wide[:, 0, :, 0, :, 0] = t.permute(3, 0, 2, 1)
    return wide[:, 0, :, 0, :, 0].permute(1, 3, 2, 0)


def tensors(c, half, layout, dev):
    dtype = torch.bfloat16 if half else torch.float32
    f32 = lambda x: None if x is None else torch.from_numpy(np.float32(x)).to(dev)  # noqa: E731
    t = {n: place(c[n], layout, dtype, dev) for n in ("q", "k", "v")}
    t |= {n: f32(c[n]) for n in ("beta", "log_decay", "h0", "g_last")}
    t["go"] = place(c["go"], layout, torch.float32, dev)
    t["resets"] = None if c["resets"] is None else torch.from_numpy(c["resets"]).to(dev)
    return t


def oracle(c, scale, adjoint=False):
    names = ("q", "k", "v", "beta", "log_decay", "h0", "resets")
    args = {n: c[n] for n in names}
    if adjoint:
        return ref.delta_scan_adjoint(**args, go=c["go"], g_last=c["g_last"], scale=scale)
    return ref.delta_scan(**args, scale=scale)


def check(got, want, rel, what, rounded=False):
    """Norm and largest error; `rounded`: the result is bfloat16."""
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, what
    if not want.size:
        return
    assert np.isfinite(got).all(), what
    e, norm = got - want, np.linalg.norm(want)
    rms = norm / np.sqrt(want.size)
    half = 2.0 ** -8 if rounded else 0.0
    assert np.linalg.norm(e) <= (rel + half) * norm + 1e-30, (what, np.linalg.norm(e) / norm)
    assert (np.abs(e) <= 16 * rel * rms + half * np.abs(want) + 1e-30).all(), (what, np.abs(e).max() / rms)
