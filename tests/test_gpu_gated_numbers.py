"""The gated linear recurrence where its numbers are at their limits: decays near
0 and near 1, and states that are not finite.

Tolerances, in u = 2^-24.  The log decay l is a product of two (rate, sigmoid)
of under 8 roundings, and exp(l) one of under 4: a step's decay is within
(8 |l| + 4) u of itself.  A product of decays held as the sum of the l is within
(8 |l_1 + .. + l_T| + 4) u; where such products are applied to a state one after
the other, each adds 4 u.  A channel's chunks are 512 steps or more with its
steps in the lanes, and 8 or more elsewhere; within one the state takes up to 64
roundings."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr
from oracle import language as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NAN, INF = float("nan"), float("inf")


def f64(t):
    return t.detach().double().cpu().numpy()


def planes(B, T, D, layout, values, dtype=torch.float32):
    """Planes [B][D][T] that hold one value a channel."""
    out = []
    for v in values:
        p = torch.empty((B, T, D) if layout == "time" else (B, D, T), dtype=dtype, device=DEV)
        p = p.transpose(1, 2) if layout == "time" else p
        v = torch.as_tensor(v, dtype=torch.float32, device=DEV)
        out.append(p.copy_(v[None, :, None].expand(B, D, T) if v.dim() else v.expand(B, D, T)))
    return out


# one shape for each way of running: a lane a channel, chunks of 64 channels, groups
# of 4 and 16 lanes, one wave, four waves, chunks of a channel
WAYS = [(1, 6, 70, "channel"), (2, 40, 70, "time"), (1, 200, 70, "time"), (1, 3, 64, "time"), (3, 15, 9, "channel"),
        (2, 60, 33, "channel"), (1, 500, 40, "channel"), (1, 9000, 600, "channel"), (1, 9000, 20, "channel"),
        (1, 5000, 2049, "channel"), (1, 40, 131100, "time")]


@pytest.mark.parametrize("B,T,D,layout", WAYS)
def test_fast_decays(B, T, D, layout):
    """A state alone (no input), at decays from e^-0.1 to e^-60 a step: every state
    and every carried gradient to its own relative accuracy."""
    l = -np.geomspace(0.1, 60.0, D) if D > 1 else np.array([-6.0])
    lam = torch.from_numpy(np.log(np.expm1(-l / 4.0))).float().to(DEV)  # softplus = -l / 4
    u = planes(B, T, D, layout, [0.0, 0.0, 0.0])  # sig(0) = 1/2 of power 8
    h0 = torch.full((B, D), 1.5, device=DEV)
    h, last = pr.gated_scan(u, lam, h0)
    exact_l = -4.0 * np.logaddexp(0.0, f64(lam))
    steps = np.arange(1, T + 1)
    want = 1.5 * np.exp(exact_l[None, :, None] * steps)
    tol = want * U * (8 * np.abs(exact_l)[None, :, None] * steps + 4 * steps.clip(max=64) + steps / 8 * 4 + 8)
    fine = np.broadcast_to(want > 1e-30, h.shape)  # float32 is denormal from 1e-38 on
    assert (np.abs(f64(h) - want) <= tol)[fine].all()
    gl = torch.full((B, D), -2.0, device=DEV)
    got = pr.gated_scan_adjoint(u, lam, h0, h, None, gh_last=gl)
    want0 = -2.0 * np.exp(exact_l * T)[None].repeat(B, 0)
    tol0 = np.abs(want0) * U * (8 * np.abs(exact_l) * T + 4 * min(T, 64) + T / 8 * 4 + 8)
    fine = np.abs(want0) > 1e-30
    assert (np.abs(f64(got["dh0"]) - want0) <= tol0)[fine].all()
    # du_r = G (a h_{t-1}) l (1 - 1/2): as accurate
    G = -2.0 * np.exp(exact_l[:, None] * (T - steps))
    want_r = (G * 1.5 * np.exp(exact_l[:, None] * steps) * exact_l[:, None] * 0.5)[None].repeat(B, 0)
    tol_r = np.abs(want_r) * U * (16 * np.abs(exact_l)[:, None] * T + 8 * min(T, 64) + T + 32)
    fine = np.abs(want_r) > 1e-30
    assert (np.abs(f64(got["du"][0]) - want_r) <= tol_r)[fine].all()


def test_fast_decays_of_one_step():
    l = -np.geomspace(0.1, 60.0, 300)
    lam = torch.from_numpy(np.log(np.expm1(-l / 4.0))).float().to(DEV)
    states = torch.full((2, 300), 1.5, device=DEV)
    pr.gated_step([torch.zeros((2, 300), device=DEV)] * 3, lam, states)
    exact_l = -4.0 * np.logaddexp(0.0, f64(lam))
    want = 1.5 * np.exp(exact_l)[None].repeat(2, 0)
    assert (np.abs(f64(states) - want) <= want * U * (8 * np.abs(exact_l) + 8)).all()


@pytest.mark.parametrize("B,T,D,layout,chunk", [(1, 262144, 4, "channel", 512), (1, 65536, 2100, "channel", 512),
                                                (1, 65536, 600, "channel", 512), (1, 262144, 64, "time", 64)])
@pytest.mark.parametrize("ur", [-6.0, -8.0, -10.0])
def test_long_memory(B, T, D, layout, chunk, ur):
    """A steady gate near no decay, over a long sequence: what is left of h0 at
    its end, and of the last state's gradient at its start."""
    decay = 0.9 + 0.099 * np.random.default_rng(D).random(D)
    lam = torch.from_numpy(np.log(np.expm1(-np.log(decay) / 8.0))).float().to(DEV)
    u = planes(B, T, D, layout, [ur, 0.0, 0.0])
    one = torch.ones((B, D), device=DEV)
    h, last = pr.gated_scan(u, lam, one)
    total = -8.0 * np.logaddexp(0.0, f64(lam)) / (1.0 + np.exp(-ur)) * T
    want = np.exp(total)[None].repeat(B, 0)
    tol = want * U * (8 * np.abs(total) + 4 * T / chunk + 64)
    fine = want > 1e-30
    assert fine.any()
    assert (np.abs(f64(last) - want) <= tol)[fine].all(), float((np.abs(f64(last) - want) / want)[fine].max())
    got = pr.gated_scan_adjoint(u, lam, one, h, None, gh_last=one)
    assert (np.abs(f64(got["dh0"]) - want) <= tol)[fine].all()
