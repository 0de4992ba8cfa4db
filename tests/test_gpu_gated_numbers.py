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


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("B,T,D,layout", WAYS)
def test_a_new_document_keeps_nothing_of_a_bad_one(B, T, D, layout, bad):
    """A document of states that are not finite, between two others: the next one
    is what it is alone, forward; backward, gradients that are not finite stay
    in the documents they come from."""
    r = np.random.default_rng(T)
    u = [p.copy_(torch.from_numpy(r.standard_normal((B, D, T)))) for p in planes(B, T, D, layout, [0.0] * 3)]
    lam, h0 = torch.randn(D, device=DEV), torch.randn((B, D), device=DEV)
    first, second = T // 3, max(T // 3 + 1, 2 * T // 3)
    resets = torch.zeros((B, T), dtype=torch.bool, device=DEV)
    resets[:, first] = resets[:, second] = True
    clean, _ = pr.gated_scan(u, lam, h0, resets=resets)
    back = pr.gated_scan_adjoint(u, lam, h0, clean, torch.ones_like(clean), resets=resets)
    for g in (0, 2):  # a gate's NaN is in the decay and the input; an input's in the state alone
        spoilt = [p.clone(memory_format=torch.preserve_format) for p in u]
        spoilt[g][:, :, first] = bad if g == 2 else NAN
        h, _ = pr.gated_scan(spoilt, lam, h0, resets=resets)
        assert torch.equal(h[..., :first], clean[..., :first])
        assert not torch.isfinite(h[..., first:second]).any()
        assert torch.equal(h[..., second:], clean[..., second:])
    # h0 that is not finite ends with the row's first document
    h, _ = pr.gated_scan(u, lam, torch.full_like(h0, bad), resets=resets)
    assert torch.equal(h[..., first:], clean[..., first:])
    # a gradient in the middle document: the first and the last one do not see it
    gh = torch.ones_like(clean)
    gh[..., second - 1] = bad
    got = pr.gated_scan_adjoint(u, lam, h0, clean, gh, resets=resets)
    for a, b in zip(got["du"], back["du"]):
        assert torch.equal(a[..., :first], b[..., :first]) and torch.equal(a[..., second:], b[..., second:])
        assert not torch.isfinite(a[..., second - 1]).all()
    if first > 0:
        assert torch.equal(got["dh0"], back["dh0"])
    # and states that are not finite, in the gradients of their own document only
    states = clean.clone(memory_format=torch.preserve_format)
    states[..., first:second] = bad
    got = pr.gated_scan_adjoint(u, lam, h0, states, torch.ones_like(clean), resets=resets)
    for a, b in zip(got["du"], back["du"]):
        assert torch.equal(a[..., :first], b[..., :first]) and torch.equal(a[..., second:], b[..., second:])


def test_the_oracle_cuts_as_well():
    u = [np.zeros((1, 1, 4)) for _ in range(3)]
    resets = np.array([[False, False, True, False]])
    h = ref.gated_scan(u, np.zeros(1), np.full((1, 1), np.nan), 8.0, resets)
    assert np.isnan(h[0, 0, :2]).all() and np.isfinite(h[0, 0, 2:]).all()


@pytest.mark.parametrize("B,T,D,layout", WAYS)
def test_any_byte_but_zero_is_a_reset(B, T, D, layout):
    r = np.random.default_rng(T)
    u = [p.copy_(torch.from_numpy(r.standard_normal((B, D, T)))) for p in planes(B, T, D, layout, [0.0] * 3)]
    lam, h0 = torch.randn(D, device=DEV), torch.randn((B, D), device=DEV)
    values = torch.from_numpy(r.choice(np.array([0, 0, 1, 2, 64, 128, 255], np.uint8), (B, T))).to(DEV)
    h, _ = pr.gated_scan(u, lam, h0, resets=values)
    want, _ = pr.gated_scan(u, lam, h0, resets=values != 0)
    assert torch.equal(h, want)
    # and they cut where they stand: a step alone from nothing
    alone, _ = pr.gated_scan(u, lam, None, resets=torch.ones_like(values))
    where = (values != 0)[:, None].expand_as(h)
    assert torch.equal(h[where], alone[where])
