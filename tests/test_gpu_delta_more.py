"""The gated delta rule on the GPU: segments of long chains in every layout, the
gradients of equal keys, results that repeat, gates whose strides differ where
nothing steps, gradients that repeat elements."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import autograd as pag
from nonlinear_rnn_amd import pararnn as pr
from tests import delta_cases as dc
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "beta", "log_decay", "h0")


def check_all(c, t, half, scale, slack=1.0):
    a = [t[n] for n in NAMES]
    o, last = pr.delta_scan(*a, resets=t["resets"])
    want, S = dc.oracle(c, scale)
    dc.check(o, want, slack * dc.FORWARD[half], "o")
    dc.check(last, S, slack * dc.FORWARD[half], "last")
    out = pr.delta_scan_adjoint(*a, t["go"], g_last=t["g_last"], resets=t["resets"])
    want = dc.oracle(c, scale, True)
    for n in ("dq", "dk", "dv", "dbeta", "dlog_decay", "dh0"):
        if out[n] is not None:
            dc.check(out[n], want[n], 2 * slack * dc.FORWARD[half], n, half and n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("layout", ["time", "slices", "apart"])
@pytest.mark.parametrize("size,docs", [((1, 2100, 1, 2, 64, 40), 0.0005), ((2, 2113, 1, 1, 100, 33), 0.0),
                                       ((1, 2900, 1, 3, 200, 20), 0.002), ((1, 2048, 1, 1, 128, 128), 0.0)])
def test_long_chains_of_few_heads_in_every_layout(size, docs, layout, half):
    c = dc.inputs(*size, half, docs=docs)
    c["log_decay"] = np.float32(0.02 * c["log_decay"]).astype(np.float64)  # a segment's state matters to the next
    check_all(c, dc.tensors(c, half, layout, DEV), half, size[4] ** -0.5)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("rate", [0.0, 1.0, 2.0])
def test_gradients_of_equal_keys_and_full_rates(rate, half):
    """At rate 2 the maps keep every rounding of 128 steps: four times the forward
    pass's bound, as its own test has it, and twice that for a gradient."""
    c = dc.inputs(1, 128, 1, 1, 16, 16, half, decay="none")
    c["k"][:] = 0.25  # 16 channels: unit length, and exact
    c["beta"][:] = rate
    check_all(c, dc.tensors(c, half, "channel", DEV), half, 0.25, 4.0)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("size,layout", [((4, 1500, 8, 8, 128, 128), "channel"), ((2, 700, 4, 12, 80, 100), "time"),
                                         ((1, 4096, 1, 2, 64, 64), "channel"), ((2, 300, 1, 2, 256, 64), "channel"),
                                         ((8, 1, 4, 4, 64, 64), "channel")])
def test_results_repeat(size, layout, half):
    """The same bits from every call, whatever the workspace held before."""
    c = dc.inputs(*size, half, docs=0.003)
    t = dc.tensors(c, half, layout, DEV)
    a = [t[n] for n in NAMES]
    first = None
    for value in (0, 255, 63, 0, 127):  # 255: NaN
        ws = [torch.full((pr_bytes(t, adjoint),), value, dtype=torch.uint8, device=DEV) for adjoint in (0, 1)]
        o, last = pr.delta_scan(*a, resets=t["resets"], workspace=ws[0])
        g = pr.delta_scan_adjoint(*a, t["go"], g_last=t["g_last"], resets=t["resets"], workspace=ws[1])
        got = dict(g, o=o, last=last)
        first = first or got
        assert all(torch.equal(got[n], first[n]) for n in got), value


def pr_bytes(t, adjoint):
    plan = pr._delta_plan(*[t[n] for n in NAMES], t["resets"], None, t["go"] if adjoint else None, None, None, adjoint)
    return max(16, plan[3])


@pytest.mark.parametrize("shape", [(3, 2, 1), (1, 1, 70), (1, 2, 1), (1, 2, 70)])
def test_gates_whose_strides_differ_where_nothing_steps(shape):
    """A slice of a wider projection beside a tensor of its own."""
    B, Hv, T = shape
    c = dc.inputs(B, T, 1, Hv, 16, 20, False)
    t = dc.tensors(c, False, "channel", DEV)
    wide = torch.zeros((B, 7, T), device=DEV) if B == 1 else torch.zeros((B, T, Hv), device=DEV).transpose(1, 2)
    beta = wide[:, 2:2 + Hv] if B == 1 else wide
    beta.copy_(t["beta"])
    assert beta.stride() != t["log_decay"].stride()
    t["beta"] = beta
    check_all(c, t, False, 0.25)
    a = [t[n] for n in NAMES]
    want = pr.delta_scan(*a)
    leaves = [x.clone(memory_format=torch.preserve_format).requires_grad_(True) for x in a]
    got = pag.delta_scan(leaves[0], leaves[1], leaves[2], beta, leaves[4], leaves[5])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    (got[0].sum() + got[1].sum()).backward()
    if T == 1:
        states = t["h0"].clone()
        o = pr.delta_step(*[x[..., 0] for x in a[:5]], states)
        dc.check(o, dc.oracle(c, 0.25)[0][..., 0], 2.0 ** -19, "step")


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("size", [(2, 70, 1, 2, 24, 40), (1, 2100, 1, 1, 64, 33)])
def test_a_gradient_that_repeats_elements(size, half):
    """The gradient of a sum, of which no copy is made."""
    c = dc.inputs(*size, half, docs=0.01)
    t = dc.tensors(c, half, "channel", DEV)
    a = [t[n] for n in NAMES]
    B, T, _, Hv, _, dv = size
    for go in (torch.ones((), device=DEV).expand(B, Hv, dv, T), t["go"][..., :1].expand(B, Hv, dv, T),
               t["go"][:, :, :1].expand(B, Hv, dv, T)):
        got = pr.delta_scan_adjoint(*a, go, resets=t["resets"])
        want = pr.delta_scan_adjoint(*a, go.contiguous(), resets=t["resets"])
        assert all(torch.equal(got[n], want[n]) for n in got)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("bad", ["q", "k", "v", "beta", "log_decay"])
def test_a_number_that_is_not_finite_leaves_earlier_chunks_alone(bad, half):
    """And, where what holds it is a document of its own, all that is before it."""
    c = dc.inputs(1, 200, 1, 2, 24, 16, half)
    t = dc.tensors(c, half, "channel", DEV)
    good = pr.delta_scan(*[t[n] for n in NAMES])[0]
    padding = torch.arange(200, device=DEV)[None] == 150
    alone = pr.delta_scan(*[t[n] for n in NAMES], resets=padding)[0]
    t[bad][..., 150:] = float("nan")
    got = pr.delta_scan(*[t[n] for n in NAMES])[0]
    assert torch.equal(got[..., :128], good[..., :128])  # chunks of 64 steps, or of 32
    got = pr.delta_scan(*[t[n] for n in NAMES], resets=padding)[0]
    assert torch.equal(got[..., :150], alone[..., :150])
    if bad != "q":
        assert bool(got[..., 150:].isnan().any())
