"""The gated delta rule on the GPU against its float64 oracle: the scan, its
backward pass and the step, at the sizes, layouts, documents and decays where
they can go wrong."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import autograd as pag
from nonlinear_rnn_amd import pararnn as pr
from oracle import delta as ref
from tests import delta_cases as dc
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

# B, T, Hk, Hv, dk, dv
SIZES = [(1, 1, 1, 1, 1, 1), (2, 2, 1, 2, 3, 5), (1, 31, 1, 1, 64, 64), (1, 32, 2, 2, 16, 31), (2, 33, 1, 3, 33, 17),
         (1, 63, 1, 1, 128, 32), (2, 64, 2, 2, 64, 33), (1, 65, 1, 1, 65, 100), (1, 128, 1, 2, 100, 1),
         (1, 130, 8, 8, 32, 16), (1, 200, 1, 1, 129, 64), (1, 97, 1, 2, 256, 48), (3, 257, 2, 4, 128, 128)]


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("size", SIZES)
def test_scan(size, half):
    c = dc.inputs(*size, half)
    t = dc.tensors(c, half, "channel", DEV)
    o, last = pr.delta_scan(t["q"], t["k"], t["v"], t["beta"], t["log_decay"], t["h0"], scale=0.7)
    want, S = dc.oracle(c, 0.7)
    dc.check(o, want, dc.FORWARD[half], "o")
    dc.check(last, S, dc.FORWARD[half], "last")


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("layout", ["time", "slices", "apart"])
@pytest.mark.parametrize("size", [(2, 70, 2, 4, 24, 40), (1, 131, 1, 1, 96, 33)])
def test_layouts(size, layout, half):
    c = dc.inputs(*size, half, docs=0.03)
    t = dc.tensors(c, half, layout, DEV)
    args = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    o, last = pr.delta_scan(*args, resets=t["resets"])
    scale = size[4] ** -0.5
    want, S = dc.oracle(c, scale)
    dc.check(o, want, dc.FORWARD[half], "o")
    dc.check(last, S, dc.FORWARD[half], "last")
    out = pr.delta_scan_adjoint(*args, t["go"], g_last=t["g_last"], resets=t["resets"])
    check_gradients(out, dc.oracle(c, scale, True), half)


def check_gradients(out, want, half):
    for n in ("dq", "dk", "dv", "dbeta", "dlog_decay", "dh0"):
        if out[n] is not None:
            dc.check(out[n], want[n], 2 * dc.FORWARD[half], n, half and n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("size", SIZES)
def test_adjoint(size, half):
    c = dc.inputs(*size, half)
    t = dc.tensors(c, half, "channel", DEV)
    out = pr.delta_scan_adjoint(t["q"], t["k"], t["v"], t["beta"], t["log_decay"], t["h0"], t["go"], g_last=t["g_last"],
                                scale=0.7)
    check_gradients(out, dc.oracle(c, 0.7, True), half)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("decay,docs", [("none", 0.0), ("none", 0.05), ("mild", 0.3), ("mild", 1.0), ("strong", 0.0),
                                        ("strong", 0.05), ("forget", 0.0), ("forget", 0.05)])
def test_documents_and_decays(decay, docs, half):
    c = dc.inputs(2, 150, 1, 2, 40, 24, half, decay=decay, docs=docs)
    t = dc.tensors(c, half, "channel", DEV)
    args = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    o, last = pr.delta_scan(*args, resets=t["resets"])
    want, S = dc.oracle(c, 40 ** -0.5)
    dc.check(o, want, dc.FORWARD[half], "o")
    dc.check(last, S, dc.FORWARD[half], "last")
    out = pr.delta_scan_adjoint(*args, t["go"], g_last=t["g_last"], resets=t["resets"])
    check_gradients(out, dc.oracle(c, 40 ** -0.5, True), half)


@pytest.mark.parametrize("half", [True, False])
def test_a_reset_at_a_chunk_and_beside_it(half):
    for first in (0, 1, 31, 32, 33, 63, 64, 65, 127, 129):
        c = dc.inputs(1, 130, 1, 1, 32, 16, half, seed=first)
        c["resets"] = np.arange(130)[None] == first
        t = dc.tensors(c, half, "channel", DEV)
        args = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
        o, last = pr.delta_scan(*args, resets=t["resets"])
        want, S = dc.oracle(c, 32 ** -0.5)
        dc.check(o, want, dc.FORWARD[half], "o")
        dc.check(last, S, dc.FORWARD[half], "last")
        out = pr.delta_scan_adjoint(*args, t["go"], g_last=t["g_last"], resets=t["resets"])
        check_gradients(out, dc.oracle(c, 32 ** -0.5, True), half)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("bad", ["q", "k", "v", "beta", "log_decay", "h0"])
def test_documents_that_are_not_finite(bad, half):
    """Documents of 50 steps, the second (for h0: the first) full of NaN and
    infinities: the others' outputs and gradients are bit for bit those of
    finite inputs."""
    c = dc.inputs(1, 200, 1, 2, 24, 16, half)
    c["resets"] = np.arange(200)[None] % 50 == 0
    if bad == "h0":
        c["resets"][0, 0] = False
    t = dc.tensors(c, half, "channel", DEV)
    names = ("q", "k", "v", "beta", "log_decay", "h0")

    def run():
        args = [t[n] for n in names]
        o, last = pr.delta_scan(*args, resets=t["resets"])
        g = pr.delta_scan_adjoint(*args, t["go"], g_last=t["g_last"], resets=t["resets"])
        return o.clone(), last.clone(), g
    good = run()
    if bad == "h0":
        t["h0"][..., ::2] = float("nan")
        t["h0"][..., 1::2] = float("inf")
        rows = slice(50, 200)
    else:
        t[bad][..., 50:100] = float("nan")
        t[bad][..., 60:70] = float("inf")
        rows = [i for i in range(200) if not 50 <= i < 100]
    got = run()
    assert torch.equal(good[0][..., rows], got[0][..., rows]) and torch.equal(good[1], got[1])
    for n in ("dq", "dk", "dv", "dbeta", "dlog_decay"):
        assert torch.equal(good[2][n][..., rows], got[2][n][..., rows]), n
    if bad != "h0":
        assert torch.equal(good[2]["dh0"], got[2]["dh0"])


@pytest.mark.parametrize("half", [True, False])
def test_far_sums_of_decays(half):
    """A step that forgets nearly everything (exp(-100)), then long memory: the
    sum of the log decays is 100 times what the later steps differ by."""
    c = dc.inputs(1, 192, 1, 1, 32, 32, half)
    c["log_decay"][:] = np.float32(-1e-3)
    c["log_decay"][..., [5, 20, 70, 71, 72, 140]] = -100.0
    t = dc.tensors(c, half, "channel", DEV)
    args = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    o, last = pr.delta_scan(*args)
    want, S = dc.oracle(c, 32 ** -0.5)
    dc.check(o, want, dc.FORWARD[half], "o")
    dc.check(last, S, dc.FORWARD[half], "last")
    check_gradients(pr.delta_scan_adjoint(*args, t["go"], g_last=t["g_last"]), dc.oracle(c, 32 ** -0.5, True), half)


@pytest.mark.parametrize("half", [True, False])
def test_equal_keys_and_full_rates(half):
    """Every key the same, beta 1 and 2: the system's matrix is full, its inverse is not."""
    for rate in (0.0, 1.0, 2.0):
        c = dc.inputs(1, 128, 1, 1, 16, 16, half, decay="none")
        c["k"][:] = 0.25  # 16 channels: unit length, and exact
        c["beta"][:] = rate
        t = dc.tensors(c, half, "channel", DEV)
        o, last = pr.delta_scan(*[t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")])
        want, S = dc.oracle(c, 0.25)
        dc.check(o, want, 4 * dc.FORWARD[half], "o")  # at rate 2 the maps keep every rounding of 128 steps
        dc.check(last, S, 4 * dc.FORWARD[half], "last")


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("size,decay,docs", [
    ((1, 2500, 1, 2, 32, 40), "mild", 0.0), ((1, 4100, 1, 1, 64, 16), "mild", 0.0005), ((2, 2113, 1, 1, 100, 33), "none", 0.0),
    ((1, 3000, 1, 3, 200, 20), "mild", 0.002), ((1, 2300, 2, 2, 16, 16), "forget", 0.0), ((1, 2048, 1, 1, 128, 128), "mild", 0.02)])
def test_long_chains_of_few_heads(size, decay, docs, half):
    """Chained in segments at once: from their maps the state before each."""
    c = dc.inputs(*size, half, decay=decay, docs=docs)
    t = dc.tensors(c, half, "channel", DEV)
    if decay == "mild":  # long memory, so that a segment's state matters to the next
        c["log_decay"] = np.float32(0.02 * c["log_decay"]).astype(np.float64)
        t["log_decay"] = torch.from_numpy(np.float32(c["log_decay"])).to(DEV)
    args = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    o, last = pr.delta_scan(*args, resets=t["resets"])
    scale = size[4] ** -0.5
    want, S = dc.oracle(c, scale)
    dc.check(o, want, dc.FORWARD[half], "o")
    dc.check(last, S, dc.FORWARD[half], "last")
    out = pr.delta_scan_adjoint(*args, t["go"], g_last=t["g_last"], resets=t["resets"])
    check_gradients(out, dc.oracle(c, scale, True), half)


@pytest.mark.parametrize("half", [True, False])
def test_segments_of_a_document_that_is_not_finite(half):
    """NaN in the first of two documents, many segments long: nothing of it in the second."""
    c = dc.inputs(1, 4000, 1, 1, 32, 32, half)
    c["resets"] = np.arange(4000)[None] == 2001
    t = dc.tensors(c, half, "channel", DEV)
    args = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]

    def run():
        o, last = pr.delta_scan(*args, resets=t["resets"])
        return o, last, pr.delta_scan_adjoint(*args, t["go"], g_last=t["g_last"], resets=t["resets"])
    good = run()
    t["v"][..., :2001] = float("nan")
    t["go"][..., :2001] = float("inf")
    got = run()
    assert torch.equal(good[0][..., 2001:], got[0][..., 2001:]) and torch.equal(good[1], got[1])
    for n in ("dq", "dk", "dv", "dbeta", "dlog_decay"):
        assert torch.equal(good[2][n][..., 2001:], got[2][n][..., 2001:]), n


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("layout", ["channel", "time", "apart"])
@pytest.mark.parametrize("size", [(1, 131, 1, 2, 200, 40), (2, 64, 1, 1, 256, 65)])
def test_many_key_channels(size, layout, half):
    """More than 128: one visit's keys and queries in LDS."""
    c = dc.inputs(*size, half, docs=0.03)
    t = dc.tensors(c, half, layout, DEV)
    a = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    want, S = dc.oracle(c, size[4] ** -0.5)
    o, last = pr.delta_scan(*a, resets=t["resets"])
    dc.check(o, want, dc.FORWARD[half], "o")
    dc.check(last, S, dc.FORWARD[half], "last")
    out = pr.delta_scan_adjoint(*a, t["go"], g_last=t["g_last"], resets=t["resets"])
    check_gradients(out, dc.oracle(c, size[4] ** -0.5, True), half)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("layout", ["channel", "time"])
@pytest.mark.parametrize("size,docs", [((32, 70, 4, 8, 20, 40), 0.05), ((64, 1, 4, 4, 64, 64), 0.0), ((16, 131, 8, 16, 70, 33), 0.0),
                                       ((4, 70, 32, 32, 128, 100), 0.02)])
def test_many_chains(size, docs, layout, half):
    """Where the chains are many a workgroup takes 64 columns."""
    c = dc.inputs(*size, half, docs=docs)
    t = dc.tensors(c, half, layout, DEV)
    a = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    want, S = dc.oracle(c, size[4] ** -0.5)
    o, last = pr.delta_scan(*a, resets=t["resets"])
    dc.check(o, want, dc.FORWARD[half], "o")
    dc.check(last, S, dc.FORWARD[half], "last")
    out = pr.delta_scan_adjoint(*a, t["go"], g_last=t["g_last"], resets=t["resets"])
    check_gradients(out, dc.oracle(c, size[4] ** -0.5, True), half)


def test_no_gradients_given_and_empty():
    c = dc.inputs(1, 70, 1, 1, 16, 16, True)
    t = dc.tensors(c, True, "channel", DEV)
    args = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    out = pr.delta_scan_adjoint(*args, None)
    assert all(not bool(x.any()) for x in out.values())
    empty = [t[n][..., :0] for n in ("q", "k", "v", "beta", "log_decay")]
    o, last = pr.delta_scan(*empty, t["h0"])
    assert o.shape == (1, 1, 16, 0) and torch.equal(last, t["h0"])
    out = pr.delta_scan_adjoint(*empty, t["h0"], None, g_last=t["g_last"])
    assert torch.equal(out["dh0"], t["g_last"]) and out["dq"].shape == (1, 1, 16, 0)
    none = [t[n][:0] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    o, last = pr.delta_scan(*none)
    assert o.shape[0] == 0 and last.shape[0] == 0
    pr.delta_scan_adjoint(*none, o)


def test_repeats_bit_for_bit_and_leaves_the_rest_alone():
    c = dc.inputs(2, 333, 2, 4, 64, 48, True, docs=0.02)
    t = dc.tensors(c, True, "channel", DEV)
    args = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    wide = torch.full((2, 4, 50, 340), 7.0, device=DEV)
    out = wide[:, :, 1:49, 3:336]
    o, last = pr.delta_scan(*args, resets=t["resets"], out=out)
    again, last2 = pr.delta_scan(*args, resets=t["resets"])
    assert torch.equal(out, again) and torch.equal(last, last2)
    wide[:, :, 1:49, 3:336] = 7.0
    assert bool((wide == 7.0).all())
    g = [pr.delta_scan_adjoint(*args, t["go"], g_last=t["g_last"], resets=t["resets"]) for _ in range(2)]
    assert all(torch.equal(g[0][n], g[1][n]) for n in g[0])


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1), (3, 1, 2, 5, 3), (5, 2, 2, 64, 64), (4, 2, 4, 65, 70), (9, 1, 3, 128, 33),
                                  (2, 1, 1, 200, 130)])
def test_step(size, half):
    B, Hk, Hv, dk, dv = size
    c = dc.inputs(B, 1, Hk, Hv, dk, dv, half, decay="forget" if B > 4 else "mild")
    t = dc.tensors(c, half, "channel", DEV)
    r = np.random.default_rng(B)
    start = np.float32(r.standard_normal((B + 2, Hv, dk, dv)))
    slots = np.int32(r.permutation(B + 2)[:B])
    if B > 2:
        slots[1], slots[2] = -1, B + 2
    states = torch.from_numpy(start).to(DEV)
    args = [t[n][..., 0] for n in ("q", "k", "v", "beta", "log_decay")]
    o = pr.delta_step(*args, states, slots=torch.from_numpy(slots).to(DEV), scale=0.7)
    want, S = ref.delta_step(*[c[n][..., 0] for n in ("q", "k", "v", "beta", "log_decay")], start, slots, 0.7)
    # sums of up to 256 products in float32, 16 rows at a time
    dc.check(o, want, 2.0 ** -19, "o")
    dc.check(states, S, 2.0 ** -19, "states")
    untouched = [s for s in range(B + 2) if s not in slots.tolist()]
    assert torch.equal(states[untouched].cpu(), torch.from_numpy(start)[untouched])


def test_steps_follow_the_scan():
    """Token by token from the scan's state gives what the scan of all gives."""
    c = dc.inputs(2, 150, 2, 4, 32, 32, True)
    t = dc.tensors(c, True, "channel", DEV)
    q, k, v, beta, g, h0 = (t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0"))
    want, S = dc.oracle(c, 32 ** -0.5)
    states = pr.delta_scan(q[..., :100], k[..., :100], v[..., :100], beta[..., :100], g[..., :100], h0)[1]
    for i in range(100, 150):
        o = pr.delta_step(q[..., i], k[..., i], v[..., i], beta[..., i], g[..., i], states)
        dc.check(o, want[..., i], 2 * dc.FORWARD[True], i)
    dc.check(states, S, 2 * dc.FORWARD[True], "states")


@pytest.mark.parametrize("shared", [False, True])
def test_autograd(shared):
    """Gradients of a loss through the operator, a key head shared and the keys
    of all heads one expanded tensor."""
    c = dc.inputs(2, 90, 2, 4, 32, 16, False, docs=0.02)
    t = dc.tensors(c, False, "channel", DEV)
    if shared:
        c["k"] = np.broadcast_to(c["k"][:, :1], c["k"].shape)
    leaves = [t[n].detach().clone().requires_grad_(True) for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    q, k, v, beta, g, h0 = leaves
    used = k[:, :1].expand(-1, 2, -1, -1) if shared else k
    o, last = pag.delta_scan(q, used, v, beta.transpose(1, 2).contiguous().transpose(1, 2), g, h0, resets=t["resets"])
    ((o * t["go"]).sum() + (last * t["g_last"]).sum()).backward()
    want = dc.oracle(c, 32 ** -0.5, True)
    if shared:
        dk = want["dk"].sum(1, keepdims=True)
        want["dk"] = np.concatenate([dk, np.zeros_like(dk)], 1)
    for n, x in zip(("dq", "dk", "dv", "dbeta", "dlog_decay", "dh0"), leaves):
        dc.check(x.grad, want[n], 2 * dc.FORWARD[False], n)


def test_autograd_of_one_output():
    c = dc.inputs(1, 70, 1, 1, 16, 16, False)
    t = dc.tensors(c, False, "channel", DEV)
    leaves = [t[n].detach().clone().requires_grad_(True) for n in ("q", "k", "v", "beta", "log_decay")]
    o, last = pag.delta_scan(*leaves)
    last.sum().backward()  # an expanded gradient
    c |= dict(h0=None, go=np.zeros_like(c["go"]), g_last=np.ones_like(c["g_last"]))
    want = dc.oracle(c, 0.25, True)
    for n, x in zip(("dq", "dk", "dv", "dbeta", "dlog_decay"), leaves):
        dc.check(x.grad, want[n], 2 * dc.FORWARD[False], n)
    with pytest.raises(RuntimeError, match="twice"):
        o, _ = pag.delta_scan(*leaves)
        (g,) = torch.autograd.grad(o.sum(), leaves[0], create_graph=True)
        g.sum().backward()
