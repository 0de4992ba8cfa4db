"""The binding's memory, on the CPU.  Who shares a workspace: several launches of
one call meet in it, so no other call's launches may come between them.  And
what gradients take up."""
import contextlib
import threading

import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture(autouse=True)
def no_streams(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())


def test_threads_do_not_share_a_workspace():
    """Threads on one stream: each keeps a buffer of its own, also where one has
    to grow, and a thread's many streams push out none of another's."""
    ws = pr.Workspace()
    got = {}

    def use(name, sizes):
        got[name] = [ws.get(n, "cpu", Stream(1)) for n in sizes]
    use("here", [64, 32])
    assert got["here"][0] is got["here"][1]

    def elsewhere():
        use("there", [64, 128])
        for h in range(2, 2 + 2 * pr.Workspace.MAX_STREAMS):
            ws.get(16, "cpu", Stream(h))
    thread = threading.Thread(target=elsewhere)
    thread.start()
    thread.join()
    assert not {b.data_ptr() for b in got["here"]} & {b.data_ptr() for b in got["there"]}
    assert ws.get(64, "cpu", Stream(1)) is got["here"][0]



def test_a_captured_call_has_a_workspace_of_its_own(monkeypatch):
    """A graph's launches keep their workspace for as long as it is replayed: it
    is neither taken from the buffers that other calls use nor left among them."""
    ws = pr.Workspace()
    cached = ws.get(64, "cpu", Stream(1))
    monkeypatch.setattr(pr, "_capturing", lambda device, stream: True)
    first, second = ws.get(64, "cpu", Stream(1)), ws.get(64, "cpu", Stream(1))
    other = ws.get(64, "cpu", Stream(2))
    assert len({b.data_ptr() for b in (cached, first, second, other)}) == 4
    assert list(ws.buf) == [(None, 1)] and ws.buf[(None, 1)] is cached
    monkeypatch.setattr(pr, "_capturing", lambda device, stream: False)
    assert ws.get(64, "cpu", Stream(1)) is cached


def gate_slices(B, D, T, gates, layout):
    u = torch.zeros((B, gates * D, T) if layout == "channel" else (B, T, gates * D))
    u = u if layout == "channel" else u.transpose(1, 2)
    return [u[:, g * D:(g + 1) * D] for g in range(3)]


@pytest.mark.parametrize("layout", ["channel", "time"])
@pytest.mark.parametrize("B,D,T,gates", [(7, 5, 6, 4), (7, 5, 6, 3), (1, 5, 6, 4), (2, 1, 6, 4), (4, 5, 1, 4), (1, 1, 1, 3)])
def test_gradients_of_gates_take_up_what_the_gates_do(B, D, T, gates, layout):
    """Gates that are slices of one projection: their gradients have the slices'
    strides, no element in common, and together no more room than the projection."""
    u = gate_slices(B, D, T, gates, layout)
    du = pr._gradient_planes(3, (B, D, T), u[0].stride(), torch.float32, "cpu")
    for g, p in enumerate(du):
        assert p.shape == (B, D, T) and p.stride() == u[0].stride()
        p.fill_(float(g))
    assert all(bool((p == g).all()) for g, p in enumerate(du))
    room = {p.untyped_storage().data_ptr(): p.untyped_storage().nbytes() for p in du}
    assert sum(room.values()) <= 4 * B * gates * D * T


@pytest.mark.parametrize("strides", [(30, 6, 1), (48, 8, 1), (1, 8, 48), (30, 1, 5), (36, 1, 6), (90, 1, 17)])
def test_gradients_of_other_planes_have_no_element_in_common(strides):
    dims = (8, 5, 6)
    du = pr._gradient_planes(3, dims, strides, torch.float32, "cpu")
    for g, p in enumerate(du):
        assert p.shape == dims and p.stride() == strides
        p.fill_(float(g))
    assert all(bool((p == g).all()) for g, p in enumerate(du))


def adjoint(**kw):
    u = gate_slices(2, 3, 5, 4, "channel")
    pr.gated_scan_adjoint(u, torch.zeros(3), None, torch.zeros(2, 3, 5), None, **kw)


def block_adjoint(gate=torch.zeros(2, 3, 5), **kw):
    pr.block_norm_adjoint(torch.zeros(2, 3, 5), torch.zeros(2, 5, 3), torch.ones(3), torch.ones(3),
                          torch.ones(2, 2, 5), None, None, gate=gate, **kw)


@pytest.mark.parametrize("call,message", [
    (lambda: adjoint(du=gate_slices(2, 3, 5, 4, "channel")[:2]), "du"),
    (lambda: adjoint(du=gate_slices(2, 3, 5, 3, "channel")), "du"),
    (lambda: adjoint(du=[p.double() for p in gate_slices(2, 3, 5, 4, "channel")]), "du"),
    (lambda: adjoint(du=[1, 2, 3]), "du"),
    (lambda: adjoint(du=gate_slices(2, 3, 5, 4, "channel")), "GPU"),
    (lambda: block_adjoint(dgate=torch.zeros(2, 3, 6)), "dgate"),
    (lambda: block_adjoint(dgate=torch.zeros(2, 3, 5).bfloat16()), "dgate"),
    (lambda: block_adjoint(dgate=torch.zeros(2, 5, 3).transpose(1, 2)), "dgate"),
    (lambda: block_adjoint(gate=None, dgate=torch.zeros(2, 3, 5)), "dgate"),
    (lambda: block_adjoint(dgate=torch.zeros(2, 3, 5)), "GPU"),
])
def test_gradients_to_write_to_are_checked(call, message):
    for _ in range(2):
        with pytest.raises(ValueError, match=message):
            call()
