"""Who shares a workspace, on the CPU: several launches of one call meet in it,
so no other call's launches may come between them."""
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
