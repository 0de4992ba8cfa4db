"""Workspaces on the GPU: graphs own theirs, and threads do not meet in one."""
import threading

import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr
from tests.gpu_util import DEV
from tests.test_gpu_language_graph import scan_case, score_case, time_major_scan_case

pytestmark = pytest.mark.gpu


def flat(x):
    if isinstance(x, torch.Tensor):
        return [x]
    return [t for v in (x.values() if isinstance(x, dict) else x) for t in flat(v)]


@pytest.mark.parametrize("case", [scan_case, time_major_scan_case, score_case])
def test_graphs_own_their_workspaces(case, monkeypatch):
    """Two graphs of the same calls, captured on the stream they were warmed up
    on.  Neither shares a workspace with the other or with eager calls, and when
    the eager calls' buffer has grown, what is allocated in its place is not
    written by a replay."""
    used = []
    get = pr.Workspace.get

    def spy(self, *a, **k):
        b = get(self, *a, **k)
        if b is not None:
            used.append(b.data_ptr())
        return b
    monkeypatch.setattr(pr.Workspace, "get", spy)
    fn, inputs = case()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = [t.clone() for t in flat(fn())]
    s.synchronize()
    eager = set(used)
    graphs = []
    for _ in range(2):
        used.clear()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = fn()
        graphs.append((g, out, set(used)))
    assert not graphs[0][2] & graphs[1][2] and not eager & (graphs[0][2] | graphs[1][2])
    size = sum(b.numel() for b in pr._ws.buf.values())
    with torch.cuda.stream(s):
        pr._ws.get(4 * size, torch.device(DEV))  # grows: the old buffer goes back to the allocator
        live = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in (size, size // 2, 512) * 8]
    s.synchronize()
    for _ in range(3):
        for g, out, _ in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(flat(out), want))
    assert all(bool((t == 7).all()) for t in live)


@pytest.mark.parametrize("case", [scan_case, time_major_scan_case, score_case])
def test_threads_on_one_stream(case):
    """Threads that call on the same stream get what one gets by itself."""
    calls = [case()[0] for _ in range(4)]
    want = [[t.clone() for t in flat(fn())] for fn in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        for _ in range(20):
            out = flat(calls[i]())
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(out, want[i])):
                wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
