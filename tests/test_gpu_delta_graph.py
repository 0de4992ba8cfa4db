"""The gated delta rule, the distillation and the logits before sampling in HIP
graphs, on other streams, by several threads, and together as a model uses them."""
import threading

import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import autograd as pag
from nonlinear_rnn_amd import pararnn as pr
from oracle import delta as ref
from tests import delta_cases as dc
from tests.gpu_util import DEV
from tests.test_gpu_graph import capture, eager_noise, flat

pytestmark = pytest.mark.gpu


def scan_case(B=2, T=300, Hk=2, Hv=4, dk=40, dv=50, half=True, layout="channel"):
    c = dc.inputs(B, T, Hk, Hv, dk, dv, half, docs=0.01)
    t = dc.tensors(c, half, layout, DEV)
    a = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]

    def fn():
        o, last = pr.delta_scan(*a, resets=t["resets"])
        return o, last, pr.delta_scan_adjoint(*a, t["go"], g_last=t["g_last"], resets=t["resets"])
    return fn, a


def segments_case():
    return scan_case(1, 2500, 1, 2, 64, 32, False, "time")  # chained in segments


def step_case():
    c = dc.inputs(5, 1, 2, 4, 64, 70, True)
    t = dc.tensors(c, True, "channel", DEV)
    a = [t[n][..., 0] for n in ("q", "k", "v", "beta", "log_decay")]
    start = torch.randn((9, 4, 64, 70), device=DEV)
    states, slots = start.clone(), torch.tensor([8, 0, -1, 3, 5], dtype=torch.int32, device=DEV)

    def fn():
        states.copy_(start)
        return pr.delta_step(*a, states, slots=slots), states.clone()
    return fn, a[:3]


def logits_case():
    x = torch.randn((3, 40000), device=DEV)  # rows in parts
    own = pr.token_logprobs(torch.randn((3, 40000), device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV), top=9)
    index, logprob = own["top_index"], own["top_logprob"]
    g = torch.randn(3, device=DEV)
    tokens = torch.randint(0, 40000, (3, 500), device=DEV)
    rep, freq = torch.full((3,), 1.3, device=DEV), torch.full((3,), 0.2, device=DEV)
    bias = (torch.randint(0, 40000, (3, 7), device=DEV), torch.randn((3, 7), device=DEV))
    allowed = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, 1250), device=DEV).int()

    def fn():
        out = pr.distill_top(x, index, logprob)
        return (out, pr.distill_top_adjoint(x, index, logprob, out["lse"], out["log_rest"], g),
                pr.adjust_logits(x, tokens=tokens, repetition=rep, frequency=freq, bias=bias, allowed=allowed))
    return fn, [x]


CASES = [scan_case, segments_case, step_case, logits_case]


@pytest.mark.parametrize("case", CASES)
def test_replays(case):
    """Each replay bitwise the eager result, also after the inputs change."""
    fn, inputs = case()
    graph, out = capture(fn)
    for i in range(4):
        if i == 2:
            for p in inputs:
                p.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in flat(out)]
        eager_noise()
        want = flat(fn())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


@pytest.mark.parametrize("case", [scan_case, segments_case, logits_case])
def test_graphs_own_their_workspaces(case, monkeypatch):
    used = []
    get = pr.Workspace.get

    def spy(self, *a, **k):
        b = get(self, *a, **k)
        if b is not None:
            used.append(b.data_ptr())
        return b
    monkeypatch.setattr(pr.Workspace, "get", spy)
    fn, _ = case()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = [t.clone() for t in flat(fn())]
    s.synchronize()
    eager, graphs = set(used), []
    for _ in range(2):
        used.clear()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = fn()
        graphs.append((g, out, set(used)))
    assert not graphs[0][2] & graphs[1][2] and not eager & (graphs[0][2] | graphs[1][2])
    for _ in range(3):
        for g, out, _ in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(flat(out), want))
        fn()


@pytest.mark.parametrize("case", [scan_case, segments_case, logits_case])
def test_streams_and_threads(case):
    """On a stream of its own, and by threads on one stream: what one call by
    itself gives."""
    calls = [case()[0] for _ in range(3)]
    want = [[t.clone() for t in flat(fn())] for fn in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for fn, s in zip(calls, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(flat(fn()))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    wrong = []

    def run(i):
        for _ in range(5):
            out = flat(calls[i]())
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(out, want[i])):
                wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_the_streams_argument_and_a_workspace_of_the_callers():
    c = dc.inputs(1, 200, 1, 2, 32, 32, True)
    t = dc.tensors(c, True, "channel", DEV)
    a = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    want = pr.delta_scan(*a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want[0])
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)  # NaN wherever it is read first
    torch.cuda.synchronize()
    got = pr.delta_scan(*a, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(got[1], want[1])
    want = pr.delta_scan_adjoint(*a, t["go"])
    got = pr.delta_scan_adjoint(*a, t["go"], workspace=torch.full((1 << 23,), 255, dtype=torch.uint8, device=DEV))
    assert all(torch.equal(got[n], want[n]) for n in want)
    with pytest.raises(RuntimeError):
        pr.delta_scan(*a, workspace=ws[:64])


def test_a_training_step_is_captured():
    """Scan, loss and both backward passes in one graph; each replay gives the
    eager gradients."""
    c = dc.inputs(2, 130, 1, 2, 32, 48, True)
    t = dc.tensors(c, True, "channel", DEV)
    leaves = [t[n].detach().clone().requires_grad_(True) for n in ("q", "k", "v", "beta", "log_decay")]
    head = torch.randn((96, 300), device=DEV).mul_(0.1).requires_grad_(True)
    own = pr.token_logprobs(torch.randn((260, 300), device=DEV), torch.zeros(260, dtype=torch.int64, device=DEV), top=5)

    def loss():
        o, _ = pag.delta_scan(*leaves)
        logits = o.flatten(1, 2).transpose(1, 2).reshape(260, 96) @ head
        return pag.distill_top(logits, own["top_index"], own["top_logprob"])["loss"].sum()
    want = torch.autograd.grad(loss(), leaves + [head])
    graph, got = capture(lambda: torch.autograd.grad(loss(), leaves + [head]))
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        eager_noise()


def test_a_capture_beside_an_eager_graph_of_the_same_leaves_is_refused():
    c = dc.inputs(1, 64, 1, 1, 16, 16, True)
    t = dc.tensors(c, True, "channel", DEV)
    leaves = [t[n].detach().clone().requires_grad_(True) for n in ("q", "k", "v", "beta", "log_decay")]
    x = torch.randn((4, 50), device=DEV, requires_grad=True)
    index, logprob = torch.zeros((4, 1), dtype=torch.int64, device=DEV), torch.full((4, 1), -1.0, device=DEV)
    alive = pag.delta_scan(*leaves)[0], pag.distill_top(x, index, logprob)["loss"]
    for fn in (lambda: pag.delta_scan(*leaves)[0], lambda: pag.distill_top(x, index, logprob)["loss"]):
        with pytest.raises(RuntimeError, match="eager graph"):
            capture(fn)
        torch.cuda.synchronize()
    with torch.no_grad():  # nothing is recorded, so nothing is in the way
        graph, out = capture(lambda: (pag.delta_scan(*leaves)[0], pag.distill_top(x, index, logprob)["loss"]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], alive[0]) and torch.equal(out[1], alive[1])
    (alive[0].sum() + alive[1].sum()).backward()  # the eager graph is as it was
    assert all(p.grad is not None and bool(p.grad.isfinite().all()) for p in leaves + [x])


def test_together_a_block_and_its_teacher():
    """A block of a model (scan, norm, projection) and the distillation of its
    logits from another's, against plain float64 mathematics."""
    B, T, H, dk, dv, V = 2, 70, 2, 32, 32, 120
    D = H * dv
    c = dc.inputs(B, T, H, H, dk, dv, True, docs=0.03)
    t = dc.tensors(c, True, "channel", DEV)
    r = np.random.default_rng(3)
    x = torch.from_numpy(r.standard_normal((B, T, D))).float().to(DEV)
    w_post, w_pre = (torch.from_numpy(1 + 0.1 * r.standard_normal(D)).float().to(DEV) for _ in range(2))
    head = torch.from_numpy(r.standard_normal((D, V)) / D ** 0.5).float().to(DEV)
    own = pr.token_logprobs(torch.from_numpy(r.standard_normal((B * T, V))).float().to(DEV),
                            torch.zeros(B * T, dtype=torch.int64, device=DEV), top=6)
    leaves = [t[n].detach().clone().requires_grad_(True) for n in ("q", "k", "v", "beta", "log_decay")]
    o, _ = pag.delta_scan(*leaves, t["h0"], resets=t["resets"])
    y, z = pag.block_norm(o.flatten(1, 2), x, w_post, w_pre, z_dtype=torch.float32)
    out = pag.distill_top(z.reshape(B * T, D) @ head, own["top_index"], own["top_logprob"])
    out["loss"].sum().backward()

    d = {n: leaf.detach().double().cpu().requires_grad_(True) for n, leaf in zip(("q", "k", "v", "beta", "g"), leaves)}
    want = plain(d, t["h0"].double().cpu(), t["resets"].cpu(), dk ** -0.5)
    h = want.flatten(1, 2).transpose(1, 2)
    norm = lambda u, w: u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-6) * w.double().cpu()
    zz = norm(x.double().cpu() + norm(h, w_post), w_pre)
    logq = torch.log_softmax(zz.reshape(B * T, D) @ head.double().cpu(), -1)
    index, p = own["top_index"].cpu(), own["top_logprob"].double().cpu().exp()
    rest = torch.log(1 - logq.exp().gather(1, index).sum(1))
    left = 1 - p.sum(1)
    loss = (p * (p.log() - logq.gather(1, index))).sum(1) + left * (left.log() - rest)
    loss.sum().backward()
    # the scan's tolerance, and as much for the steps behind it, which are float32 but
    # for the head's product, of 64 terms as well
    tol = 4 * dc.FORWARD[True]
    dc.check(out["loss"].detach(), loss.detach().numpy(), tol, "loss")
    for n, leaf in zip(("q", "k", "v"), leaves):  # rounded to bfloat16: half a step is 2^-8
        dc.check(leaf.grad, d[n].grad.numpy(), 2 * tol + 2.0 ** -8, n)
    for n, leaf in zip(("beta", "g"), leaves[3:]):
        dc.check(leaf.grad, d[n].grad.numpy(), 2 * tol, n)


def plain(d, h0, resets, scale):
    """The recurrence step by step, for autograd."""
    S, out = h0, []
    for i in range(d["q"].shape[-1]):
        q, k, v = (d[n][..., i] for n in ("q", "k", "v"))
        S = torch.where(resets[:, i, None, None, None], 0.0, S * d["g"][..., i, None, None].exp())
        w = d["beta"][..., i, None] * (v - torch.einsum("bhk,bhkv->bhv", k, S))
        S = S + k[..., None] * w[..., None, :]
        out.append(scale * torch.einsum("bhk,bhkv->bhv", q, S))
    return torch.stack(out, -1)


def test_together_generating():
    """Token by token with states in a pool: step, norm, head, logits adjusted,
    the most likely token; captured, with the history written by the graph."""
    B, H, dk, dv, V, L = 3, 2, 64, 64, 500, 12
    D = H * dv
    gen = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *s: torch.randn(s, device=DEV, generator=gen)
    table, head = rand(V, D), rand(D, V) / D ** 0.5
    maps = [rand(D, H * dk) / D ** 0.5, rand(D, H * dk) / D ** 0.5, rand(D, D) / D ** 0.5]
    w = torch.ones(D, device=DEV)
    states = torch.zeros((B + 2, H, dk, dv), device=DEV)
    slots = torch.tensor([4, 1, 2], dtype=torch.int32, device=DEV)
    history, lengths = torch.zeros((B, L + 1), dtype=torch.int64, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
    rep, prompt = torch.full((B,), 1e6, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
    presence = torch.full((B,), 1e4, device=DEV)
    allowed = torch.full((1, (V + 31) // 32), -1, dtype=torch.int32, device=DEV)
    allowed[0, 0] = 0  # the first 32 tokens are not to be said
    rows = torch.zeros(B, dtype=torch.int32, device=DEV)

    def token():
        x = table[history.gather(1, (lengths - 1).long()[:, None])[:, 0]]
        q, k = (torch.nn.functional.normalize((x @ m).view(B, H, dk), dim=-1).bfloat16() for m in maps[:2])
        v = (x @ maps[2]).view(B, H, dv).bfloat16()
        o = pr.delta_step(q, k, v, torch.full((B, H), 0.5, device=DEV), torch.full((B, H), -0.1, device=DEV), states,
                          slots=slots)
        z = pr.block_norm(o.flatten(1)[:, :, None], x[:, None], w, w, z_dtype=torch.float32)[1]
        logits = pr.adjust_logits(z[:, 0] @ head, tokens=history, lengths=lengths, prompt=prompt, repetition=rep,
                                  presence=presence, allowed=allowed, allowed_rows=rows)
        best = pr.token_logprobs(logits, history[:, 0].contiguous(), top=1)["top_index"][:, 0]
        history.scatter_(1, lengths.long()[:, None], best[:, None])
        lengths.add_(1)
        return logits

    def restart():
        states.zero_(), history.zero_(), lengths.fill_(1)
    for _ in range(L):
        token()
    want = history.clone()
    said = want[:, 1:].cpu().numpy()
    assert (said >= 32).all() and (said < V).all()
    assert all(len(set(row)) == L for row in said)  # what was said is not said again
    assert not states[0].any() and not states[3].any() and states[4].any()
    restart()
    graph, _ = capture(lambda: token())
    restart()
    for _ in range(L):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(history, want)


@pytest.mark.parametrize("name", ["q", "v", "o"])
def test_offsets_past_32_bits(name):
    """Two rows whose places are more than 2^32 elements apart."""
    far = 2 ** 32 + 64
    c = dc.inputs(2, 70, 1, 1, 16, 16, True)
    t = dc.tensors(c, True, "channel", DEV)
    a = [t[n] for n in ("q", "k", "v", "beta", "log_decay", "h0")]
    want = pr.delta_scan(*a)
    where = {"q": 0, "v": 2}.get(name)
    dtype = torch.float32 if name == "o" else torch.bfloat16
    room = torch.empty(far + 16 * 70, dtype=dtype, device=DEV)
    apart = torch.as_strided(room, (2, 1, 16, 70), (far, 1120, 70, 1))
    if where is None:
        got = pr.delta_scan(*a, out=apart)
    else:
        apart.copy_(a[where])
        a[where] = apart
        got = pr.delta_scan(*a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
