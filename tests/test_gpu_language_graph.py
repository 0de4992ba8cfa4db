"""The operators of language models in a HIP graph: captured once, replayed with
eager work between, each replay bitwise the eager result, also after the inputs
change in place."""
import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr
from tests.gpu_util import DEV
from tests.test_gpu_graph import capture, eager_noise, flat

pytestmark = pytest.mark.gpu


def scan_case():
    u = [torch.randn((2, 40, 9000), device=DEV).bfloat16() for _ in range(3)]  # several spans
    lam, h0, gh = torch.randn(40, device=DEV), torch.randn((2, 40), device=DEV), torch.randn((2, 40, 9000), device=DEV)

    def fn():
        h, last = pr.gated_scan(u, lam, h0)
        return h, last, pr.gated_scan_adjoint(u, lam, h0, h, gh)
    return fn, u


def time_major_scan_case():
    u = [torch.randn((2, 2000, 70), device=DEV).transpose(1, 2) for _ in range(3)]  # several chunks
    lam, h0 = torch.randn(70, device=DEV), torch.randn((2, 70), device=DEV)
    gh = torch.randn((2, 2000, 70), device=DEV).transpose(1, 2)

    def fn():
        h, last = pr.gated_scan(u, lam, h0)
        return h, last, pr.gated_scan_adjoint(u, lam, h0, h, gh)
    return fn, u


def step_case():
    u = [torch.randn((5, 300), device=DEV) for _ in range(3)]
    lam, start = torch.randn(300, device=DEV), torch.randn((9, 300), device=DEV)
    states, slots = start.clone(), torch.tensor([8, 0, -1, 3, 5], dtype=torch.int32, device=DEV)

    def fn():
        states.copy_(start)
        return pr.gated_step(u, lam, states, slots=slots), states.clone()
    return fn, u


def block_case():
    h, gate = torch.randn((2, 500, 70), device=DEV), torch.randn((2, 500, 70), device=DEV).bfloat16()
    x, gy = torch.randn((2, 70, 500), device=DEV), torch.randn((2, 70, 500), device=DEV)
    w = torch.rand(500, device=DEV) + 0.5
    gz = torch.randn((2, 70, 500), device=DEV).bfloat16()

    def fn():
        y, z, rstd = pr.block_norm(h, x, w, w, gate=gate)
        return y, z, rstd, pr.block_norm_adjoint(h, x, w, w, rstd, gy, gz, gate=gate)
    return fn, [h, gate, x]


def score_case():
    x = torch.randn((3, 30000), device=DEV)  # rows in parts
    tokens, g = torch.tensor([5, -1, 29999], device=DEV), torch.randn(3, device=DEV)

    def fn():
        out = pr.token_logprobs(x, tokens, top=7)
        return out, pr.token_logprobs_adjoint(x, tokens, out["lse"], out["entropy"], g_logprob=g, g_entropy=g)
    return fn, [x]


@pytest.mark.parametrize("case", [scan_case, time_major_scan_case, step_case, block_case, score_case])
def test_replays(case):
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
