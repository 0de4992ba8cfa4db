"""The gated recurrence and the gradient of the token scores on the GPU, every
element within its own bound (language_bounds.py; that the bounds reject zeros,
missing pieces and missing terms at these sizes is tested on the CPU)."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr
from tests import language_bounds as lb
from tests.gpu_util import DEV
from tests.test_language_bounds import SCANS, SCORES, scan_case

pytestmark = pytest.mark.gpu


def dev(x, half=False):
    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return t if t.dtype == torch.bool else t.to(torch.bfloat16 if half else torch.float32)


def plane(x, layout, half=False):
    t = dev(x, half)
    return t if layout == "channel" else t.transpose(1, 2).contiguous().transpose(1, 2)


def f64(t):
    return t.double().cpu().numpy()


def inside(got, want, tol, what):
    bad = lb.outside(f64(got), want, tol)
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(f64(got) - want) / tol).max()))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("layout", ["channel", "time"])
@pytest.mark.parametrize("B,T,D", sorted({c[:3] for c in SCANS}))
def test_scan(B, T, D, layout, half):
    c = scan_case(B, T, D, half)
    u = [plane(p, layout, half) for p in c["u"]]
    lam, h0, resets, gl = (dev(c[k]) for k in ("lam", "h0", "resets", "gl"))
    h, last = pr.gated_scan(u, lam, h0, power=c["power"], resets=resets)
    want, tol = lb.scan(c)
    inside(h, want, tol, "h")
    assert torch.equal(last, h[..., -1].contiguous())
    gh = torch.empty_strided(h.shape, h.stride(), device=DEV).copy_(dev(c["gh"]))
    got = pr.gated_scan_adjoint(u, lam, h0, h, gh, gh_last=gl, power=c["power"], resets=resets)
    want, tol = lb.scan_adjoint(c, f64(h), layout, half)
    for g, name in enumerate("rix"):
        inside(got["du"][g], want["du"][g], tol["du"][g], "du_" + name)
    inside(got["dh0"], want["dh0"], tol["dh0"], "dh0")
    inside(got["dlam"], want["dlam"], tol["dlam"], "dlam")


@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("N,V,masked", SCORES)
def test_score_adjoint(N, V, masked, half, scale):
    c = lb.score_inputs(N, V, half, masked)
    x, tokens = dev(c["x"], half), torch.from_numpy(c["tokens"]).to(DEV)
    out = pr.token_logprobs(x, tokens, scale=scale)
    g = [dev(v) for v in c["g"]]
    got = pr.token_logprobs_adjoint(x, tokens, out["lse"], out["entropy"], g_logprob=g[0], g_entropy=g[1],
                                    g_lse=g[2], scale=scale)
    want, tol = lb.score_adjoint(c, scale, half)
    inside(got, want, tol, "dlogits")
