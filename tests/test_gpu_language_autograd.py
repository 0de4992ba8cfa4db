"""The differentiable forms of the operators of language models, as a training
program uses their results: edited in place, differentiated once, on slices of
one projection."""
import pytest
import torch

from nonlinear_rnn_amd import autograd as pag
from nonlinear_rnn_amd import pararnn as pr
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def scores(**kw):
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.randn((5, 300), generator=g, device=DEV)
    tokens = torch.tensor([3, -1, 7, 299, 0], device=DEV)
    return x.requires_grad_(True), tokens


@pytest.mark.parametrize("edit", ["mul_", "masked_fill_"])
def test_log_probabilities_may_be_edited_in_place(edit):
    """Masking a loss in place, with the other outputs in it too."""
    mask = torch.tensor([True, False, False, True, False], device=DEV)
    grads = []
    for in_place in (False, True):
        x, tokens = scores()
        out = pag.token_logprobs(x, tokens)
        lp = out["logprob"]
        if in_place:
            lp.mul_(~mask) if edit == "mul_" else lp.masked_fill_(mask, 0.0)
        else:
            lp = lp * ~mask
        (lp.sum() + out["entropy"].sum() + out["lse"].sum()).backward()
        grads.append(x.grad)
    assert torch.equal(*grads)


def test_outputs_of_a_score_are_tensors_of_their_own():
    x, tokens = scores()
    out = pr.token_logprobs(x.detach(), tokens, top=2)
    before = {k: v.clone() for k, v in out.items()}
    versions = {k: v._version for k, v in out.items()}
    out["logprob"].fill_(7.0)
    for k in ("entropy", "lse", "top_index", "top_logprob"):
        assert torch.equal(out[k], before[k]) and out[k]._version == versions[k]


def second_derivative(loss, leaf):
    (first,) = torch.autograd.grad(loss, leaf, create_graph=True)
    (first.square().sum() + leaf.square().sum()).backward()


def test_a_second_derivative_is_refused():
    """Not left out: with a penalty on the gradient, the part that goes through the
    operator would be missing."""
    x, tokens = scores()
    with pytest.raises(RuntimeError, match="differentiate twice"):
        second_derivative(pag.token_logprobs(x, tokens)["logprob"].sum(), x)
    u = [torch.randn((2, 3, 20), device=DEV, requires_grad=True) for _ in range(3)]
    with pytest.raises(RuntimeError, match="differentiate twice"):
        second_derivative(pag.gated_scan(u, torch.randn(3, device=DEV))[0].square().sum(), u[0])
    x = torch.randn((2, 5, 8), device=DEV, requires_grad=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        second_derivative(pag.block_norm(None, x, None, torch.ones(8, device=DEV))[1].square().sum(), x)


@pytest.mark.parametrize("layout", ["channel", "time"])
def test_gradients_of_one_projection(layout):
    """Gates that are slices of one projection: gradients next to each other, or
    written to the slices of one tensor, are those of separate planes."""
    B, D, T = 3, 20, 70
    u = torch.randn((B, 4 * D, T) if layout == "channel" else (B, T, 4 * D), device=DEV)
    du = torch.empty_like(u)
    u, du = (p if layout == "channel" else p.transpose(1, 2) for p in (u, du))
    gates, dgates = ([p[:, g * D:(g + 1) * D] for g in range(4)] for p in (u, du))
    lam, x = torch.randn(D, device=DEV), torch.randn((B, T, D), device=DEV)
    w = torch.rand(D, device=DEV) + 0.5
    h, _ = pr.gated_scan(gates[:3], lam)
    _, _, rstd = pr.block_norm(h, x, w, w, gate=gates[3])
    gh, gy = torch.empty_strided(h.shape, h.stride(), device=DEV).normal_(), torch.randn_like(x)
    one = pr.gated_scan_adjoint(gates[:3], lam, None, h, gh)
    two = pr.gated_scan_adjoint([p.clone(memory_format=torch.contiguous_format) for p in gates[:3]], lam, None,
                                h.contiguous(), gh.contiguous()) if layout == "channel" else one
    into = pr.gated_scan_adjoint(gates[:3], lam, None, h, gh, du=dgates[:3])
    for a, b, c, d in zip(one["du"], two["du"], into["du"], dgates):
        assert torch.equal(a, b) and torch.equal(a, c) and c.data_ptr() == d.data_ptr()
    kw = dict(gate=gates[3])
    new = pr.block_norm_adjoint(h, x, w, w, rstd, gy, None, **kw)
    into = pr.block_norm_adjoint(h, x, w, w, rstd, gy, None, dgate=dgates[3], **kw)
    assert into["dgate"].data_ptr() == dgates[3].data_ptr() and torch.equal(dgates[3], new["dgate"])
    assert all(torch.equal(a, b) for a, b in zip(one["du"], dgates))  # and nothing of its neighbours
