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
