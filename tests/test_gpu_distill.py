"""Distillation from top tokens on the GPU: every element within a bound of the
float64 oracle, at the sizes, lists and masks where it can go wrong."""
import math

import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import autograd as pag
from nonlinear_rnn_amd import pararnn as pr
from oracle import logits as ref
from tests import distill_bounds as bounds
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def case(N, V, k, half, masked=0.0, seed=0, full=False):
    """A student and the list of a teacher that agrees in part; row 1 has no
    entry, row 2 one twice, row 3 allows only two tokens, which the list holds."""
    r = np.random.default_rng(seed + 31 * V + N)
    x = torch.from_numpy(np.float32(2.5 * r.standard_normal((N, V)) + r.standard_normal((N, 1))))
    x = (x.bfloat16() if half else x).double().numpy()
    x[r.random((N, V)) < masked] = -np.inf
    if N > 3 and V > 4:
        x[3] = -np.inf
        x[3, [1, 4]] = 0.5
    t = 0.8 * x + 1.5 * r.standard_normal((N, V))
    with np.errstate(invalid="ignore"):
        t = t - np.max(t, 1, keepdims=True)
        t = np.float32(t - np.log(np.exp(t).sum(1, keepdims=True)))
    index = np.argsort(-t, 1, kind="stable")[:, :min(k, V)]
    lp = np.take_along_axis(t, index, 1)
    index = np.where(np.isfinite(lp), index, -1)
    if k > V:
        index = np.concatenate([index, np.full((N, k - V), -1)], 1)
        lp = np.concatenate([lp, np.full((N, k - V), -np.inf, np.float32)], 1)
    if N > 1:
        index[1] = -1
    if N > 2 and k > 2:
        index[2, 2] = index[2, 0]
        lp[2] -= np.float32(0.5)  # the probabilities still sum to less than one
    return dict(x=x, index=index.astype(np.int64), logprob=lp.astype(np.float64))


def put(c, half):
    return (torch.from_numpy(c["x"]).to(torch.bfloat16 if half else torch.float32).to(DEV),
            torch.from_numpy(c["index"]).to(DEV), torch.from_numpy(c["logprob"]).float().to(DEV))


def close(got, want, tol, what):
    got = got.double().cpu().numpy()
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - want) <= tol)
    assert ok.all(), (what, np.argwhere(~ok)[:5].tolist(), got[~ok][:5], want[~ok][:5])


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("N,V,k,masked", [(1, 1, 1, 0.0), (5, 3, 2, 0.0), (5, 7, 9, 0.0), (4, 100, 5, 0.5), (7, 1001, 20, 0.0),
                                          (3, 4096, 64, 0.6), (2, 8193, 1, 0.0), (5, 50003, 300, 0.3),
                                          (1300, 257, 7, 0.1), (2, 140001, 1024, 0.0)])
def test_loss_and_gradient(N, V, k, masked, tail, half):
    c = case(N, V, k, half, masked)
    x, index, lp = put(c, half)
    out = pr.distill_top(x, index, lp, tail=tail, scale=0.8)
    want, tol = bounds.loss(c, tail, 0.8)
    for name in want:
        close(out[name], want[name], tol[name], name)
    g = np.float32(np.random.default_rng(1).standard_normal(N)).astype(np.float64)
    want, tol = bounds.gradient(c, g, tail, 0.8, half)
    args = (x, index, lp, out["lse"], out["log_rest"], torch.from_numpy(g).float().to(DEV))
    grad = pr.distill_top_adjoint(*args, tail=tail, scale=0.8)
    close(grad, want, tol, "gradient")
    again = pr.distill_top(x, index, lp, tail=tail, scale=0.8)
    assert all(torch.equal(out[n], again[n]) for n in out)
    inplace = pr.distill_top_adjoint(*args, tail=tail, scale=0.8, out=x)
    assert inplace.data_ptr() == x.data_ptr() and torch.equal(inplace, grad)


def test_rows_that_are_apart():
    c = case(6, 1000, 8, True)
    x, index, lp = put(c, True)
    wide = torch.zeros((6, 1013), dtype=torch.bfloat16, device=DEV)
    wide[:, 5:1005] = x
    out = torch.full((6, 1021), 7.0, dtype=torch.bfloat16, device=DEV)
    a, b = pr.distill_top(x, index, lp), pr.distill_top(wide[:, 5:1005], index, lp)
    close(b["loss"], a["loss"].double().cpu().numpy(), 1e-5, "loss")
    g = torch.rand(6, device=DEV)
    got = pr.distill_top_adjoint(wide[:, 5:1005], index, lp, a["lse"], a["log_rest"], g, out=out[:, 3:1003])
    assert torch.equal(got, pr.distill_top_adjoint(x, index, lp, a["lse"], a["log_rest"], g))
    out[:, 3:1003] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("half", [True, False])
def test_edges(half):
    """Rows that allow nothing, listed tokens that are masked, indices past the
    vocabulary, NaN and infinite logits: each stays in its row."""
    c = case(8, 300, 4, half)
    c["x"][4] = -np.inf
    c["x"][5, c["index"][5, 0]] = -np.inf
    c["index"][6, 1] = 300
    x, index, lp = put(c, half)
    x[7, 17] = float("nan")
    out = pr.distill_top(x, index, lp)
    want, tol = bounds.loss({**c, "x": np.where(np.arange(8)[:, None] == 7, 0.0, c["x"])}, True)
    loss = out["loss"].cpu().numpy()
    assert math.isinf(loss[4]) and math.isinf(loss[5]) and math.isnan(loss[6]) and math.isnan(loss[7])
    keep = [0, 1, 2, 3]
    close(out["loss"][keep], want["loss"][keep], tol["loss"][keep], "loss")
    grad = pr.distill_top_adjoint(x, index, lp, out["lse"], out["log_rest"], torch.ones(8, device=DEV))
    assert not bool(grad[4].any()) and not bool(grad[1].any()) and bool(torch.isfinite(grad[[0, 2, 3, 5]]).all())
    x[0, 3] = float("inf")
    assert not math.isfinite(float(pr.distill_top(x, index, lp)["loss"][0]))
    none = pr.distill_top(x, index[:, :0], lp[:, :0])
    assert not bool(none["loss"].any())
    assert not bool(pr.distill_top_adjoint(x, index[:, :0], lp[:, :0], out["lse"], out["log_rest"],
                                           torch.ones(8, device=DEV)).any())
    assert pr.distill_top(x[:0], index[:0], lp[:0])["loss"].shape == (0,)


def test_student_that_agrees():
    """Nearly all of the student's mass on the list: what it leaves is summed, not
    the difference from one."""
    c = case(4, 2000, 16, False)
    for n in (0, 2):
        c["x"][n, c["index"][n]] += 30.0
    x, index, lp = put(c, False)
    c["x"] = x.double().cpu().numpy()
    out = pr.distill_top(x, index, lp)
    want, tol = bounds.loss(c, True)
    assert want["log_rest"][0] < -20
    for name in want:
        close(out[name], want[name], tol[name], name)


def test_autograd_and_the_teachers_own_list():
    """From a teacher's logits through token_logprobs to the student's gradient,
    against differences of the loss."""
    g = torch.Generator(DEV).manual_seed(0)
    teacher = torch.randn((3, 500), generator=g, device=DEV)
    x = torch.randn((3, 500), generator=g, device=DEV).requires_grad_(True)
    top = pr.token_logprobs(teacher, torch.full((3,), -1, device=DEV), top=12)
    out = pag.distill_top(x, top["top_index"], top["top_logprob"])
    out["loss"].sum().backward()
    want = ref.distill_top_adjoint(x.detach().cpu().numpy(), top["top_index"].cpu().numpy(),
                                   top["top_logprob"].double().cpu().numpy(), np.ones(3))
    assert np.abs(x.grad.cpu().numpy() - want).max() < 1e-5
    same = pag.distill_top(teacher, top["top_index"], top["top_logprob"])["loss"]
    assert float(same.abs().max()) < 1e-5  # a student that is the teacher
    with pytest.raises(RuntimeError, match="twice"):
        (gx,) = torch.autograd.grad(pag.distill_top(x, top["top_index"], top["top_logprob"])["loss"].sum(), x,
                                    create_graph=True)
        gx.sum().backward()
