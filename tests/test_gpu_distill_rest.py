"""The distillation's gradient where the student leaves next to nothing to the
tokens that are not listed, and where an index is past the vocabulary.

Bounds, u = 2^-24.  A token that is not listed has the share r exp(d) / s of the
gradient, d = scale (x - max) and s the sum of these exponentials: d is rounded
three times (a difference, two products), so exp(d) is within 6 u (1 + |d|) of
itself; s within (V / 256 + 32) u (a thread's share, then a tree) and what its
terms are off by; r = 1 - P within 4 u P + u.  Nearer than e^-64 the share comes
from lse and log q_rest instead, which hold three such sums and are float32 numbers
of up to 64 + |lse|, with five roundings of that size; q_j (P + r) comes with it.  A
listed token has q within such a sum and 64 u, and p within 16 u.  Rounding to
bfloat16: half a step, 2^-8."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr
from oracle import logits as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def case(V, far, half, scale):
    """Rows whose other tokens lie `far` below the listed ones: about it, all at the
    same place; a row without a remainder, and one like any other."""
    r = np.random.default_rng(V)
    dtype = torch.bfloat16 if half else torch.float32
    x = np.full((4, V), far / scale if far > -1e5 else far)
    if far > -1e5:
        x[0] += r.standard_normal(V)
    x[3] = r.standard_normal(V)
    index = np.stack([r.permutation(V)[:5] for _ in range(4)])
    index[1, 3:] = -1
    for n in range(3):
        x[n, index[n][index[n] >= 0]] = r.standard_normal((index[n] >= 0).sum())
    p = r.dirichlet(np.ones(5), 4) * np.array([[0.7], [0.9], [1.0], [0.6]])
    x = torch.from_numpy(x).float().clamp(min=torch.finfo(dtype).min).to(dtype)
    return x, index, np.float32(np.log(p)).astype(np.float64)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("V,scale", [(5, 1.0), (1000, 1.0), (40001, 0.5)])
@pytest.mark.parametrize("far", [-10.0, -50.0, -63.0, -80.0, -100.0, -1000.0, -1e9, -3.5e38])
def test_shares_of_next_to_nothing(far, V, scale, half):
    x, index, lp = case(V, far, half, scale)
    g = np.array([1.0, -0.5, 2.0, 1.5])
    dev = [x.to(DEV), torch.from_numpy(index).to(DEV), torch.from_numpy(lp).float().to(DEV)]
    out = pr.distill_top(*dev, scale=scale)
    args = (*dev, out["lse"], out["log_rest"], torch.from_numpy(g).float().to(DEV))
    grad = pr.distill_top_adjoint(*args, scale=scale)
    x = x.double().numpy()
    want = ref.distill_top_adjoint(x, index, lp, g, True, scale)
    p = np.where(index >= 0, np.exp(lp), 0.0)
    P = p.sum(1)
    tol = np.zeros_like(want)
    for n in range(4):
        listed = index[n][index[n] >= 0]
        others = np.ones(V, bool)
        others[listed] = False
        base = (3 * (V / 256 + 32) + 64) * U
        tol[n, listed] = (P[n] + 1) * base + 16 * U * p[n][index[n] >= 0]
        if not others.any():
            continue
        lse = float(ref.distill_top(x[n:n + 1], index[n:n + 1], lp[n:n + 1], True, scale)["lse"][0])
        d = scale * (x[n] - x[n][others].max())
        size = np.abs(d) + max(0.0, (d.max() if d.max() < 70 else 0.0) + abs(lse))
        share = np.exp(np.minimum(d, 0.0)) / np.exp(d[others]).sum()
        terms = base + 12 * U * (1 + size)
        off = share * (terms + terms[others].max() + (4 * P[n] + 1) * U) + np.exp(np.minimum(scale * x[n] - lse, 0)) * terms
        tol[n, others] = off[others]
    tol = scale * np.abs(g)[:, None] * tol + 1e-36
    if half:
        tol += 2.0 ** -8 * (np.abs(want) + tol)
    got = grad.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - want) - tol
    assert (off <= 0).all(), (np.argwhere(off > 0)[:5].tolist(), got[off > 0][:5], want[off > 0][:5])
    if V > 5:  # a softmax's gradient: what the list takes the others give
        assert (np.abs(got.sum(1)) <= tol.sum(1)).all()
    inplace = pr.distill_top_adjoint(*args, scale=scale, out=dev[0])
    assert inplace.data_ptr() == dev[0].data_ptr() and torch.equal(inplace, grad)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("V", [300, 50001])
def test_an_index_past_the_vocabulary(V, half):
    """Its loss is NaN; so is the whole row's gradient, and no other's."""
    g = torch.Generator(DEV).manual_seed(V)
    x = torch.randn((4, V), generator=g, device=DEV).to(torch.bfloat16 if half else torch.float32)
    x[3] = -float("inf")
    index = torch.randint(0, V, (4, 6), generator=g, device=DEV)
    lp = torch.full((4, 6), -2.0, device=DEV)
    good, ones = index.clone(), torch.ones(4, device=DEV)
    index[1, 4], index[3, 0] = V, 2 ** 40
    out, fine = pr.distill_top(x, index, lp), pr.distill_top(x, good, lp)
    assert out["loss"].isnan().tolist() == [False, True, False, True]
    grad = pr.distill_top_adjoint(x, index, lp, out["lse"], out["log_rest"], ones)
    want = pr.distill_top_adjoint(x, good, lp, fine["lse"], fine["log_rest"], ones)
    assert bool(grad[[1, 3]].isnan().all()) and torch.equal(grad[[0, 2]], want[[0, 2]])


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("V", [5, 1000, 40001])
@pytest.mark.parametrize("at", [5000.0, -5000.0, -1e9, -3.5e38])
def test_rows_far_from_zero(at, V, tail, half):
    """Logits of 5000 and more, a row that a finite mask left nothing of: lse as a
    float32 holds no log V beside them, so q comes from the row's own maximum and sum,
    with the roundings of a share."""
    r = np.random.default_rng(V)
    dtype = torch.bfloat16 if half else torch.float32
    x = np.full((3, V), at)
    x[1] += 40 * r.standard_normal(V)
    x[2] = r.standard_normal(V)
    x = torch.from_numpy(x).float().clamp(min=torch.finfo(dtype).min).to(dtype)
    index = np.stack([r.permutation(V)[:4] for _ in range(3)])
    lp = np.float32(np.log(r.dirichlet(np.ones(4), 3) * 0.8)).astype(np.float64)
    dev = [x.to(DEV), torch.from_numpy(index).to(DEV), torch.from_numpy(lp).float().to(DEV)]
    out = pr.distill_top(*dev, tail=tail)
    args = (*dev, out["lse"], out["log_rest"], torch.ones(3, device=DEV))
    grad = pr.distill_top_adjoint(*args, tail=tail)
    x = x.double().numpy()
    want = ref.distill_top_adjoint(x, index, lp, np.ones(3), tail)
    d = x - x.max(1, keepdims=True)
    q = np.exp(d) / np.exp(d).sum(1, keepdims=True)
    listed = np.zeros((3, V), bool)
    np.put_along_axis(listed, index, True, 1)
    p = np.exp(lp)
    left = np.where(tail, 1 - p.sum(1, keepdims=True), 0.0)
    e = np.where(listed, -np.inf, d)
    e = e - e.max(1, keepdims=True)
    share = np.exp(e) / np.exp(e).sum(1, keepdims=True)
    terms = (3 * (V / 256 + 32) + 64) * U + 12 * U * (1 + np.where(np.abs(d) < 200, np.abs(d), 0.0) + 12)
    most = np.where(np.abs(d) < 30, terms, 0.0).max(1, keepdims=True)
    tol = (2 * q + left * share) * (terms + most + 5 * U / 0.2) + np.where(listed, 16 * U, 0.0) + 1e-36
    if half:
        tol += 2.0 ** -8 * (np.abs(want) + tol)
    got = grad.double().cpu().numpy()
    off = np.abs(got - want) - tol
    assert (off <= 0).all(), (np.argwhere(~(off <= 0))[:5].tolist(), got[~(off <= 0)][:5], want[~(off <= 0)][:5])
    inplace = pr.distill_top_adjoint(*args, tail=tail, out=dev[0])
    assert torch.equal(inplace, grad)
