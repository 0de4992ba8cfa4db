"""Logits before sampling on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr
from oracle import logits as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def case(N, V, L, M, half, masks, seed=0):
    r = np.random.default_rng(seed + V + 7 * N)
    x = torch.from_numpy(np.float32(3 * r.standard_normal((N, V))))
    x = (x.bfloat16() if half else x).float()
    x[r.random((N, V)) < 0.1] = -float("inf")
    tokens = (V * r.random((N, L)) ** 3).astype(np.int64)
    tokens[r.random((N, L)) < 0.1] = -1
    tokens[r.random((N, L)) < 0.05] = V
    f32 = lambda v: np.float32(v)  # noqa: E731
    c = dict(x=x, tokens=tokens, lengths=r.integers(-1, L + 3, N).astype(np.int32),
             prompt=r.integers(0, L + 1, N).astype(np.int32), repetition=f32(1 + 0.5 * r.random(N)),
             presence=f32(r.random(N)), frequency=f32(0.3 * r.random(N)), bias=None, allowed=None, allowed_rows=None)
    if M:
        index = r.integers(-1, V + 1, (N, M))
        index[:, -1] = index[:, 0]  # twice: the last one counts
        c["bias"] = (index, f32(4 * r.standard_normal((N, M))))
    if masks:
        words = r.integers(-2 ** 31, 2 ** 31, (masks, (V + 31) // 32)).astype(np.int32)
        c |= dict(allowed=words, allowed_rows=r.integers(-1, masks + 1, N).astype(np.int32))
    return c


def call(c, half, names=None, **kw):
    x = c["x"].to(torch.bfloat16 if half else torch.float32).to(DEV)
    put = lambda v: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(DEV)  # noqa: E731
    args = {n: put(c[n]) for n in ("tokens", "lengths", "prompt", "repetition", "presence", "frequency", "allowed",
                                   "allowed_rows") if names is None or n in names}
    if c["bias"] is not None and (names is None or "bias" in names):
        args["bias"] = tuple(put(v) for v in c["bias"])
    return x, pr.adjust_logits(x, **args, **kw)


def check(got, c, half, names=None):
    """A product or quotient, two products and two sums, each within 2^-24 of what
    it adds up: 8 x 2^-24 of the magnitudes, and half a step of bfloat16."""
    args = {n: c[n] for n in ("tokens", "lengths", "prompt", "repetition", "presence", "frequency", "allowed",
                              "allowed_rows", "bias") if names is None or n in names}
    want = ref.adjust_logits(c["x"].numpy(), **args)
    got = got.double().cpu().numpy()
    assert (np.isneginf(got) == np.isneginf(want)).all()
    live = ~np.isneginf(want)
    L = 0 if c["tokens"] is None else c["tokens"].shape[1]
    size = np.abs(want) + 2 * np.abs(np.where(np.isfinite(c["x"].numpy()), c["x"].numpy(), 0)) + 0.3 * L + 20
    tol = 8 * 2.0 ** -24 * size + (2.0 ** -8 * 1.01 * np.abs(want) if half else 0.0)
    assert (np.abs(got[live] - want[live]) <= tol[live]).all()


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("N,V,L,M,masks", [(1, 1, 1, 0, 0), (3, 31, 5, 2, 1), (2, 33, 100, 0, 3), (5, 8191, 40, 3, 2),
                                           (4, 8192, 1000, 0, 0), (3, 8201, 3, 70, 4), (7, 50003, 5000, 300, 2),
                                           (600, 500, 20, 2, 9)])
def test_all_together(N, V, L, M, masks, half):
    c = case(N, V, L, M, half, masks)
    x, got = call(c, half)
    check(got, c, half)
    assert torch.equal(got, call(c, half)[1])
    inplace = call(c, half)[0]
    put = lambda v: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(DEV)  # noqa: E731
    args = {n: put(c[n]) for n in ("tokens", "lengths", "prompt", "repetition", "presence", "frequency", "allowed",
                                   "allowed_rows")}
    bias = None if c["bias"] is None else tuple(put(v) for v in c["bias"])
    assert pr.adjust_logits(inplace, **args, bias=bias, out=inplace) is inplace and torch.equal(inplace, got)


@pytest.mark.parametrize("names", [[], ["tokens"], ["tokens", "repetition"], ["tokens", "presence", "lengths"],
                                   ["tokens", "frequency", "prompt"], ["bias"], ["allowed", "allowed_rows"]])
def test_each_by_itself(names):
    c = case(6, 1037, 60, 5, False, 4)
    x, got = call(c, False, names)
    if not names or names == ["tokens"]:
        assert torch.equal(got, x)
    check(got, c, False, names)


def test_rows_that_are_apart_and_a_mask_for_each():
    c = case(4, 777, 30, 0, True, 4)
    c["allowed_rows"] = None
    _, want = call(c, True)
    wide = torch.zeros((4, 801), dtype=torch.bfloat16, device=DEV)
    wide[:, 3:780] = c["x"].bfloat16().to(DEV)
    tokens = torch.zeros((4, 50), dtype=torch.int64, device=DEV)
    tokens[:, 7:37] = torch.from_numpy(c["tokens"]).to(DEV)
    masks = torch.zeros((4, 40), dtype=torch.int32, device=DEV)
    masks[:, :25] = torch.from_numpy(c["allowed"]).to(DEV)
    out = torch.full((4, 790), 7.0, dtype=torch.bfloat16, device=DEV)
    rest = {n: torch.from_numpy(c[n]).to(DEV) for n in ("lengths", "prompt", "repetition", "presence", "frequency")}
    pr.adjust_logits(wide[:, 3:780], tokens=tokens[:, 7:37], allowed=masks[:, :25], out=out[:, 5:782], **rest)
    assert torch.equal(out[:, 5:782], want)
    out[:, 5:782] = 7.0
    assert bool((out == 7.0).all())


def test_logits_that_are_not_finite():
    x = torch.tensor([[float("nan"), float("inf"), -float("inf"), 1.0, -2.0]], device=DEV)
    tokens = torch.arange(5, device=DEV)[None]
    two = torch.full((1,), 2.0, device=DEV)
    allowed = torch.tensor([[0b01110]], dtype=torch.int32, device=DEV)
    got = pr.adjust_logits(x, tokens=tokens, repetition=two, presence=two, allowed=allowed)[0].tolist()
    assert got == [-float("inf"), float("inf"), -float("inf"), -1.5, -float("inf")]
    assert torch.isnan(pr.adjust_logits(x, tokens=tokens, repetition=two)[0, 0])


def test_empty():
    x = torch.randn((3, 40), device=DEV)
    assert torch.equal(pr.adjust_logits(x, tokens=torch.zeros((3, 0), dtype=torch.int64, device=DEV)), x)
    assert pr.adjust_logits(x[:0]).shape == (0, 40) and pr.adjust_logits(x[:, :0]).shape == (3, 0)


def test_sampling_together():
    """A step of a server: the adjusted logits' alternatives are the ones that the
    grammar allows."""
    c = case(8, 2000, 50, 4, True, 3)
    c["allowed_rows"][:] = np.arange(8) % 4 - 1
    _, x = call(c, True)
    out = pr.token_logprobs(x, torch.full((8,), -1, device=DEV), top=5)
    want = ref.adjust_logits(c["x"].numpy(), **{n: c[n] for n in c if n != "x"})
    for n in range(8):
        for j in out["top_index"][n].tolist():
            assert j >= 0 and np.isfinite(want[n, j])
