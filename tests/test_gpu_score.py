"""Token scores on the GPU against the float64 oracle.

Tolerance.  A log probability is d - log s: d = scale (x - m) has two
roundings of its size, the exponentials' sum is within 2^-24 (V / 256 + 24)
(chains of a lane, then a tree; 4 ulp an exponential), which its log turns into
an absolute error; so 2^-24 (4 |d| + V / 256 + 32), and for the entropy, whose
terms are d exp(d), the same with the row's mean |d| (below 32 here).  lse adds
a rounding of its own size.  A gradient is p times its coefficients: relative
2^-24 (4 |log p| + 64) of their sum, |log p| below 128 where p is not 0."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_amd import autograd as pag
from nonlinear_rnn_amd import pararnn as pr
from oracle import language as ref
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
INF = float("inf")


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, want, tol):
    got, want = f64(got), np.asarray(want)
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine) and np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    assert (np.abs(got - want)[fine] <= np.broadcast_to(tol, got.shape)[fine]).all(), (
        float(np.abs(got - want)[fine].max()))


def check(x, tokens, top=0, scale=1.0, adjoint=True):
    N, V = x.shape
    out = pr.token_logprobs(x, tokens, top=top, scale=scale)
    want = ref.token_logprobs(f64(x), tokens.cpu().numpy(), top, scale)
    base = EPS * (V / 256 + 32)
    mag = np.where(np.isfinite(want["lse"]), np.abs(want["lse"]), 0)
    d = np.where(np.isfinite(want["logprob"]), np.abs(want["logprob"]), 0)
    near(out["lse"], want["lse"], base + 4 * EPS * (mag + 64))
    near(out["logprob"], want["logprob"], base + 4 * EPS * (d + 32))
    near(out["entropy"], want["entropy"], base * 2 + 4 * EPS * 64)
    if top:
        assert np.array_equal(out["top_index"].cpu().numpy(), want["top_index"])
        near(out["top_logprob"], want["top_logprob"], base + 4 * EPS * 64)
    if not adjoint:
        return out
    r = np.random.default_rng(N + V)
    g = [torch.from_numpy(r.standard_normal(N)).float().to(DEV) for _ in range(3)]
    got = pr.token_logprobs_adjoint(x, tokens, out["lse"], out["entropy"], g_logprob=g[0],
                                    g_entropy=g[1], g_lse=g[2], scale=scale)
    exact = ref.token_logprobs_adjoint(f64(x), tokens.cpu().numpy(), *[f64(v) for v in g], scale)
    bf16 = x.dtype == torch.bfloat16
    # lse and entropy are the forward's float32 values: their errors enter too
    coefficients = scale * (np.abs(f64(g[0])) + np.abs(f64(g[2])) + np.abs(f64(g[1])) * 64)[:, None]
    tol = (2 * base + EPS * (4 * 128 + 64 + 4 * mag[:, None])) * coefficients
    near(got, exact, tol + (2.0 ** -8 * np.abs(exact) if bf16 else 0))
    assert got.dtype == x.dtype
    return out


def logits(N, V, dtype=torch.float32, seed=0, std=3.0, masked=0.0, stride=None):
    r = np.random.default_rng(seed + 31 * N + V)
    x = std * r.standard_normal((N, V)) + 2 * r.standard_normal((N, 1))
    x[r.random((N, V)) < masked] = -INF
    buf = torch.full((N, stride or V), 50.0, dtype=dtype, device=DEV)  # what lies past the row would show
    buf[:, :V] = torch.from_numpy(x).to(DEV).to(dtype)
    tokens = torch.from_numpy(r.integers(0, V, N)).to(DEV)
    if N > 2:
        tokens[1] = -1
    return buf[:, :V], tokens


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (2, 63), (5, 64), (4, 257), (3, 1000), (2, 4097),
                                 (300, 129), (1, 70001), (2, 131072)])
@pytest.mark.parametrize("top", [0, 1, 7, 64])
def test_scores(N, V, dtype, top):
    x, tokens = logits(N, V, dtype)
    check(x, tokens, top, adjoint=top == 7)


@pytest.mark.parametrize("N,V", [(1100, 2049), (600, 8192), (600, 8193)])
@pytest.mark.parametrize("top", [0, 20])
def test_rows_of_a_wave(N, V, top):
    test_scores(N, V, torch.float32, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("stride", [1001, 1003, 1024])
def test_padded_rows(dtype, stride):
    x, tokens = logits(6, 1001, dtype, stride=stride)
    check(x, tokens, 5)
    check(x[:, 3:990], tokens.clamp(max=980), 5)  # a row that starts at any element


@pytest.mark.parametrize("scale", [0.05, 0.7, 3.0])
def test_scale(scale):
    x, tokens = logits(7, 3001)
    check(x, tokens, 9, scale)


@pytest.mark.parametrize("masked", [0.3, 0.99, 1.0])
@pytest.mark.parametrize("V", [50, 40000])
def test_masked_tokens(masked, V):
    x, tokens = logits(9, V, masked=masked)
    x[4] = -INF
    x[5] = -INF
    x[5, V // 2] = 1.5       # one token allowed
    x[6, int(tokens[6])] = -INF  # the given token masked
    check(x, tokens, 20)


def test_the_types_lowest_value_is_a_value():
    """A mask that adds the type's lowest value is finite: such tokens count."""
    x, tokens = logits(3, 300)
    low = torch.finfo(torch.float32).min
    x[:, 10:] = low
    out = check(x, tokens.clamp(max=9), 12, adjoint=False)
    assert out["top_index"][:, 10:].tolist() == [[10, 11]] * 3
    x[1] = low  # nothing but the lowest value: equal chances
    out = pr.token_logprobs(x, tokens, top=2)
    assert abs(float(out["entropy"][1]) - np.log(300)) < 1e-5
    assert out["top_index"][1].tolist() == [0, 1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [100, 5000, 66000])
def test_equal_logits_go_lowest_first(V, dtype):
    r = np.random.default_rng(V)
    x = torch.from_numpy(r.integers(-2, 3, (6, V)).astype(np.float32)).to(DEV).to(dtype)
    x[0] = 1.0
    x[1] = -0.0
    x[1, 40:] = 0.0  # zeros of either sign are equal
    check(x, torch.zeros(6, dtype=torch.int64, device=DEV), 64)


@pytest.mark.parametrize("order", ["up", "down", "last"])
@pytest.mark.parametrize("N", [1, 300])
def test_sorted_rows(order, N):
    """Orders in which every token, or the last alone, is a new alternative."""
    x = torch.linspace(-20, 20, 9000, device=DEV).repeat(N, 1)
    if order == "down":
        x = x.flip(1).contiguous()
    if order == "last":
        x[:, :-1] = -3.0
    check(x[:3], torch.zeros(min(N, 3), dtype=torch.int64, device=DEV), 50, adjoint=False)
    out = pr.token_logprobs(x, torch.zeros(N, dtype=torch.int64, device=DEV), top=50)
    assert (out["top_index"] == out["top_index"][:1]).all()


def test_infinities_and_nan():
    x, tokens = logits(4, 200)
    x[0, 7] = float("nan")
    x[1, 9] = INF
    x[2] = -INF
    x[2, 3] = float("nan")
    out = check(x, tokens.abs(), 3, adjoint=False)
    assert torch.isnan(out["lse"][:3]).all() and torch.isfinite(out["lse"][3])


def test_tokens_outside_the_vocabulary():
    x, _ = logits(4, 100)
    tokens = torch.tensor([-1, -100, 100, 2 ** 40], device=DEV)
    out = pr.token_logprobs(x, tokens)
    assert out["logprob"][:2].tolist() == [0.0, 0.0] and torch.isnan(out["logprob"][2:]).all()
    g = torch.ones(4, device=DEV)
    grad = pr.token_logprobs_adjoint(x, tokens, out["lse"], g_logprob=g)
    assert not grad[:2].any() and torch.isfinite(grad).all()


def test_in_place_gradient():
    x, tokens = logits(9, 1003, torch.bfloat16, stride=1010)
    out = pr.token_logprobs(x, tokens)
    g = torch.linspace(-1, 1, 9, device=DEV)
    want = pr.token_logprobs_adjoint(x, tokens, out["lse"], out["entropy"], g_logprob=g, g_entropy=g)
    got = pr.token_logprobs_adjoint(x, tokens, out["lse"], out["entropy"], g_logprob=g, g_entropy=g, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)


def test_empty_sizes():
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    out = pr.token_logprobs(torch.empty((0, 50), device=DEV), none, top=3)
    assert out["logprob"].shape == (0,) and out["top_index"].shape == (0, 3)
    out = pr.token_logprobs(torch.empty((2, 0), device=DEV), torch.tensor([-1, 0], device=DEV), top=2)
    assert out["lse"].tolist() == [-INF, -INF] and out["top_index"].tolist() == [[-1, -1]] * 2
    assert out["logprob"][0] == 0 and torch.isnan(out["logprob"][1])


def test_offsets_past_32_bits():
    far = 2 ** 30 + 5
    x, tokens = logits(3, 400, torch.bfloat16)
    big = torch.as_strided(torch.zeros(2 * far + 400, dtype=torch.bfloat16, device=DEV), (3, 400), (far, 1))
    big.copy_(x)
    a, b = pr.token_logprobs(big, tokens, top=5), pr.token_logprobs(x, tokens, top=5)
    for k in ("logprob", "entropy", "lse", "top_logprob"):
        near(a[k], f64(b[k]), EPS * 100 * 8)
    assert torch.equal(a["top_index"], b["top_index"])
    g = torch.ones(3, device=DEV)
    out = torch.as_strided(torch.zeros(2 * far + 400, dtype=torch.bfloat16, device=DEV), (3, 400), (far, 1))
    pr.token_logprobs_adjoint(big, tokens, b["lse"], g_logprob=g, out=out)
    want = pr.token_logprobs_adjoint(x, tokens, b["lse"], g_logprob=g)
    assert torch.equal(out, want)


@pytest.mark.parametrize("N", [2, 600])
def test_another_stream_and_repeatable(N):
    x, tokens = logits(N, 30011, torch.bfloat16)
    s = torch.cuda.Stream()
    a = pr.token_logprobs(x, tokens, top=10)
    torch.cuda.synchronize()
    b = pr.token_logprobs(x, tokens, top=10, stream=s)
    s.synchronize()
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_autograd():
    x, tokens = logits(6, 500, masked=0.2)
    x.requires_grad_(True)
    out = pag.token_logprobs(x, tokens, top=3, scale=0.9)
    (-out["logprob"].sum() + 0.1 * out["entropy"].sum() + 0.01 * out["lse"].square().sum()).backward()
    g = [-np.ones(6), np.full(6, 0.1), 0.02 * f64(out["lse"])]
    want = ref.token_logprobs_adjoint(f64(x), tokens.cpu().numpy(), *g, 0.9)
    near(x.grad, want, EPS * 800)
    assert not out["top_logprob"].requires_grad
