"""Pins of the float64 oracle of the language-model operators: its backward
passes against central differences of its forward passes, and limits that can
be worked out by hand.  Step 1e-6 in float64: the differences are good to
about 1e-9 of the function's size, the tolerance leaves a factor of 100."""
import numpy as np
import pytest

from oracle import language as ref


def differences(f, x, g_of, eps=1e-6):
    """Central differences of <f(x), g> in every element of x."""
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += eps
        lo[i] -= eps
        out[i] = (g_of(f(hi)) - g_of(f(lo))) / (2 * eps)
    return out


def near(a, b, tol=1e-7):
    assert np.abs(a - b).max() <= tol * max(1.0, np.abs(b).max())


@pytest.mark.parametrize("docs", [False, True])
def test_gated_scan_adjoint_is_the_derivative(docs):
    r = np.random.default_rng(1)
    B, D, T, power = 2, 3, 7, 4.0
    u = [r.standard_normal((B, D, T)) for _ in range(3)]
    lam, h0 = r.standard_normal(D), r.standard_normal((B, D))
    resets = r.random((B, T)) < 0.3 if docs else None
    gh, gl = r.standard_normal((B, D, T)), r.standard_normal((B, D))
    h = ref.gated_scan(u, lam, h0, power, resets)
    got = ref.gated_scan_adjoint(u, lam, h0, h, gh, power, resets, gl)

    def loss(out):
        return (out * gh).sum() + (out[..., -1] * gl).sum()
    for g in range(3):
        near(got["du"][g], differences(lambda p: ref.gated_scan(u[:g] + [p] + u[g + 1:], lam, h0, power, resets), u[g], loss))
    near(got["dlam"], differences(lambda p: ref.gated_scan(u, p, h0, power, resets), lam, loss))
    near(got["dh0"], differences(lambda p: ref.gated_scan(u, lam, p, power, resets), h0, loss))


def test_gated_scan_limits():
    T = 5
    u = [np.full((1, 1, T), v) for v in (-800.0, 3.0, 2.0)]  # no decay: the state is kept
    assert np.array_equal(ref.gated_scan(u, np.zeros(1), np.full((1, 1), 1.5), 8.0), np.full((1, 1, T), 1.5))
    u[0][:] = 800.0  # full decay: the input alone
    got = ref.gated_scan(u, np.full(1, 50.0), np.full((1, 1), 1.5), 8.0)
    near(got, np.full((1, 1, T), 2.0 / (1 + np.exp(-3.0))), 1e-12)


@pytest.mark.parametrize("with_h,with_gate", [(True, True), (True, False), (False, False)])
def test_block_norm_adjoint_is_the_derivative(with_h, with_gate):
    r = np.random.default_rng(2)
    B, T, D = 2, 3, 5
    h = r.standard_normal((B, D, T)) if with_h else None
    gate = r.standard_normal((B, D, T)) if with_gate else None
    x, wp, wn = r.standard_normal((B, T, D)), r.standard_normal(D), r.standard_normal(D)
    gy, gz = r.standard_normal((B, T, D)), r.standard_normal((B, T, D))
    kw = dict(scale=0.7, eps=1e-3)
    got = ref.block_norm_adjoint(h, x, wp, wn, gy, gz, gate, **kw)

    def loss(out):
        return (out[0] * gy).sum() + (out[1] * gz).sum()
    near(got["dx"], differences(lambda p: ref.block_norm(h, p, wp, wn, gate, **kw), x, loss))
    near(got["dw_pre"], differences(lambda p: ref.block_norm(h, x, wp, p, gate, **kw), wn, loss))
    if with_h:
        near(got["dh"], differences(lambda p: ref.block_norm(p, x, wp, wn, gate, **kw), h, loss))
        near(got["dw_post"], differences(lambda p: ref.block_norm(h, x, p, wn, gate, **kw), wp, loss))
    if with_gate:
        near(got["dgate"], differences(lambda p: ref.block_norm(h, x, wp, wn, p, **kw), gate, loss))


def test_token_logprobs_adjoint_is_the_derivative():
    r = np.random.default_rng(3)
    N, V, scale = 4, 6, 0.8
    x = 2 * r.standard_normal((N, V))
    tokens = np.array([0, 5, -1, 2])
    g = [r.standard_normal(N) for _ in range(3)]

    def loss(o):
        return (o["logprob"] * g[0]).sum() + (o["entropy"] * g[1]).sum() + (o["lse"] * g[2]).sum()
    near(ref.token_logprobs_adjoint(x, tokens, *g, scale), differences(lambda p: ref.token_logprobs(p, tokens, 0, scale), x, loss))


def test_token_logprobs_limits():
    x = np.full((3, 4), -np.inf)
    x[1] = 0.0
    x[2, 3] = 7.0
    out = ref.token_logprobs(x, [0, 2, 3], 3)
    assert out["lse"][0] == -np.inf and out["logprob"][0] == -np.inf and out["entropy"][0] == 0
    near(out["logprob"][1], -np.log(4.0), 1e-15)
    near(out["entropy"][1], np.log(4.0), 1e-15)
    assert out["logprob"][2] == 0 and out["entropy"][2] == 0
    assert out["top_index"].tolist() == [[-1, -1, -1], [0, 1, 2], [3, -1, -1]]
