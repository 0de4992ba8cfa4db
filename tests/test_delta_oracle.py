"""The oracle of the gated delta rule: its gradients against differences, its
documents against runs of their own, and the chunked form that the kernels
compute against the steps."""
import numpy as np
import pytest

from oracle import delta as ref


def case(seed, B=2, Hk=1, Hv=2, dk=3, dv=2, T=9, docs=True):
    r = np.random.default_rng(seed)
    k = r.standard_normal((B, Hk, dk, T))
    k /= np.linalg.norm(k, axis=2, keepdims=True)
    return dict(q=r.standard_normal((B, Hk, dk, T)), k=k, v=r.standard_normal((B, Hv, dv, T)),
                beta=r.random((B, Hv, T)), log_decay=-r.random((B, Hv, T)), h0=r.standard_normal((B, Hv, dk, dv)),
                resets=r.random((B, T)) < 0.3 if docs else None)


@pytest.mark.parametrize("seed", range(3))
def test_gradients_against_differences(seed):
    """Central differences of step 1e-5 of a loss of size 10: 1e-10 from the third
    derivative, 1e-10 from float64's rounding."""
    c, r = case(seed), np.random.default_rng(seed + 100)
    go, gl = r.standard_normal(c["v"].shape), r.standard_normal(c["h0"].shape)

    def loss(c):
        o, S = ref.delta_scan(**c, scale=0.7)
        return (o * go).sum() + (S * gl).sum()
    got = ref.delta_scan_adjoint(**c, go=go, g_last=gl, scale=0.7)
    for name in ("q", "k", "v", "beta", "log_decay", "h0"):
        for i in r.choice(c[name].size, 6, replace=False):
            at = np.unravel_index(i, c[name].shape)
            two = []
            for e in (1e-5, -1e-5):
                x = c[name].copy()
                x[at] += e
                two.append(loss(c | {name: x}))
            assert abs((two[0] - two[1]) / 2e-5 - got["d" + name][at]) < 1e-7, (name, at)


def test_documents_by_themselves():
    c = case(5, B=1, T=12, docs=False)
    cut = 7
    whole, last = ref.delta_scan(**{**c, "resets": (np.arange(12) == cut)[None]})
    parts = [{n: c[n][..., s] for n in ("q", "k", "v", "beta", "log_decay")} for s in (slice(0, cut), slice(cut, 12))]
    first = ref.delta_scan(**parts[0], h0=c["h0"])[0]
    second, S = ref.delta_scan(**parts[1])
    assert np.allclose(whole, np.concatenate([first, second], -1), atol=1e-14) and np.allclose(last, S, atol=1e-14)
    forget = c["log_decay"].copy()
    forget[..., cut] = -np.inf
    c["h0"][:] = np.nan  # nothing of it is left behind the step that forgets
    again, S = ref.delta_scan(**{**c, "log_decay": forget, "resets": None})
    assert np.allclose(again[..., cut:], second, atol=1e-14) and np.allclose(last, S, atol=1e-14)


def test_chunk_form():
    """(I + A) W = R, o and S' of a chunk of 9 steps as one."""
    c = case(6, B=1, Hv=1, docs=False)
    q, k, v = (c[n][0, 0].T for n in ("q", "k", "v"))
    b, G, S = c["beta"][0, 0], np.cumsum(c["log_decay"][0, 0]), c["h0"][0, 0]
    D = np.exp(G[:, None] - G[None, :])
    A = np.tril(b[:, None] * (k @ k.T) * D, -1)
    W = np.linalg.solve(np.eye(9) + A, b[:, None] * (v - np.exp(G)[:, None] * (k @ S)))
    o = np.exp(G)[:, None] * (q @ S) + np.tril((q @ k.T) * D) @ W
    last = np.exp(G[-1]) * S + (np.exp(G[-1] - G)[:, None] * k).T @ W
    want, S = ref.delta_scan(**c)
    assert np.allclose(o.T, want[0, 0], atol=1e-13) and np.allclose(last, S[0, 0], atol=1e-13)
