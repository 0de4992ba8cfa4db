"""The oracle of the distillation and of the logits before sampling, on the CPU."""
import numpy as np
import pytest

from oracle import logits as ref


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("seed", range(3))
def test_distillation_against_differences(seed, tail):
    """Central differences: steps of 1e-5 leave 1e-10 of a third derivative of
    about 1 and 1e-16 / 1e-5 of roundings."""
    r = np.random.default_rng(seed)
    N, V, k, scale = 3, 11, 4, 0.7
    x, g = r.standard_normal((N, V)), r.standard_normal(N)
    index = np.stack([r.permutation(V)[:k] for _ in range(N)])
    index[1, 2], index[2] = -1, -1
    logprob = np.log(r.dirichlet(np.ones(k + 3), N)[:, :k])
    got = ref.distill_top_adjoint(x, index, logprob, g, tail, scale)
    for n in range(N):
        for j in range(V):
            e = np.zeros_like(x)
            e[n, j] = 1e-5
            up, down = (ref.distill_top(x + s * e, index, logprob, tail, scale)["loss"] for s in (1, -1))
            assert abs((up - down) @ g / 2e-5 - got[n, j]) < 1e-8
    assert ref.distill_top(x, index, logprob, tail, scale)["loss"][2] == 0 and not got[2].any()


def test_a_whole_list_is_the_divergence():
    r = np.random.default_rng(5)
    p = r.dirichlet(np.ones(7))
    x = r.standard_normal((1, 7))
    loss = ref.distill_top(x, np.arange(7)[None], np.log(p)[None])["loss"][0]
    q = np.exp(x[0]) / np.exp(x[0]).sum()
    assert abs(loss - (p * np.log(p / q)).sum()) < 1e-12


def test_adjusted_logits():
    """Each rule by hand."""
    x = np.array([[2.0, -2.0, 1.0, 4.0, 0.5]])
    got = ref.adjust_logits(x, tokens=np.array([[0, 1, 3, 3, -1, 9]]), lengths=np.array([6]), prompt=np.array([2]),
                            repetition=np.array([2.0]), presence=np.array([0.25]), frequency=np.array([0.5]),
                            bias=(np.array([[4, 4]]), np.array([[7.0, 1.0]])), allowed=np.array([[0b11011]], np.int32))
    assert np.array_equal(got, [[1.0, -4.0, -np.inf, 2.0 - 2 * 0.5 - 0.25, 1.5]])
