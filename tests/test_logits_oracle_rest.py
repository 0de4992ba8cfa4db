"""The distillation's oracle where the student leaves next to nothing to the
tokens that are not listed, on the CPU."""
import numpy as np
import pytest

from oracle import logits as ref


@pytest.mark.parametrize("far", [-20.0, -100.0, -1000.0])
def test_gradient_against_differences(far):
    """Central differences of step 1e-5 of a loss of 300 at most: 1e-10 from the
    third derivative, 300 * 1e-16 / 1e-5 from roundings."""
    r = np.random.default_rng(3)
    x = far + r.standard_normal((1, 9))
    index = np.array([[4, 7]])
    x[0, index[0]] = [0.3, -0.2]
    lp = np.log([[0.5, 0.2]])
    got = ref.distill_top_adjoint(x, index, lp, np.ones(1))
    assert abs(got.sum()) < 1e-14 and (got[0, [0, 1, 2, 3, 5, 6, 8]] < -1e-3).all()
    for j in range(9):
        e = np.zeros_like(x)
        e[0, j] = 1e-5
        up, down = (ref.distill_top(x + s * e, index, lp)["loss"][0] for s in (1, -1))
        assert abs((up - down) / 2e-5 - got[0, j]) < 3e-8


@pytest.mark.parametrize("mask", [-1e9, float(np.finfo(np.float32).min)])
def test_a_finite_mask_is_shared_evenly(mask):
    x = np.full((1, 1001), mask)
    x[0, 5] = 0.0
    got = ref.distill_top_adjoint(x, np.array([[5]]), np.log([[0.7]]), np.ones(1))
    assert np.allclose(np.delete(got[0], 5), -0.3 / 1000, rtol=1e-12) and abs(got.sum()) < 1e-12


@pytest.mark.parametrize("all_at", [-1e9, float(np.finfo(np.float32).min)])
def test_a_row_of_one_finite_mask_is_even(all_at):
    got = ref.distill_top_adjoint(np.full((1, 1001), all_at), np.array([[5]]), np.log([[0.7]]), np.ones(1))
    assert np.allclose(np.delete(got[0], 5), 1 / 1001 - 0.3 / 1000, atol=1e-15) and abs(got[0, 5] - (1 / 1001 - 0.7)) < 1e-15
