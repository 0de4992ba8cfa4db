"""Strides that the gated delta rule takes, on the CPU: tensors pass every check
of the binding but the last one, and the C ABI gets as far as the workspace."""
import ctypes

import pytest
import torch

from nonlinear_rnn_amd import pararnn as pr
from tests.test_delta_refusals import INVALID, NULL, WORKSPACE, common, heads, shape, step


@pytest.mark.parametrize("B,Hv,T", [(2, 3, 1), (1, 3, 5), (1, 1, 5), (1, 3, 1)])
def test_gates_differ_only_where_nothing_steps(B, Hv, T):
    dense = torch.zeros(B, Hv, T)
    other = torch.zeros(B, T, Hv).transpose(1, 2) if T == 1 else torch.zeros(B, Hv + 4, T)[:, 1:1 + Hv]
    assert dense.stride() != other.stride()
    for beta, g in ((dense, other), (other, dense)):
        with pytest.raises(ValueError, match="GPU"):
            pr.delta_scan(**heads(B=B, Hv=Hv, T=T, beta=beta, log_decay=g))
        if T == 1:
            with pytest.raises(ValueError, match="GPU"):
                step(q=torch.zeros(B, 1, 3), k=torch.zeros(B, 1, 3), v=torch.zeros(B, Hv, 4), beta=beta[..., 0],
                     log_decay=g[..., 0], states=torch.zeros(3, Hv, 3, 4))


def test_gates_that_differ_are_refused():
    with pytest.raises(ValueError, match="strides"):
        pr.delta_scan(**heads(B=1, Hv=2, T=5, log_decay=torch.zeros(1, 5, 2).transpose(1, 2)))
    with pytest.raises(ValueError, match="strides"):
        step(log_decay=torch.zeros(2, 2).t(), beta=torch.zeros(2, 2))


@pytest.mark.parametrize("o", [[0, 0, 0, 0], [120, 30, 0, 1], [30, 30, 5, 1]])
def test_a_gradient_of_the_output_may_repeat_elements(o):
    """It is only read; the output itself may not."""
    a, head = common(dict(sh=shape(o=o)))
    call = pr.load().pararnn_delta_scan_adjoint
    assert call(*head, a["go"], NULL, ctypes.byref(a["g"]), NULL, 0, NULL) == WORKSPACE
    assert pr.load().pararnn_delta_scan(*head, a["o"], NULL, NULL, 0, NULL) == INVALID
    _, head = common(dict(sh=shape(o=[120, 30, -5, 1])))
    assert call(*head, a["go"], NULL, ctypes.byref(a["g"]), NULL, 0, NULL) == INVALID
