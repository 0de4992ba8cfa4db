"""Captures beside graphs of the same leaves, on the CPU: the operators' GPU work
and the question which stream is current are stood in for; the graphs and the
nodes that collect the leaves' gradients are torch's own."""
import pytest
import torch

from nonlinear_rnn_amd import autograd as pag
from nonlinear_rnn_amd import pararnn as pr


class Current:
    stream, captured = 0, False

    def __call__(self, t):
        return self.stream, self.captured


@pytest.fixture
def on(monkeypatch):
    """on(stream, captured): what is current from here on."""
    now = Current()

    def distill(logits, index, logprob, **_):
        return dict(loss=logits.sum(1), lse=logits.sum(1), log_rest=logits.sum(1))
    monkeypatch.setattr(pag, "_stream_of", now)
    monkeypatch.setattr(pr, "distill_top", distill)
    monkeypatch.setattr(pr, "delta_scan", lambda q, k, v, *_, **__: (v.float() * 1, q.new_zeros(1, 2, 3, 4)))

    def set_to(stream, captured=False):
        now.stream, now.captured = stream, captured
    return set_to


def distill_top():
    x = torch.zeros((2, 5), requires_grad=True)
    return [x], lambda: pag.distill_top(x, torch.zeros((2, 1), dtype=torch.int64), torch.zeros(2, 1))["loss"]


def delta_scan():
    t = [torch.zeros(s, requires_grad=True) for s in ((1, 2, 3, 5), (1, 2, 3, 5), (1, 2, 4, 5), (1, 2, 5), (1, 2, 5))]
    return t, lambda: pag.delta_scan(*t)[0]


OPERATORS = pytest.mark.parametrize("operator", [distill_top, delta_scan])


@OPERATORS
@pytest.mark.parametrize("stream", [0, 5])
def test_one_eager_graph_alive(operator, stream, on):
    leaves, fn = operator()
    on(stream)
    alive = fn()
    on(7, True)
    for _ in range(2):
        with pytest.raises(RuntimeError, match="eager graph"):
            fn()
    with torch.no_grad():
        fn()  # nothing is recorded, so nothing is in the way
    del alive
    fn()


@OPERATORS
def test_a_warm_up_on_the_captures_stream_beside_it(operator, on):
    leaves, fn = operator()
    on(0)
    alive = fn()
    on(7)
    fn(), fn()
    on(7, True)
    with pytest.raises(RuntimeError, match="eager graph"):
        fn()
    assert alive.requires_grad


@OPERATORS
def test_another_operators_graph(operator, on):
    """Whatever stream it was recorded on, it is not the warm-up's."""
    leaves, fn = operator()
    on(0)
    alive = leaves[-1] * 2
    on(7)
    fn()
    on(7, True)
    with pytest.raises(RuntimeError, match="eager graph"):
        fn()
    del alive
    fn()


@OPERATORS
def test_what_is_taken(operator, on):
    leaves, fn = operator()
    on(7)
    fn()  # let go of
    on(9, True)
    first = fn(), fn()  # twice in one capture
    on(0)
    eager = fn()
    on(9, True)
    second = fn()  # the node is the capture's own
    del first, eager, second
    on(8, True)
    twice = leaves[-1] * 2  # in the same capture
    held = fn(), fn()
    on(3, True)
    with pytest.raises(RuntimeError, match="eager graph"):  # the other capture's graph
        fn()
    assert twice.requires_grad and held[0].requires_grad


def test_inputs_that_are_no_leaves(on):
    x = torch.zeros((2, 5), requires_grad=True)
    on(0)
    y = x * 1
    alive = pag.distill_top(y, torch.zeros((2, 1), dtype=torch.int64), torch.zeros(2, 1))["loss"]
    on(7, True)
    pag.distill_top(y, torch.zeros((2, 1), dtype=torch.int64), torch.zeros(2, 1))
    assert alive.requires_grad
