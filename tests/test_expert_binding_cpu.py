"""Checks of the experts' and dropout's bindings that need no device: tensors that say they are on one, a library
that only notes what reaches it."""
import pytest

torch = pytest.importorskip("torch")

import newton_schulz_frobenius_gb300 as mg  # noqa: E402


class On(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def on(t):
    return t.as_subclass(On)


def bf(*shape):
    return on(torch.zeros(shape, dtype=torch.bfloat16))


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return mg.MUON_OK
        return call


@pytest.fixture
def reached(monkeypatch):
    library = Library()
    monkeypatch.setattr(mg, "lib", lambda: library)
    monkeypatch.setattr(mg, "_raw_stream", (lambda device: 0, lambda: 0))
    return library.calls


def refused(reached, call):
    reached.clear()
    with pytest.raises(ValueError):
        call()
    assert not reached


def test_weights_in_another_order_are_refused(reached):
    """k x tokens has as many elements as tokens x k, in another order."""
    tokens, k, hidden = 6, 2, 8
    row_of, bounds = on(torch.zeros(tokens, k, dtype=torch.int32)), on(torch.zeros(4, dtype=torch.int32))
    ys, dy = bf(tokens * k, hidden), bf(tokens, hidden)
    for shape in ((k, tokens), (3, 4)):
        w = on(torch.ones(shape))
        refused(reached, lambda: mg.muon_expert_combine(ys, row_of, bounds, weights=w))
        refused(reached, lambda: mg.muon_expert_combine_backward(dy, ys, row_of, bounds, w))
    for shape in ((tokens, k), (tokens * k,), (tokens, k, 1)):
        w = on(torch.ones(shape))
        mg.muon_expert_combine(ys, row_of, bounds, weights=w)
        _, dw = mg.muon_expert_combine_backward(dy, ys, row_of, bounds, w)
        assert dw.shape == (tokens, k)
    assert reached == ["muon_expert_combine", "muon_expert_combine_backward"] * 3
