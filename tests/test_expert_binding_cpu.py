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


def test_given_gradients_that_overlap_are_refused(reached):
    """The products read their operands while the weights' gradients are written."""
    rows, experts, hidden, ffn = 6, 2, 8, 16
    x, gate, up, dh = bf(rows, hidden), bf(rows, ffn), bf(rows, ffn), bf(rows, ffn)
    size = experts * ffn * hidden
    pool = on(torch.zeros(4 * size, dtype=torch.bfloat16))

    def part(at):
        return pool[at:at + size].view(experts, ffn, hidden)
    wg, wu, dg = part(0), part(size), part(2 * size)
    bounds = on(torch.zeros(experts + 1, dtype=torch.int32))

    def glu(**kw):
        return mg.muon_expert_glu_backward(x, wg, wu, gate, up, dh, bounds, **kw)

    def linear(**kw):
        return mg.muon_expert_linear_backward(x, wg, dh, bounds, **kw)
    for kw in (dict(dw_gate=dg, dw_up=dg), dict(dw_gate=wg), dict(dw_up=wg), dict(dw_gate=wu), dict(dw_up=part(2 * size - 1)),
               dict(dw_gate=dg, dw_up=part(2 * size + 8)), dict(dw_gate=part(size + 8))):
        refused(reached, lambda: glu(**kw))
    for kw in (dict(dw=wg), dict(dw=part(size - 1)), dict(dw=part(1))):
        refused(reached, lambda: linear(**kw))
    got = glu(dw_gate=dg, dw_up=part(3 * size))         # next to each other
    assert got[1] is dg and reached == ["muon_expert_glu_backward"]
    assert linear(dw=wu)[1] is wu


def test_dropout_out_that_overlaps_is_refused(reached):
    """out may be x or residual, element for element, but no shifted part of them."""
    pool = on(torch.zeros(400, dtype=torch.float32))
    x, residual = pool[:100], pool[100:200]
    for out in (pool[1:101], pool[99:199], pool[101:201], pool[150:250]):
        refused(reached, lambda: mg.muon_dropout(x, 0.5, residual=residual, out=out))
    state = on(torch.zeros(2, dtype=torch.int64))
    refused(reached, lambda: mg.muon_dropout(state.view(torch.float32), 0.5, state=state, out=state.view(torch.float32)))
    for out in (x, residual, pool[200:300], pool[300:]):
        assert mg.muon_dropout(x, 0.5, residual=residual, out=out) is out
    assert mg.muon_dropout(x, 0.5, residual=x, out=x) is x
    assert reached == ["muon_dropout"] * 5


def test_the_experts_products_can_be_armed():
    """The bounded-wait test hook knows their kernel; arming is host state only."""
    from newton_schulz_frobenius_gb300 import _build
    _build.build()
    mg.muon_debug_arm_stall(mg.STALL_EXPERT, 1 << 20)
    mg.muon_debug_arm_stall(0)
    for kernel, stage in ((mg.STALL_EXPERT, -1), (mg.STALL_EXPERT, (1 << 20) + 1), (mg.STALL_EXPERT + 1, 0)):
        with pytest.raises(mg.MuonError):
            mg.muon_debug_arm_stall(kernel, stage)
