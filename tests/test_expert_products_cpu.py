"""Argument checks of the experts' products: every refusal happens before any
device use (placeholder pointers)."""
import ctypes

import pytest

P = 0x10000


@pytest.fixture(scope="module")
def mg():
    from newton_schulz_frobenius_gb300 import _build
    _build.build()
    import newton_schulz_frobenius_gb300 as pkg
    pkg.lib()
    return pkg


def run(mg, name, a):
    return getattr(mg.lib(), name)(*a.values(), None, ctypes.byref(ctypes.c_int64(0)), None)


def glu_forward(mg, **kw):
    a = dict(x=P, w=P, w2=P, bounds=P, y=P, gate=P, up=P, rows=4, experts=2, hidden=64, ffn=32, dtype=mg.MUON_BF16, act=0)
    return run(mg, "muon_expert_glu_forward", {**a, **kw})


def glu_backward(mg, **kw):
    a = dict(x=P, w=P, w2=P, gate=P, up=P, dy=P, bounds=P, dx=P, dw=P, dw2=P, rows=4, experts=2, hidden=64, ffn=32,
             dtype=mg.MUON_BF16, act=0)
    return run(mg, "muon_expert_glu_backward", {**a, **kw})


def linear_forward(mg, **kw):
    a = dict(x=P, w=P, bounds=P, y=P, rows=4, experts=2, hidden=64, ffn=32, dtype=mg.MUON_BF16)
    return run(mg, "muon_expert_linear_forward", {**a, **kw})


def linear_backward(mg, **kw):
    a = dict(x=P, w=P, dy=P, bounds=P, dx=P, dw=P, rows=4, experts=2, hidden=64, ffn=32, dtype=mg.MUON_BF16)
    return run(mg, "muon_expert_linear_backward", {**a, **kw})


CALLS = [glu_forward, glu_backward, linear_forward, linear_backward]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad", [dict(x=None), dict(w=None), dict(bounds=None), dict(rows=-1), dict(rows=(1 << 24) + 1),
                                 dict(experts=0), dict(experts=1025), dict(hidden=0), dict(hidden=(1 << 20) + 1),
                                 dict(ffn=0), dict(ffn=(1 << 20) + 1), dict(x=P + 1), dict(w=P + 1), dict(bounds=P + 2)],
                         ids=str)
def test_refusals(mg, call, bad):
    assert call(mg, **bad) == mg.MUON_EINVAL and mg.last_error_message()


def test_own_refusals(mg):
    for call in (glu_forward, linear_forward):
        assert call(mg, y=None) == mg.MUON_EINVAL
    for call in (glu_backward, linear_backward):
        assert call(mg, dy=None) == mg.MUON_EINVAL
    for call in (glu_forward, glu_backward):
        assert call(mg, act=3) == mg.MUON_EINVAL and call(mg, act=-1) == mg.MUON_EINVAL
        assert call(mg, w2=None) == mg.MUON_EINVAL and call(mg, gate=None) == mg.MUON_EINVAL
    assert glu_backward(mg, dw2=None) == mg.MUON_EINVAL


@pytest.mark.parametrize("call", CALLS)
def test_types(mg, call):
    assert call(mg, dtype=mg.MUON_F32) == mg.MUON_EDTYPE and call(mg, dtype=9) == mg.MUON_EDTYPE


def test_nothing_asked_for(mg):
    for call in (glu_forward, linear_forward):
        assert call(mg, rows=0, x=None) == mg.MUON_OK
    assert glu_backward(mg, dx=None, dw=None, dw2=None) == mg.MUON_OK
    assert linear_backward(mg, dx=None, dw=None) == mg.MUON_OK


def test_binding_refuses(mg):
    import torch
    x, w, b = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(3, 4, 8, dtype=torch.bfloat16), torch.zeros(4).int()
    for call in (lambda: mg.muon_expert_glu_forward(x, w, w, b), lambda: mg.muon_expert_linear_forward(x, w, b),
                 lambda: mg.muon_expert_glu_backward(x, w, w, x, x, x, b), lambda: mg.muon_expert_linear_backward(x, w, x, b)):
        with pytest.raises(ValueError):
            call()                              # not on the device
