"""Argument checks of the gated feed-forward block through the C ABI: every
refusal happens before any device use (placeholder pointers)."""
import pytest

P = 0x10000


@pytest.fixture(scope="module")
def mg():
    from newton_schulz_frobenius_gb300 import _build
    _build.build()
    import newton_schulz_frobenius_gb300 as pkg
    pkg.lib()
    return pkg


def forward(mg, **kw):
    a = dict(x=P, wg=P, wu=P, h=P, gate=P, up=P, tokens=4, hidden=64, ffn=32, dtype=mg.MUON_BF16, act=0)
    a.update(kw)
    return mg.lib().muon_glu_forward(*a.values(), None)


def backward(mg, **kw):
    a = dict(x=P, wg=P, wu=P, gate=P, up=P, dh=P, dx=P, dwg=P, dwu=P, tokens=4, hidden=64, ffn=32,
             dtype=mg.MUON_BF16, act=0)
    a.update(kw)
    return mg.lib().muon_glu_backward(*a.values(), None)


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("bad", [dict(x=None), dict(wg=None), dict(wu=None), dict(gate=None), dict(up=None),
                                 dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(hidden=0), dict(ffn=0),
                                 dict(hidden=(1 << 20) + 1), dict(ffn=(1 << 20) + 1), dict(act=3), dict(act=-1),
                                 dict(x=P + 1)], ids=str)
def test_refusals(mg, call, bad):
    assert call(mg, **bad) == mg.MUON_EINVAL
    assert mg.last_error_message()


def test_own_refusals(mg):
    assert forward(mg, h=None) == mg.MUON_EINVAL
    assert backward(mg, dh=None) == mg.MUON_EINVAL
    assert backward(mg, dwu=None) == mg.MUON_EINVAL
    assert backward(mg, dwg=None) == mg.MUON_EINVAL


@pytest.mark.parametrize("call", [forward, backward])
def test_types(mg, call):
    assert call(mg, dtype=mg.MUON_F32) == mg.MUON_EDTYPE
    assert call(mg, dtype=9) == mg.MUON_EDTYPE


def test_nothing_asked_for(mg):
    assert forward(mg, tokens=0) == mg.MUON_OK
    assert backward(mg, dx=None, dwg=None, dwu=None) == mg.MUON_OK


def test_binding_refuses(mg):
    import torch
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mg.muon_glu_forward(x, w, w)            # not on the device
