"""Argument checks of the experts' rows and of dropout: every refusal happens
before any device use (placeholder pointers)."""
import pytest

P = 0x10000


@pytest.fixture(scope="module")
def mg():
    from newton_schulz_frobenius_gb300 import _build
    _build.build()
    import newton_schulz_frobenius_gb300 as pkg
    pkg.lib()
    return pkg


def sort(mg, **kw):
    a = dict(experts=P, index=mg.MUON_I32, slots=8, num=4, row_of=P, slot_of=P, bounds=P)
    a.update(kw)
    return mg.lib().muon_expert_sort(*a.values(), None)


def dispatch(mg, **kw):
    a = dict(x=P, ld=64, tokens=4, k=2, hidden=64, dtype=mg.MUON_BF16, row_of=P, bounds=P, num=4, out=P)
    a.update(kw)
    return mg.lib().muon_expert_dispatch(*a.values(), None)


def combine(mg, **kw):
    a = dict(x=P, tokens=4, k=2, hidden=64, dtype=mg.MUON_BF16, row_of=P, bounds=P, num=4, weights=P, residual=P, ld=64,
             out=P)
    a.update(kw)
    return mg.lib().muon_expert_combine(*a.values(), None)


def backward(mg, **kw):
    a = dict(dy=P, ld=64, x=P, tokens=4, k=2, hidden=64, dtype=mg.MUON_BF16, row_of=P, bounds=P, num=4, weights=P,
             out=P, dw=P)
    a.update(kw)
    return mg.lib().muon_expert_combine_backward(*a.values(), None)


def dropout(mg, **kw):
    a = dict(x=P, residual=P, y=P, n=8, dtype=mg.MUON_BF16, p=0.1, seed=0, offset=0, state=P)
    a.update(kw)
    return mg.lib().muon_dropout(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(experts=None), dict(row_of=None), dict(slot_of=None), dict(bounds=None),
                                 dict(slots=-1), dict(slots=(1 << 24) + 1), dict(num=0), dict(num=1025),
                                 dict(row_of=P + 2), dict(index=64, experts=P + 4)], ids=str)
def test_sort_refuses(mg, bad):
    assert sort(mg, **bad) == mg.MUON_EINVAL and mg.last_error_message()


@pytest.mark.parametrize("call", [dispatch, combine, backward])
@pytest.mark.parametrize("bad", [dict(x=None), dict(row_of=None), dict(bounds=None), dict(out=None), dict(tokens=-1),
                                 dict(tokens=(1 << 23) + 1), dict(k=0), dict(k=1025), dict(hidden=0),
                                 dict(hidden=(1 << 20) + 1), dict(num=0), dict(num=1025), dict(ld=63), dict(x=P + 1),
                                 dict(row_of=P + 2)], ids=str)
def test_rows_refuse(mg, call, bad):
    assert call(mg, **bad) == mg.MUON_EINVAL and mg.last_error_message()


@pytest.mark.parametrize("bad", [dict(dy=None), dict(weights=None), dict(dw=None), dict(dw=P + 1)], ids=str)
def test_backward_refuses(mg, bad):
    assert backward(mg, **bad) == mg.MUON_EINVAL


@pytest.mark.parametrize("bad", [dict(x=None), dict(y=None), dict(n=-1), dict(n=(1 << 40) + 1), dict(p=-0.01),
                                 dict(p=1.01), dict(p=float("nan")), dict(x=P + 1), dict(residual=P + 1),
                                 dict(state=P + 4)], ids=str)
def test_dropout_refuses(mg, bad):
    assert dropout(mg, **bad) == mg.MUON_EINVAL and mg.last_error_message()


def test_types(mg):
    assert sort(mg, index=7) == mg.MUON_EDTYPE
    for call in (dispatch, combine, backward, dropout):
        assert call(mg, dtype=9) == mg.MUON_EDTYPE


def test_nothing_to_do(mg):
    for call in (dispatch, combine, backward):
        assert call(mg, tokens=0, x=None) == mg.MUON_OK
    assert dropout(mg, n=0, x=None) == mg.MUON_OK


def test_binding_refuses(mg):
    import torch
    x, i = torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mg.muon_dropout(x, 0.5)                 # not on the device
    with pytest.raises(ValueError):
        mg.muon_expert_sort(i, 4)
    with pytest.raises(ValueError):
        mg.muon_expert_dispatch(x, i, i[0])
    with pytest.raises(ValueError):
        mg.muon_expert_combine(x, i, i[0])
    with pytest.raises(ValueError):
        mg.muon_expert_combine_backward(x, x, i, i[0], x)
