"""Argument checks of the vocabulary losses through the C ABI: every refusal
happens before any device use.  The pointers are placeholders, so calls that
would pass the checks are only made where there is no CUDA device."""
import pytest

P = 0x10000


@pytest.fixture(scope="module")
def mg():
    from newton_schulz_frobenius_gb300 import _build
    _build.build()
    import newton_schulz_frobenius_gb300 as pkg
    pkg.lib()
    return pkg


def distill(mg, **kw):
    a = dict(logits=P, ld=64, rows=4, vocab=64, dtype=mg.MUON_BF16, idx=P, idx_dtype=mg.MUON_I32, val=P,
             val_dtype=mg.MUON_BF16, k=8, lse=None, weights=None, temperature=1.0, loss=P, grad=P, ldg=64)
    a.update(kw)
    return mg.lib().muon_distill_loss(*a.values(), None)


def policy(mg, **kw):
    a = dict(logits=P, ld=64, rows=4, vocab=64, dtype=mg.MUON_BF16, tok=P, tok_dtype=mg.MUON_I64, adv=P, old=P,
             ref=P, weights=None, temperature=1.0, lo=0.2, hi=0.2, kl=0.1, loss=P, logp=P, grad=P, ldg=64)
    a.update(kw)
    return mg.lib().muon_policy_loss(*a.values(), None)


def preference(mg, **kw):
    a = dict(logits=P, ld=64, rows=4, vocab=64, dtype=mg.MUON_BF16, tok=P, tok_dtype=mg.MUON_I64, bounds=P,
             bounds_dtype=mg.MUON_I32, pairs=1, ref=None, weights=None, beta=0.1, margin=0.0, smoothing=0.0,
             average=0, loss=P, seq=P, grad=P, ldg=64)
    a.update(kw)
    return mg.lib().muon_preference_loss(*a.values(), None)


NAN, INF = float("nan"), float("inf")
SHARED = [dict(logits=None), dict(grad=None), dict(rows=-1), dict(rows=1 << 31), dict(vocab=0),
          dict(vocab=(1 << 19) + 1, ld=1 << 21, ldg=1 << 21), dict(ld=63), dict(ldg=63), dict(ld=65),
          dict(ld=1 << 61, ldg=1 << 61), dict(logits=P + 1), dict(grad=P + 64), dict(loss=None)]


@pytest.mark.parametrize("bad", SHARED, ids=str)
@pytest.mark.parametrize("call", [distill, policy, preference])
def test_shared_refusals(mg, call, bad):
    assert call(mg, **bad) == mg.MUON_EINVAL
    assert mg.last_error_message()


@pytest.mark.parametrize("call", [distill, policy, preference])
def test_unknown_types_are_refused(mg, call):
    assert call(mg, dtype=7) == mg.MUON_EDTYPE
    assert call(mg, **{"idx_dtype" if call is distill else "tok_dtype": 0}) == mg.MUON_EDTYPE


@pytest.mark.parametrize("call,bad", [
    (distill, dict(k=0)), (distill, dict(k=1025)), (distill, dict(idx=None)), (distill, dict(val=None)),
    (distill, dict(temperature=0.0)), (distill, dict(temperature=-1.0)), (distill, dict(temperature=NAN)),
    (distill, dict(temperature=INF)), (distill, dict(temperature=1e-40)),
    (policy, dict(tok=None)), (policy, dict(adv=None)), (policy, dict(logp=None)), (policy, dict(ref=None)),
    (policy, dict(lo=-0.1)), (policy, dict(lo=1.1)), (policy, dict(hi=-0.1)), (policy, dict(hi=NAN)),
    (policy, dict(kl=INF)), (policy, dict(temperature=0.0)),
    (preference, dict(tok=None)), (preference, dict(bounds=None)), (preference, dict(seq=None)),
    (preference, dict(pairs=-1)), (preference, dict(pairs=1 << 30)), (preference, dict(beta=NAN)),
    (preference, dict(margin=INF)), (preference, dict(smoothing=-0.1)), (preference, dict(smoothing=1.5)),
], ids=lambda v: str(v) if isinstance(v, dict) else v.__name__)
def test_own_refusals(mg, call, bad):
    assert call(mg, **bad) == mg.MUON_EINVAL


def test_more_types(mg):
    assert distill(mg, val_dtype=9) == mg.MUON_EDTYPE
    assert preference(mg, bounds_dtype=3) == mg.MUON_EDTYPE


def test_no_rows_is_valid(mg):
    assert distill(mg, rows=0, logits=None, grad=None, idx=None, val=None, loss=None) == mg.MUON_OK
    assert policy(mg, rows=0, logits=None, grad=None, tok=None, adv=None, loss=None, logp=None) == mg.MUON_OK
    assert preference(mg, rows=0, pairs=0, logits=None, grad=None, tok=None, bounds=None, loss=None,
                      seq=None) == mg.MUON_OK


def test_good_arguments_reach_the_device(mg):
    import torch
    if torch.cuda.is_available():
        pytest.skip("placeholder pointers: host-only check")
    for call in (distill, policy, preference):
        assert call(mg) not in (mg.MUON_OK, mg.MUON_EINVAL, mg.MUON_EDTYPE)      # stops at the missing device
    assert policy(mg, ref=None, old=None, kl=0.0) not in (mg.MUON_OK, mg.MUON_EINVAL)


def test_binding_refuses_tensors_it_cannot_pass(mg):
    import torch
    x = torch.zeros(2, 8)
    tok = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        mg.muon_policy_loss(x, tok, torch.zeros(2))              # not on the device
    with pytest.raises(ValueError):
        mg.muon_preference_loss(x, tok, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        mg.muon_distill_loss(x, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3))
