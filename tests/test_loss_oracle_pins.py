"""Pins of the vocabulary-loss oracle: its gradients against central
differences of its own losses, and closed forms.  Step 1e-5 in fp64: the
difference quotient carries a truncation error of order 1e-10 and a rounding
error of order 1e-16 |loss| / 1e-5, so 1e-7 of the row's scale is ample."""
import numpy as np
import pytest

from oracle import loss_oracle as lo


def _differences(total, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = 1e-5
        g[i] = (total(x + d) - total(x - d)) / 2e-5
    return g


@pytest.mark.parametrize("temperature", [0.7, 1.0, 2.5])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_is_the_difference_quotient(temperature, tail):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(3, 11)) * 2
    idx = np.array([[0, 4, 10], [2, 2, -1], [7, 11, 3]])     # a repeated index, two paddings
    t = rng.normal(size=(3, 3)) * 2
    lse = np.array([2.5, 3.0, 4.0]) if tail else None
    kw = dict(lse=lse, weights=[1.0, 0.5, 2.0], temperature=temperature)
    loss, grad = lo.distill(x, idx, t, **kw)
    num = _differences(lambda y: lo.distill(y, idx, t, **kw)[0].sum(), x)
    assert np.abs(grad - num).max() < 1e-7


def test_distill_of_the_teachers_own_logits_is_zero():
    rng = np.random.default_rng(4)
    x = rng.normal(size=(2, 6))
    idx = np.tile(np.arange(6), (2, 1))
    loss, grad = lo.distill(x, idx, x + 3.0)
    assert np.abs(loss).max() < 1e-14 and np.abs(grad).max() < 1e-14
    lse = np.log(np.exp(x).sum(1))
    loss, grad = lo.distill(x, idx[:, :3], x[:, :3], lse=lse)       # the rest as one class
    assert np.abs(loss).max() < 1e-14 and np.abs(grad).max() < 1e-14


@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_gradient_is_the_difference_quotient(kl):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(6, 9))
    tok = np.array([0, 8, 3, 3, -100, 5])
    kw = dict(ref=rng.normal(size=6) - 2, weights=[1, 1, 0.5, 1, 1, 0], temperature=0.8, clip_low=0.2,
              clip_high=0.3, kl=kl)
    base = lo.policy(x, tok, np.ones(6), **{**kw, "old": np.zeros(6)})[1]
    kw["old"] = base + np.array([0.0, 0.5, -0.5, 0.1, 0.0, 0.0])     # ratios 1, below, above, inside
    adv = np.array([1.0, -1.0, 1.0, -2.0, 1.0, 1.0])
    loss, logp, grad = lo.policy(x, tok, adv, **kw)
    num = _differences(lambda y: lo.policy(y, tok, adv, **kw)[0].sum(), x)
    assert np.abs(grad - num).max() < 1e-7
    if not kl:
        assert not grad[1].any() and not grad[2].any()       # both clipped on the favoured side
    assert not grad[4].any() and not grad[5].any() and loss[4] == loss[5] == 0


@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient_is_the_difference_quotient(average):
    rng = np.random.default_rng(6)
    x = rng.normal(size=(12, 7))
    tok = np.array([1, -100, 3, 6, 0, 2, -1, -1, 5, 4, 4, 2])
    bounds = [0, 3, 6, 8, 11]                # the second pair's chosen sequence has no label; row 11 is outside
    kw = dict(ref=rng.normal(size=4), weights=[1.0, 0.5], beta=0.7, margin=0.2, smoothing=0.1, average=average)
    loss, seq, grad = lo.preference(x, tok, bounds, **kw)
    num = _differences(lambda y: lo.preference(y, tok, bounds, **kw)[0].sum(), x)
    assert np.abs(grad - num).max() < 1e-7
    assert seq[2] == 0 and not grad[11].any() and not grad[1].any()


def test_preference_closed_form():
    """Two-entry rows: log-probabilities of 1/2 each, so h = 0 without a reference."""
    loss, seq, grad = lo.preference(np.zeros((2, 2)), np.array([0, 1]), [0, 1, 2], beta=2.0)
    assert np.allclose(loss, np.log(2)) and np.allclose(seq, -np.log(2))
    assert np.allclose(grad, [[-0.5, 0.5], [-0.5, 0.5]])
