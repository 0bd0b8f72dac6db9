"""Rows of the vocabulary losses at the ends of the number range: what has no
value says so in the loss as in the gradient, what has one gets it."""
import numpy as np
import pytest

from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


def cu(a, dtype=torch.float32):
    return torch.tensor(a, dtype=dtype, device="cuda")


def logits(rows, vocab, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * 2.5).to(DT[dtype]).cuda()


@pytest.mark.parametrize("kl", [0.0, 0.1])
@pytest.mark.parametrize("with_old", [False, True])
@pytest.mark.parametrize("dtype,vocab", [("f32", 40), ("bf16", 5003), ("f16", 70001)])
def test_policy_rows_without_a_value_have_no_loss(mg, dtype, vocab, with_old, kl):
    """No finite logit, a NaN logit, a NaN old value or a NaN advantage: loss and gradient are NaN, and the rows
    beside them are what they are alone."""
    x = logits(6, vocab, dtype, 1)
    x[1] = -INF
    x[2, vocab // 2] = NAN
    old, adv = cu([-3.0] * 6), cu([1.0, -1.0, 0.5, 2.0, 1.5, -2.0])
    old[3] = NAN
    adv[4] = NAN
    kw = dict(old_logp=old if with_old else None, ref_logp=cu([-2.0] * 6) if kl else None, kl_coef=kl)
    loss, logp, g = mg.muon_policy_loss(x, cu([1, 3, 5, 7, 9, 11], torch.int64), adv, **kw)
    bad = [1, 2, 4] + ([3] if with_old else [])
    for r in range(6):
        assert bool(torch.isnan(loss[r])) == (r in bad), r
        assert bool(torch.isnan(g[r]).all() if r in bad else not torch.isnan(g[r]).any()), r
    assert torch.isnan(logp[1:3]).all() and torch.isfinite(logp[3:]).all()
    one = dict(kw, old_logp=old[5:] if with_old else None, ref_logp=cu([-2.0]) if kl else None)
    alone = mg.muon_policy_loss(x[5:], cu([11], torch.int64), adv[5:], **one)
    assert torch.equal(alone[0], loss[5:]) and torch.equal(alone[2], g[5:])


def test_policy_ratio_beyond_the_range(mg):
    """exp(logp - old) over the largest fp32 number: with no advantage the row has loss and gradient 0, with a
    positive one the clipped loss and gradient 0."""
    x = logits(3, 500, "f32", 2)
    x[:, 7] = 30.0                              # logp near 0
    adv = cu([0.0, 1.5, 0.0])
    old = cu([-100.0, -100.0, -INF])
    loss, logp, g = mg.muon_policy_loss(x, cu([7, 7, 7], torch.int64), adv, old, clip_high=0.25)
    assert loss.tolist() == [0.0, -1.875, 0.0] and not g.any()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,vocab", [("f32", 40), ("bf16", 5003), ("f16", 70001)])
def test_distill_rows_without_a_distribution_have_no_loss(mg, dtype, vocab, tail):
    """No finite logit or a NaN logit, with entries listed and with padding alone: loss and gradient are NaN."""
    x = logits(6, vocab, dtype, 3)
    x[1] = x[2] = -INF
    x[3, vocab - 1] = x[4, vocab - 1] = NAN
    idx = cu([[1, 9, -1]] * 6, torch.int64)
    idx[2] = idx[4] = idx[5] = -1
    t = cu([[1.0, 2.0, 3.0]] * 6)
    lse = cu([3.0] * 6) if tail else None
    loss, g = mg.muon_distill_loss(x, idx, t, teacher_lse=lse)
    for r in range(6):
        nan = 1 <= r <= 4
        assert bool(torch.isnan(loss[r])) == nan, r
        assert bool(torch.isnan(g[r]).all() if nan else torch.isfinite(g[r]).all()), r
    assert loss[5] == 0 if not tail else abs(loss[5].item()) < 1e-6


@pytest.mark.parametrize("smoothing", [0.0, 0.25, 1.0])
@pytest.mark.parametrize("side", [0, 1])
def test_preference_with_a_banned_label(mg, side, smoothing):
    """A label of probability 0 on one side: h is -inf or inf, each sigmoid's logarithm 0 or infinite, and the
    gradient, whose sigmoids are 0 and 1, finite.  Smoothing's own term follows the same rule."""
    x = logits(4, 60, "f32", 4)
    tok = np.array([3, 5, 7, 9])
    x[2 * side, tok[2 * side]] = -INF
    bounds = [0, 2, 4]
    loss, seq, g = mg.muon_preference_loss(x, cu(tok, torch.int64), cu(bounds, torch.int64), beta=0.5,
                                           label_smoothing=smoothing)
    weight = smoothing if side else 1 - smoothing       # of the term that is infinite
    assert loss[0].item() == (INF if weight else 0.0)
    assert seq[side].item() == -INF and torch.isfinite(seq[1 - side])
    # dL/dh is weight or -weight; the rows' softmax is finite, and 0 at the banned label
    X = x.double().cpu().numpy()
    q = np.exp(X - X.max(1, keepdims=True))
    q /= q.sum(1, keepdims=True)
    one = np.zeros_like(q)
    one[np.arange(4), tok] = 1
    dh = weight if side else -weight
    want = 0.5 * dh * np.array([1, 1, -1, -1.0])[:, None] * (one - q)
    assert np.abs(g.double().cpu().numpy() - want).max() <= 2.0 ** -21 * 32      # 32: the spread of the logits


def test_preference_smoothed_loss_far_from_the_margin(mg):
    """-log sigmoid(-h) at h near -30 is e^h: within e^h times the error of h (a few roundings of 32)."""
    x = logits(2, 60, "f32", 5)
    tok, bounds = np.array([3, 5]), np.array([0, 1, 2])
    loss, _, _ = mg.muon_preference_loss(x, cu(tok, torch.int64), cu(bounds, torch.int64), margin=30.0, beta=0.25,
                                         label_smoothing=1.0)
    want, _, _ = lo.preference(x.double().cpu().numpy(), tok, bounds, margin=30.0, beta=0.25, smoothing=1.0)
    assert 0 < want[0] < 1e-11
    assert abs(loss[0].item() / want[0] - 1) <= 4 * 2.0 ** -24 * 32 + 2.0 ** -20
