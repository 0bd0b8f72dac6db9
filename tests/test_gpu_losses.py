"""The vocabulary losses on the GPU against the fp64 oracle.

Bars, derived from fp32 arithmetic (eps = 2^-24 per rounding).  A row whose
finite |z - max z| reaches R gets log-probabilities within
D = 2^-21 (R + 16): the exponents carry at most four roundings of a number of
size R, the sum of exponentials at most log2(V) <= 16 more, and the logarithm
and the subtraction one each.  A factor f of the gradient that is computed
from them is within f D, a probability q within q D, so

    |g - g*| <= half an ulp of the storage type + D S (q + t) + cancellations

with S the row's largest factor and t the sparse part (1 at the token, p at
the teacher's entries).  The teacher's remainder 1 - sum p carries an absolute
error of 2^-21, which reaches the entries outside its set as 2^-21 q / q_r.
"""
import numpy as np
import pytest

from oracle import loss_oracle as lo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -25}
INF = float("inf")


def matrix(rows, vocab, dtype, seed, layout="plain", scale=2.5):
    """Logits on the device: contiguous, with a pitch of its own, or off every 16-byte boundary."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g) * scale).to(DT[dtype])
    return place(x, layout)


def place(x, layout):
    rows, vocab = x.shape
    if layout == "plain":
        return x.cuda()
    pad, off = {"pitch": (24, 0), "odd": (3, 5)}[layout]
    buf = torch.full((rows * (vocab + pad) + off + 64,), 77.0, dtype=x.dtype, device="cuda")
    v = buf[off:off + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    v.copy_(x)
    return v


def f64(t):
    return t.detach().double().cpu().numpy()


def spread(x, temperature=1.0):
    """The largest finite |z - max z| of each row, and D."""
    z = np.where(np.isfinite(x), x, np.nan) / temperature
    m = np.nanmax(z, axis=1, keepdims=True)
    R = np.nan_to_num(np.nanmax(m - z, axis=1))
    return 2.0 ** -21 * (R + 16)


def softmax(x, temperature=1.0):
    z = x / temperature
    e = np.exp(z - z.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def check_grad(got, want, err, dtype):
    bound = ULP[dtype] * np.abs(want) * 1.01 + TINY[dtype] + err
    bad = np.abs(got - want) > bound
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert not bad.any(), (int(bad.sum()), np.abs(got - want)[bad].max(), bound[bad].min())


VOCABS = [1, 2, 7, 8, 33, 1000, 4099, 32000, 50257, 70001, 131072, 270001]
LAYOUTS = ["plain", "pitch", "odd"]


def policy_inputs(x, rows, seed, temperature):
    rng = np.random.default_rng(seed)
    X = f64(x)
    tok = rng.integers(0, X.shape[1], rows)
    lp = np.log(softmax(X, temperature))[np.arange(rows), tok]
    ratio = rng.choice([0.5, 0.9, 1.0, 1.1, 1.6], rows)
    old = (lp - np.log(ratio)).astype(np.float32)
    ref = (lp + rng.normal(size=rows) * 0.5).astype(np.float32)
    adv = rng.normal(size=rows).astype(np.float32)
    w = rng.choice([0.0, 1.0, 0.25], rows, p=[0.2, 0.4, 0.4]).astype(np.float32)
    return X, tok, old, ref, adv, w


def cu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def check_policy(mg, x, dtype, seed=0, temperature=1.0, kl=0.1, grad=None, stream=None, tok=None, w=None,
                 index=torch.int64):
    rows = x.shape[0]
    X, tk, old, ref, adv, ww = policy_inputs(x, rows, seed, temperature)
    tok = tk if tok is None else tok
    w = ww if w is None else w
    args = [cu(tok, index), cu(adv)]
    kw = dict(old_logp=cu(old), ref_logp=cu(ref), weights=cu(w), temperature=temperature, clip_high=0.3, kl_coef=kl,
              grad=grad, stream=stream)
    torch.cuda.synchronize()
    loss, logp, g = mg.muon_policy_loss(x, *args, **kw)
    torch.cuda.synchronize()
    X = np.where((np.asarray(w) == 0)[:, None], 0.0, X)         # rows out of the loss may hold anything
    L, lp, G = lo.policy(X, tok, adv, old=old, ref=ref, weights=w, temperature=np.float64(temperature), clip_low=0.2,
                         clip_high=0.3, kl=float(np.float32(kl)))
    D = spread(X, temperature)
    live = (w != 0) & (tok >= 0) & (tok < X.shape[1])
    r = np.where(live, np.exp(lp - old), 0.0)
    S = w * (np.abs(adv) * r + kl * (1 + np.exp(np.where(live, ref - lp, 0.0))))
    assert np.all(np.abs(f64(logp) - lp) <= D + 1e-6)
    assert np.all(np.abs(f64(loss) - L) <= 2 * S * (D + 2.0 ** -20) + 1e-30)
    one = np.zeros_like(X)
    one[np.arange(rows)[live], np.asarray(tok)[live]] = 1.0
    check_grad(f64(g), G, (2 * S * (D + 2.0 ** -20) / temperature)[:, None] * (softmax(X, temperature) + one), dtype)
    assert not f64(g)[~live].any() and not f64(loss)[~live].any()
    return loss, logp, g


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_policy_sizes(mg, dtype, vocab):
    for layout in LAYOUTS:
        check_policy(mg, matrix(5, vocab, dtype, vocab, layout), dtype, seed=vocab)


@pytest.mark.parametrize("temperature,kl", [(0.6, 0.0), (1.7, 0.05), (30.0, 1.0)])
def test_policy_temperature_and_kl(mg, temperature, kl):
    check_policy(mg, matrix(33, 5003, "bf16", 1), "bf16", seed=2, temperature=temperature, kl=kl)


@pytest.mark.parametrize("rows", [1, 2, 151, 700, 2500])
def test_policy_rows(mg, rows):
    check_policy(mg, matrix(rows, 1031, "f16", rows), "f16", seed=rows, index=torch.int32)


def test_policy_first_step_without_old_values(mg):
    x = matrix(7, 999, "f32", 3)
    X, tok, _, _, adv, _ = policy_inputs(x, 7, 3, 1.0)
    loss, logp, g = mg.muon_policy_loss(x, cu(tok), cu(adv))
    L, lp, G = lo.policy(X, tok, adv)
    D = spread(X)
    one = np.zeros_like(X)
    one[np.arange(7), tok] = 1
    assert np.all(np.abs(f64(loss) - L) <= 1e-6 * np.abs(adv))
    check_grad(f64(g), G, (np.abs(adv) * 2 * D)[:, None] * (softmax(X) + one), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_policy_masked_rows_may_hold_anything(mg, dtype):
    x = matrix(6, 777, dtype, 9)
    x[1] = float("nan")
    x[2] = INF
    x[4] = -INF
    tok = np.array([5, 1, 2, 776, -100, 777])       # two labels outside the vocabulary
    w = np.array([1, 0, 0, 0.5, 1, 1], np.float32)
    xs = x.clone()
    xs[[1, 2, 4]] = 0
    rows = x.shape[0]
    X, _, old, ref, adv, _ = policy_inputs(xs, rows, 1, 1.0)
    loss, logp, g = mg.muon_policy_loss(x, cu(tok), cu(adv), cu(old), cu(ref), cu(w), kl_coef=0.1)
    L, lp, G = lo.policy(X, tok, adv, old=old, ref=ref, weights=w, kl=float(np.float32(0.1)))
    for r in (1, 2, 4, 5):
        assert not f64(g)[r].any() and f64(loss)[r] == 0 and f64(logp)[r] == 0
    D = spread(X)
    assert np.all(np.abs(f64(logp) - lp) <= D + 1e-6)
    assert np.all(np.isfinite(f64(g)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_banned_entries_and_the_lowest_value(mg, dtype):
    """-inf and the type's lowest value in the row; a row all of the lowest value is uniform."""
    low = torch.finfo(DT[dtype]).min
    x = matrix(4, 203, dtype, 11)
    x[0, 100:] = -INF
    x[1, ::2] = low
    x[2] = low
    x[3, :202] = -INF                           # one entry left
    tok = np.array([3, 1, 17, 202])
    adv = np.ones(4, np.float32)
    for temperature in (0.5, 1.0, 2.0):
        loss, logp, g = mg.muon_policy_loss(x, cu(tok), cu(adv), temperature=temperature)
        X = f64(x)
        q = softmax(X, temperature)
        one = np.zeros_like(q)
        one[np.arange(4), tok] = 1
        D = np.array([2.0 ** -21 * 60] * 4)
        check_grad(f64(g), -(one - q) / temperature, (D / temperature)[:, None] * (q + one), dtype)
        assert np.all(np.abs(f64(logp) - np.log(q[np.arange(4), tok])) <= D)
        assert not f64(g)[0, 100:].any() and not f64(g)[3].any()


def test_row_without_a_finite_logit_gives_nan(mg):
    x = torch.full((1, 40), -INF, device="cuda")
    loss, logp, g = mg.muon_policy_loss(x, cu(np.array([1])), cu(np.ones(1, np.float32)))
    assert np.isnan(f64(g)).all() and np.isnan(f64(logp)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [500, 50257, 131072])
def test_gradient_in_place_and_beside(mg, dtype, vocab):
    """In place of the logits, and into a matrix with other alignment, both equal the plain call bit for bit;
    columns between the rows stay as they were."""
    x = matrix(9, vocab, dtype, 5, "pitch")
    _, _, want = check_policy(mg, x, dtype, seed=4)
    for layout in LAYOUTS:
        out = place(torch.zeros(9, vocab, dtype=DT[dtype]), layout)
        check_policy(mg, x, dtype, seed=4, grad=out)
        assert torch.equal(out, want)
        if layout != "plain":
            pad = out.as_strided((9, out.stride(0) - vocab), (out.stride(0), 1), out.storage_offset() + vocab)
            assert bool((pad == 77.0).all())
    X, tok, old, ref, adv, w = policy_inputs(x, 9, 4, 1.0)
    _, _, g = mg.muon_policy_loss(x, cu(tok), cu(adv), cu(old), cu(ref), cu(w), clip_high=0.3, kl_coef=0.1, grad=x)
    assert g is x and torch.equal(x, want)


def test_other_stream_and_repeat(mg):
    x = matrix(64, 33001, "bf16", 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = check_policy(mg, x, "bf16", seed=8)
    b = check_policy(mg, x, "bf16", seed=8, stream=s)
    c = check_policy(mg, x, "bf16", seed=8)
    for u, v, t in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, t)


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

def teacher(x, k, seed, temperature, tail, index=torch.int32, dtype=None):
    rows, vocab = x.shape
    rng = np.random.default_rng(seed)
    kk = min(k, vocab)
    idx = np.stack([rng.permutation(vocab)[:kk] for _ in range(rows)])
    t = (rng.normal(size=(rows, kk)) * 2 + 4).astype(np.float32)
    t = cu(t).to(x.dtype if dtype is None else dtype)
    for r in range(rows):                       # a student near its teacher on part of the set
        x[r, torch.from_numpy(idx[r][::2]).cuda()] = t[r, ::2].to(x.dtype)
    lse = None
    if tail:
        z = f64(t) / temperature
        m = z.max(1)
        lse = (m + np.log(np.exp(z - m[:, None]).sum(1)) - np.log(rng.uniform(0.3, 0.999, rows))).astype(np.float32)
    return cu(idx, index), t, None if lse is None else cu(lse)


def check_distill(mg, x, idx, t, lse, dtype, temperature=1.0, weights=None, grad=None):
    w = np.ones(x.shape[0], np.float32) if weights is None else weights
    X = f64(x)
    X = np.where((w == 0)[:, None], 0.0, X)
    loss, g = mg.muon_distill_loss(x, idx, t, teacher_lse=lse, weights=cu(w), temperature=temperature, grad=grad)
    torch.cuda.synchronize()
    ids, T = idx.cpu().numpy(), np.nan_to_num(f64(t), nan=0.0)
    L, G = lo.distill(X, ids, T, lse=None if lse is None else f64(lse), weights=w, temperature=temperature)
    D = spread(X, temperature) + spread(np.nan_to_num(T, neginf=0.0), temperature) + 2.0 ** -20
    q = softmax(X, temperature)
    sparse = np.zeros_like(q)
    extra = np.zeros_like(q)
    la = np.zeros(len(X))
    for r in range(len(X)):
        ok = (ids[r] >= 0) & (ids[r] < X.shape[1])
        z = T[r][ok] / temperature
        if not len(z):
            continue
        p = np.exp(z - (z.max() + np.log(np.exp(z - z.max()).sum()) if lse is None else f64(lse)[r]))
        np.add.at(sparse[r], ids[r][ok], p)
        la[r] = (p * (np.abs(np.log(np.maximum(p, 1e-300))) + np.abs(np.log(np.maximum(q[r][ids[r][ok]], 1e-300))) + 1)).sum()
        if lse is not None:
            out = np.ones(X.shape[1], bool)
            out[ids[r][ok]] = False
            qr = q[r][out].sum()
            rest = 1 - p.sum()
            if qr > 0 and rest > 0:
                extra[r] = np.where(out, q[r] / qr, 0) * (2.0 ** -21 + D[r] * rest) + q[r] * 2.0 ** -21
                la[r] += (rest + 2.0 ** -21 / D[r]) * (abs(np.log(rest / qr)) + 2)
    scale = (w * temperature)[:, None]
    assert np.all(np.abs(f64(loss) - L) <= w * temperature ** 2 * D * (la + 1))
    check_grad(f64(g), G, scale * (D[:, None] * (2 * q + 2 * sparse) + extra), dtype)
    return loss, g


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_distill_sizes(mg, vocab, dtype, tail):
    for k, layout in ((1, "odd"), (17, "plain"), (64, "pitch"), (300, "odd")):
        x = matrix(4, vocab, dtype, vocab + k, layout)
        idx, t, lse = teacher(x, k, vocab + k, 1.0, tail)
        check_distill(mg, x, idx, t, lse, dtype)


@pytest.mark.parametrize("temperature", [0.5, 2.0, 8.0])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_temperature_weights_and_types(mg, temperature, tail):
    x = matrix(40, 9001, "bf16", 21)
    idx, t, lse = teacher(x, 50, 22, temperature, tail, index=torch.int64, dtype=torch.float32)
    w = np.random.default_rng(1).choice([0.0, 1.0, 0.125], 40).astype(np.float32)
    x[int(np.flatnonzero(w == 0)[0])] = float("nan")
    check_distill(mg, x, idx, t, lse, "bf16", temperature=temperature, weights=w)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_repeated_and_padded_entries(mg, tail):
    x = matrix(5, 600, "f32", 23)
    idx, t, lse = teacher(x, 12, 24, 1.0, tail, index=torch.int64)
    idx[0, 5] = idx[0, 0]
    idx[0, 7] = idx[0, 0]
    idx[1, 3:] = -1
    idx[2, 4] = 1 << 40
    idx[2, 5] = 600
    idx[3, :] = -100                            # nothing listed
    t[1, 3:] = float("nan")                     # padding holds anything
    t[3, :] = float("nan")
    t[4, 2] = -INF                              # listed with probability 0
    if tail:                                    # masses below one with the repeats counted
        z = f64(t)
        ok = ((idx >= 0) & (idx < 600)).cpu().numpy()
        z = np.where(ok, z, -np.inf)
        m = np.where(ok.any(1), z.max(1), 0.0)
        s = np.exp(z - m[:, None]).sum(1)
        lse = cu((m + np.log(np.where(s > 0, s, 1.0)) + 0.3).astype(np.float32))
    loss, g = check_distill(mg, x, idx, t, lse, "f32")
    assert f64(loss)[3] == 0 and np.abs(f64(g)[3]).max() <= 2.0 ** -20


def test_distill_whole_vocabulary_listed(mg):
    """Every entry listed: nothing is outside, and the rest's term drops out."""
    x = matrix(3, 40, "f32", 25)
    idx, t, lse = teacher(x, 40, 26, 1.0, True)
    check_distill(mg, x, idx, t, lse, "f32")


def test_distill_a_thousand_entries(mg):
    x = matrix(3, 5000, "bf16", 27)
    idx, t, lse = teacher(x, 1024, 28, 1.0, True)
    check_distill(mg, x, idx, t, lse, "bf16")


@pytest.mark.parametrize("tail", [False, True])
def test_distill_in_place(mg, tail):
    x = matrix(6, 40001, "f16", 29)
    idx, t, lse = teacher(x, 33, 30, 1.0, tail)
    loss, want = check_distill(mg, x, idx, t, lse, "f16")
    loss2, g = mg.muon_distill_loss(x, idx, t, teacher_lse=lse, grad=x)
    assert torch.equal(g, want) and torch.equal(loss, loss2)


# ---------------------------------------------------------------------------
# preference
# ---------------------------------------------------------------------------

def check_preference(mg, x, tok, bounds, ref, w, dtype, beta=0.1, margin=0.0, smoothing=0.0, average=False,
                     index=torch.int64, grad=None):
    X = f64(x)
    loss, seq, g = mg.muon_preference_loss(x, cu(tok, index), cu(np.array(bounds), index), None if ref is None else cu(ref),
                                           None if w is None else cu(w), beta=beta, margin=margin,
                                           label_smoothing=smoothing, average=average, grad=grad)
    torch.cuda.synchronize()
    live = (tok >= 0) & (tok < X.shape[1])
    Xs = np.where(live[:, None], X, 0.0)
    f = lambda v: float(np.float32(v))       # noqa: E731  as the library receives it
    L, S, G = lo.preference(Xs, tok, bounds, ref=ref, weights=w, beta=f(beta), margin=f(margin), smoothing=f(smoothing),
                            average=average)
    D = spread(Xs)
    pairs = (len(bounds) - 1) // 2
    e_seq = np.array([(D * live)[bounds[i]:bounds[i + 1]].sum() for i in range(2 * pairs)])
    if average:
        n = np.array([max(1, live[bounds[i]:bounds[i + 1]].sum()) for i in range(2 * pairs)])
        e_seq = e_seq / n
    assert np.all(np.abs(f64(seq) - S) <= e_seq + 2.0 ** -23 * np.abs(S))
    eh = beta * (e_seq[0::2] + e_seq[1::2]) + 2.0 ** -22 * (np.abs(margin) + beta * (
        np.abs(S - (0 if ref is None else ref))).reshape(-1, 2).sum(1) if pairs else 0)
    ww = np.ones(pairs) if w is None else w
    assert np.all(np.abs(f64(loss) - L) <= ww * (eh + 2.0 ** -21 * (np.abs(L / np.where(ww == 0, 1, ww)) + 1)))
    err = np.zeros_like(X)
    q = softmax(Xs)
    for s in range(2 * pairs):
        for r in range(bounds[s], bounds[s + 1]):
            if live[r]:
                c = np.abs(G[r][tok[r]] / max(1 - q[r][tok[r]], 1e-9))
                share = ww[s // 2] * beta / (n[s] if average else 1)
                err[r] = q[r] * (c * 2 * D[r] + share * (eh[s // 2] + 2.0 ** -21))
                err[r][tok[r]] += share * (eh[s // 2] + 2.0 ** -21) + c * 2 * D[r]
    check_grad(f64(g), G, err, dtype)
    return loss, seq, g


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [2, 33, 1000, 4099, 32000, 70001, 131072, 270001])
def test_preference_sizes(mg, dtype, vocab):
    rng = np.random.default_rng(vocab)
    bounds = [0, 3, 4, 4, 9, 14, 20]            # an empty chosen sequence, one token, several
    for layout in LAYOUTS:
        x = matrix(21, vocab, dtype, vocab, layout)
        tok = rng.integers(0, vocab, 21)
        tok[[1, 10]] = -100
        check_preference(mg, x, tok, bounds, (rng.normal(size=6) * 3 - 20).astype(np.float32),
                         np.array([1.0, 0.5, 2.0], np.float32), dtype, beta=0.3)


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("smoothing,margin", [(0.0, 0.0), (0.1, 0.5)])
def test_preference_options(mg, average, smoothing, margin):
    rng = np.random.default_rng(7)
    x = matrix(60, 2011, "bf16", 31)
    x[50:] = float("nan")                       # rows outside every sequence and unlabelled rows are not read
    x[5] = INF
    tok = rng.integers(0, 2011, 60)
    tok[5] = -1
    tok[50:] = -100
    tok[30:35] = 2011                           # a rejected sequence without labels
    bounds = [0, 10, 20, 30, 35, 41, 50]
    w = np.array([1.0, 0.25, 0.0], np.float32)
    loss, seq, g = check_preference(mg, x, tok, bounds, None, w, "bf16", beta=0.5, margin=margin, smoothing=smoothing,
                                    average=average, index=torch.int32)
    assert f64(loss)[2] == 0 and not f64(g)[35:].any() and f64(seq)[3] == 0


def test_preference_rows_outside_every_sequence_get_zeros(mg):
    x = matrix(10, 100, "f32", 33)
    tok = np.arange(10)
    _, _, g = check_preference(mg, x, tok, [2, 4, 7], None, None, "f32")
    assert not f64(g)[:2].any() and not f64(g)[7:].any()


def test_preference_saturated_pairs(mg):
    """Margins far beyond the exponent's range: loss |h| or 0, gradients finite."""
    x = matrix(4, 50, "f32", 34)
    tok = np.array([1, 2, 3, 4])
    ref = np.array([3000.0, 0.0, -3000.0, 0.0], np.float32)
    check_preference(mg, x, tok, [0, 1, 2, 3, 4], ref, None, "f32", beta=1.0)


def test_preference_offsets_beyond_the_rows_are_clamped(mg):
    x = matrix(4, 64, "f32", 35)
    tok = np.array([1, 2, 3, 4])
    a = mg.muon_preference_loss(x, cu(tok), cu(np.array([0, 2, 4])))
    b = mg.muon_preference_loss(x, cu(tok), cu(np.array([-5, 2, 1 << 40])))
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_preference_long_and_in_place(mg):
    rng = np.random.default_rng(8)
    rows = 900
    x = matrix(rows, 4001, "f16", 36)
    tok = rng.integers(0, 4001, rows)
    bounds = [0, 300, 500, 501, 900]
    ref = (rng.normal(size=4) * 5 - np.array([2600, 1750, 9, 3500])).astype(np.float32)
    loss, seq, want = check_preference(mg, x, tok, bounds, ref, None, "f16", beta=0.02)
    out = mg.muon_preference_loss(x, cu(tok), cu(np.array(bounds)), cu(ref), beta=0.02, grad=x)
    assert torch.equal(out[2], want) and torch.equal(out[0], loss)


def test_nothing_to_do(mg):
    x = torch.empty(0, 32, device="cuda", dtype=torch.bfloat16)
    z = torch.empty(0, dtype=torch.int64, device="cuda")
    f = torch.empty(0, device="cuda")
    assert mg.muon_policy_loss(x, z, f)[2].shape == (0, 32)
    assert mg.muon_distill_loss(x, z.view(0, 1), torch.empty(0, 1, device="cuda"))[0].numel() == 0
    # pairs of empty sequences: h = 0
    loss, seq, _ = mg.muon_preference_loss(x, z, torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert abs(float(loss[0]) - np.log(2)) < 1e-6 and not bool(seq.any())


def test_rows_past_32_bit_offsets(mg):
    """Element offsets beyond 2^31: the last rows of a 4.3 GB matrix equal the same rows on their own."""
    rows, vocab = 16500, 131072
    x = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda").normal_()
    tok = torch.randint(0, vocab, (rows,), device="cuda")
    adv = torch.ones(rows, device="cuda")
    w = torch.zeros(rows, device="cuda")
    w[-3:] = 1.0
    _, lp, g = mg.muon_policy_loss(x, tok, adv, weights=w)
    _, lp2, g2 = mg.muon_policy_loss(x[-3:].clone(), tok[-3:], adv[-3:])
    assert torch.equal(g[-3:], g2) and torch.equal(lp[-3:], lp2)


def test_refusals_on_the_device(mg):
    x = matrix(4, 64, "bf16", 37)
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    adv = torch.ones(4, device="cuda")
    with pytest.raises(mg.MuonError) as e:
        mg.muon_policy_loss(x, tok, adv, kl_coef=0.1)           # a KL term without a reference
    assert e.value.status == mg.MUON_EINVAL
    with pytest.raises(ValueError):
        mg.muon_policy_loss(x.t(), tok, adv)                    # columns, not rows, contiguous
    with pytest.raises(ValueError):
        mg.muon_policy_loss(x[:1].expand(4, 64), tok, adv)      # rows on top of one another
    with pytest.raises(ValueError):
        mg.muon_policy_loss(x, tok[:3], adv)
    with pytest.raises(TypeError):
        mg.muon_policy_loss(x, tok.float(), adv)
    with pytest.raises(TypeError):
        mg.muon_policy_loss(x, tok, adv.double())
    with pytest.raises(TypeError):
        mg.muon_policy_loss(x.double(), tok, adv)
    with pytest.raises(ValueError):
        mg.muon_policy_loss(x, tok, adv, grad=torch.empty(4, 63, dtype=x.dtype, device="cuda"))
    with pytest.raises(mg.MuonError):
        mg.muon_policy_loss(x[:2], tok[:2], adv[:2], grad=x[1:3])       # overlapping, not the same
    with pytest.raises(mg.MuonError):
        mg.muon_distill_loss(x, torch.zeros(4, 1025, dtype=torch.int32, device="cuda"),
                             torch.zeros(4, 1025, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [5, 50, 1003, 4099, 50257, 131077])
def test_gradient_rows_on_another_alignment_than_the_logits(mg, dtype, vocab):
    """The gradient's rows start elsewhere between 16-byte boundaries than the
    logits': the same bits, and nothing beside them is written."""
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    rows = 9
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randn(rows, vocab, device="cuda", generator=g).to(dt)
    tok = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    tok[1], tok[2] = 0, vocab - 1
    adv = torch.randn(rows, device="cuda", generator=g)
    w = torch.ones(rows, device="cuda")
    w[4] = 0.0
    k = min(vocab, 7)
    idx = torch.stack([torch.randperm(vocab, device="cuda", generator=g)[:k] for _ in range(rows)])
    tv = torch.randn(rows, k, device="cuda", generator=g)
    lse = torch.logsumexp(tv, 1) + 0.2
    b = torch.tensor([0, 2, 5, 6, 8], dtype=torch.int32, device="cuda")
    calls = [lambda o: mg.muon_policy_loss(x, tok, adv, weights=w, grad=o),
             lambda o: mg.muon_distill_loss(x, idx, tv, weights=w, grad=o),
             lambda o: mg.muon_distill_loss(x, idx, tv, teacher_lse=lse, weights=w, grad=o),
             lambda o: mg.muon_preference_loss(x, tok, b, grad=o)]
    for call in calls:
        want = torch.empty_like(x)
        call(want)
        for pitch in (vocab + 16, vocab + 9):
            for off in range(8):
                buf = torch.full((rows, pitch), 7.0, device="cuda", dtype=dt)
                got = buf[:, off:off + vocab]
                call(got)
                assert torch.equal(got, want), (pitch, off)
                got.fill_(7.0)
                assert bool((buf == 7.0).all()), (pitch, off)
