"""Dropout on the GPU against the fp64 oracle: the mask bit for bit, values within
one fp32 product and sum (2^-23 of each) and one rounding to the type."""
import numpy as np
import pytest

from oracle import expert_oracle as eo

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 1e-44, "bf16": 1e-37, "f16": 2.0 ** -25}


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


def rand(n, dtype, seed, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.empty(n + off + 8, dtype=DT[dtype], device="cuda")
    v = buf[off:off + n]
    v.copy_(torch.randn(n, generator=g, device="cuda"))
    return v


def f64(t):
    return t.detach().double().cpu().numpy()


def check(mg, x, p, seed, offset, dtype, residual=None, **kw):
    X, R = f64(x), None if residual is None else f64(residual)
    y = mg.muon_dropout(x, p, residual=residual, **(kw or dict(seed=seed, offset=offset)))
    want = eo.dropout(X, p, seed, offset, R)
    size = np.abs(want - (0 if R is None else R)) + np.abs(want)
    assert (np.abs(f64(y) - want) <= HALF[dtype] * 1.001 * np.abs(want) + 2.0 ** -23 * size + TINY[dtype]).all()
    if residual is None and p > 0:
        cut = int(np.floor(p * 65536 + 0.5))
        keep = eo.drop_bits(X.size, seed, offset).reshape(X.shape) >= cut
        assert np.array_equal(f64(y) != 0, keep & (X != 0))
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 2048, 4099, 40000])
def test_values(mg, n, dtype):
    x, r = rand(n, dtype, 1), rand(n, dtype, 2)
    check(mg, x, 0.1, 3, 4, dtype)
    check(mg, x, 0.5, -1, -2, dtype, residual=r)                     # all 64 bits of both
    check(mg, x, 0.3, (1 << 40) + 5, (1 << 35) + 1, dtype)
    check(mg, x, 0.0, 3, 4, dtype, residual=r)
    assert not mg.muon_dropout(x, 1.0, seed=3).any()
    assert torch.equal(mg.muon_dropout(x, 1.0, seed=3, residual=r), r)
    assert torch.equal(mg.muon_dropout(x, 0.0, seed=3), x)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("off", [1, 2, 3, 5])
def test_alignment(mg, off, dtype):
    for a, b in ((off, off), (0, off), (off, 0)):
        check(mg, rand(1003, dtype, 1, a), 0.2, 9, 1, dtype, residual=rand(1003, dtype, 2, b))
    out = rand(1003, dtype, 4, off)
    x = rand(1003, dtype, 1)
    assert mg.muon_dropout(x, 0.2, seed=9, out=out) is out and torch.equal(out, mg.muon_dropout(x, 0.2, seed=9))


def test_shapes_share_the_mask(mg):
    """The mask follows the element's index, whatever the shape."""
    x = rand(6 * 35, "f32", 1)
    flat = mg.muon_dropout(x, 0.4, seed=7, offset=2)
    assert torch.equal(mg.muon_dropout(x.view(6, 35), 0.4, seed=7, offset=2).view(-1), flat)
    assert torch.equal(mg.muon_dropout(x.view(2, 3, 35), 0.4, seed=7, offset=2).view(-1), flat)
    assert torch.equal(mg.muon_dropout(x[:100].clone(), 0.4, seed=7, offset=2), flat[:100])
    assert mg.muon_dropout(x[:0], 0.4).numel() == 0
    for other in (dict(seed=8, offset=2), dict(seed=7, offset=3), dict(seed=7, offset=2 + (1 << 32))):
        assert not torch.equal(mg.muon_dropout(x, 0.4, **other), flat)


def test_state_on_the_device(mg):
    x = rand(5000, "bf16", 1)
    state = torch.tensor([(1 << 50) + 3, 17], device="cuda")
    y = check(mg, x, 0.25, (1 << 50) + 3, 17, "bf16", state=state)
    state[1] += 1
    assert not torch.equal(mg.muon_dropout(x, 0.25, state=state), y)
    state[1] -= 1
    assert torch.equal(mg.muon_dropout(x, 0.25, state=state), y)


def test_in_place(mg):
    for dtype in ("bf16", "f32"):
        for off in (0, 1):
            x, r = rand(3001, dtype, 1, off), rand(3001, dtype, 2, off)
            want = mg.muon_dropout(x, 0.3, seed=5, residual=r)
            version = r._version
            assert mg.muon_dropout(x, 0.3, seed=5, residual=r, out=r) is r and torch.equal(r, want) and r._version > version
            r2 = rand(3001, dtype, 2, off)
            mg.muon_dropout(x, 0.3, seed=5, residual=r2, out=x)
            assert torch.equal(x, want)


def test_what_is_dropped_does_not_count(mg):
    x = rand(4096, "f32", 1)
    keep = mg.muon_dropout(torch.ones_like(x), 0.5, seed=3) != 0
    for bad in (float("inf"), float("nan")):
        y = mg.muon_dropout(torch.where(keep, x, torch.full_like(x, bad)), 0.5, seed=3)
        assert torch.equal(y, mg.muon_dropout(x, 0.5, seed=3))


def test_gradient_is_the_same_call(mg):
    """d/dx of <dy, residual + dropout(x)> is dropout(dy): a linear map with a diagonal matrix."""
    x, dy = rand(999, "f32", 1), rand(999, "f32", 2)
    eye = mg.muon_dropout(torch.ones_like(x), 0.4, seed=11)
    assert torch.equal(mg.muon_dropout(dy, 0.4, seed=11), dy * eye)
    h = mg.muon_dropout(x + 0.5 * dy, 0.4, seed=11).double() - mg.muon_dropout(x - 0.5 * dy, 0.4, seed=11).double()
    assert ((h - mg.muon_dropout(dy, 0.4, seed=11).double()).abs() <= 2.0 ** -20 * (x.abs() + dy.abs()).double()).all()


def test_share_of_dropped(mg):
    """2^24 elements: the share kept is within five deviations of the probability, sqrt(p (1 - p) / n) each, and so is
    that of neighbours both dropped."""
    n = 1 << 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    for p in (0.1, 0.5):
        cut = int(np.floor(p * 65536 + 0.5)) / 65536
        gone = mg.muon_dropout(x, p, seed=1234, offset=p > 0.2) == 0
        assert abs(gone.double().mean().item() - cut) <= 5 * (cut * (1 - cut) / n) ** 0.5
        both = (gone[1:] & gone[:-1]).double().mean().item()
        assert abs(both - cut * cut) <= 5 * 2 * (cut * cut / n) ** 0.5


def test_many_elements(mg):
    """More elements than 32 bits index: the last ones have their own numbers (their block counts in 64 bits)."""
    n = (1 << 31) + 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = mg.muon_dropout(x, 0.5, seed=21, offset=6, out=x)
    first = (n - 24) // 8
    bits = [v for b in range(first, first + 3)
            for w in eo.philox4x32((b & eo.M32, b >> 32, 6, 0), (21, 0)) for v in (w & 0xFFFF, w >> 16)]
    assert (y[-24:] != 0).tolist() == [v >= 32768 for v in bits]


def test_refusals(mg):
    x = rand(16, "bf16", 1)
    for bad in (dict(p=-0.5), dict(p=1.5), dict(p=float("nan"))):
        with pytest.raises(mg.MuonError):
            mg.muon_dropout(x, **bad)
    for kw in (dict(residual=x[:8]), dict(residual=x.float()), dict(out=x.float()), dict(state=torch.zeros(3, device="cuda").long()),
               dict(state=torch.zeros(2).long())):
        with pytest.raises(ValueError):
            mg.muon_dropout(x, 0.1, **kw)
    with pytest.raises(ValueError):
        mg.muon_dropout(x.view(4, 4).t(), 0.1)
    with pytest.raises(TypeError):
        mg.muon_dropout(x, 0.1, state=torch.zeros(2, device="cuda"))
    with pytest.raises(TypeError):
        mg.muon_dropout(x.double(), 0.1)
