"""The gated feed-forward block at the ends of the number range and of its sizes."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
INF = float("inf")


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dtype])


@pytest.mark.parametrize("ffn", [128, 77])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_gate_beyond_the_range(mg, dtype, act, ffn):
    """A gate that its rounding made infinite has the activation's limits: 0 and slope 0 below, the gate itself and
    slope 1 above, as at the type's largest numbers.  A NaN stays one."""
    x, dh, up = rand((40, 64), dtype, 1), rand((40, ffn), dtype, 2), rand((40, ffn), dtype, 3)
    wg, wu = rand((ffn, 64), dtype, 4, 0.125), rand((ffn, 64), dtype, 5, 0.125)
    gate = rand((40, ffn), dtype, 6)
    big = torch.finfo(DT[dtype]).max

    def back(value, columns):
        g = gate.clone()
        g[7:9, columns] = value
        return mg.muon_glu_backward(x, wg, wu, g, up, dh, act=act)

    low = back(-INF, slice(3, 6))
    for got, want in zip(low, back(-big, slice(3, 6))):
        assert torch.equal(got, want) and torch.isfinite(got).all()
    high = back(INF, slice(3, 6))[1]
    assert torch.equal(high, back(big, slice(3, 6))[1]) and torch.isfinite(high).all()
    nan = back(float("nan"), slice(3, 6))[1]
    assert torch.isnan(nan[3:6]).all() and torch.isfinite(nan[:3]).all() and torch.isfinite(nan[6:]).all()


def test_a_gate_beyond_the_range_from_the_forward_pass(mg):
    """fp16 products at -70000 round to -inf in the saved gate; h is 0 there, and so is what flows back."""
    x = torch.full((3, 8), 100.0, dtype=torch.float16, device="cuda")
    x[1:] = 0.5
    wg = torch.full((16, 8), -87.5, dtype=torch.float16, device="cuda")
    wu = torch.full((16, 8), 0.25, dtype=torch.float16, device="cuda")
    h, gate, up = mg.muon_glu_forward(x, wg, wu)
    assert (gate[0] == -INF).all() and not h[0].any()
    dx, dwg, dwu = mg.muon_glu_backward(x, wg, wu, gate, up, torch.ones_like(h))
    assert not dx[0].any() and all(torch.isfinite(t).all() for t in (dx, dwg, dwu))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,hidden,ffn", [(65600, 72, 40), (300001, 264, 136), (1 << 18, 33, 300)])
def test_weight_gradients_over_many_tokens(mg, dtype, tokens, hidden, ffn):
    """Sums of one sign, the worst case of an accumulator that truncates: 65536 terms of it at most, 2^-23 of the
    sum per 16 terms, then one rounding.  gate = 32 and powers of two keep dg and du exact: silu(32) = 32 and
    silu'(32) = 1 in fp32.  Columns of several sizes spread the results over a power of two, so that the mean of the
    errors shows what truncation takes from all of them: the roundings leave it 2^-12 (five deviations of bf16's,
    2^-8 / sqrt(3 n), over the smallest n of 2880 entries)."""
    g = torch.Generator(device="cuda").manual_seed(tokens)

    def positive(cols):
        size = torch.rand((1, cols), generator=g, device="cuda") * 0.5 + 0.5
        return (size * (torch.rand((tokens, cols), generator=g, device="cuda") * 0.5 + 0.5)).to(DT[dtype])

    x, dh = positive(hidden), positive(ffn) * 2.0 ** -13
    gate, up = torch.full_like(dh, 32.0), torch.full_like(dh, 16.0)
    w = torch.zeros(ffn, hidden, dtype=x.dtype, device="cuda")
    dx, dwg, dwu = mg.muon_glu_backward(x, w, w, gate, up, dh)
    assert not dx.any()
    ref = sum(dh[k:k + 32768].double().T @ x[k:k + 32768].double() for k in range(0, tokens, 32768))
    short = 4096 * 2.0 ** -23
    for got, want in ((dwg, 16 * ref), (dwu, 32 * ref)):
        err = got.double() / want - 1
        assert err.abs().max().item() <= short + {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype] + 2.0 ** -20
        assert abs(err.mean().item()) <= short + 2.0 ** -12


def test_input_gradient_over_a_wide_block(mg):
    """2 ffn beyond 65536 terms: dX in parts, ragged and crossing from dG Wg to dU Wu.  Per part of at most 1024
    k-blocks 2^-11 of the magnitudes' sum at worst; over random signs the running sum is far below it."""
    tokens, hidden, ffn = 300, 200, 40001
    x, dh = rand((tokens, hidden), "f16", 1), rand((tokens, ffn), "f16", 2)
    wg, wu = rand((ffn, hidden), "f16", 3, 0.01), rand((ffn, hidden), "f16", 4, 0.01)
    gate, up = torch.full_like(dh, 32.0), torch.full_like(dh, 0.5)
    dx, dwg, dwu = mg.muon_glu_backward(x, wg, wu, gate, up, dh)
    want = (dh.double() * 0.5) @ wg.double() + (dh.double() * 32) @ wu.double()
    size = (dh.double().abs() * 0.5) @ wg.double().abs() + (dh.double().abs() * 32) @ wu.double().abs()
    assert ((dx.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -11 * size).all()
    for got, ref in ((dwg, (dh.double() * 0.5).T @ x.double()), (dwu, (dh.double() * 32).T @ x.double())):
        assert ((got.double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -14 * ref.abs().max()).all()
