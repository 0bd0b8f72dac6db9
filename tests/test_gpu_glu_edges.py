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
