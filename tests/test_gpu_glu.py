"""The gated feed-forward block on the GPU against the fp64 oracle.

Bars.  A product over K terms accumulated in fp32 by the tensor core (which
truncates: at most 2^-23 of the running magnitude per step of 16 terms) is
within K/16 2^-23 S of the exact one, S the sum of the terms' magnitudes; S is
computed exactly here.  Each result is rounded once: half an ulp, 2^-8 (bf16) or
2^-11 (fp16) of its value at most.  In the backward pass dg and du are rounded
to the type as well, which moves a product by at most half an ulp of each of
its terms: u S; the activations and their gradients carry another 2^-20 of
their magnitudes' bound (1.2 + |g|) each.
"""
import numpy as np
import pytest

from oracle import glu_oracle as go

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 1e-37, "f16": 2.0 ** -25}
EPS = 2.0 ** -20


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


def f64(t):
    return t.detach().double().cpu().numpy()


def inputs(tokens, hidden, ffn, dtype, seed=0, off=0):
    g = torch.Generator().manual_seed(seed + 131 * tokens + 7 * hidden + ffn)

    def m(rows, cols, std):
        a = (torch.randn(rows, cols, generator=g) * std).to(DT[dtype])
        buf = torch.empty(rows * cols + off + 8, dtype=DT[dtype], device="cuda")
        v = buf[off:off + rows * cols].view(rows, cols)      # off != 0: rows off 16-byte boundaries
        v.copy_(a)
        return v
    return m(tokens, hidden, 1.0), m(ffn, hidden, hidden ** -0.5), m(ffn, hidden, hidden ** -0.5), m(tokens, ffn, 0.5)


def acc(K, S):
    return (K / 16 + 2) * 2.0 ** -23 * S


def close(got, want, err, dtype, what):
    bound = ULP[dtype] * 1.01 * np.abs(want) + TINY[dtype] + err
    d = np.abs(f64(got) - want)
    assert not (d > bound).any(), (what, int((d > bound).sum()), (d - bound).max(), want.shape)


def check_forward(mg, x, wg, wu, dtype, act="silu", save=True, stream=None):
    out = mg.muon_glu_forward(x, wg, wu, act=act, save=save, stream=stream)
    torch.cuda.synchronize()
    assert mg.muon_sync_status() == mg.MUON_OK
    X, G, U = f64(x), f64(wg), f64(wu)
    K = X.shape[1]
    h, gate, up = go.forward(X, G, U, act)
    eg, eu = acc(K, np.abs(X) @ np.abs(G).T), acc(K, np.abs(X) @ np.abs(U).T)
    eh = np.abs(up) * (1.2 * eg + EPS * np.abs(gate)) + np.abs(go.act(gate, act)) * eu + 1.2 * eg * eu
    if save:
        close(out[0], h, eh, dtype, "h")
        close(out[1], gate, eg, dtype, "gate")
        close(out[2], up, eu, dtype, "up")
    else:
        close(out, h, eh, dtype, "h")
    return out


def check_backward(mg, x, wg, wu, gate, up, dh, dtype, act="silu", **kw):
    dx, dwg, dwu = mg.muon_glu_backward(x, wg, wu, gate, up, dh, act=act, **kw)
    torch.cuda.synchronize()
    assert mg.muon_sync_status() == mg.MUON_OK
    X, Wg, Wu, G, U, D = (f64(t) for t in (x, wg, wu, gate, up, dh))
    want = go.backward(X, Wg, Wu, G, U, D, act)
    dg, du = np.abs(D * U * go.act_grad(G, act)), np.abs(D * go.act(G, act))
    u = ULP[dtype] * 1.01
    eg = u * dg + TINY[dtype] + np.abs(D * U) * EPS * (1.2 + np.abs(G))
    eu = u * du + TINY[dtype] + np.abs(D) * EPS * np.abs(G)
    T, F = D.shape
    if dx is not None:
        S = (dg + eg) @ np.abs(Wg) + (du + eu) @ np.abs(Wu)
        close(dx, want[0], eg @ np.abs(Wg) + eu @ np.abs(Wu) + acc(2 * F, S), dtype, "dx")
    close(dwg, want[1], eg.T @ np.abs(X) + acc(T, (dg + eg).T @ np.abs(X)), dtype, "dw_gate")
    close(dwu, want[2], eu.T @ np.abs(X) + acc(T, (du + eu).T @ np.abs(X)), dtype, "dw_up")
    return dx, dwg, dwu


SHAPES = [(1, 1, 1), (1, 8, 8), (2, 64, 16), (7, 33, 5), (31, 72, 40), (64, 128, 128), (65, 200, 130), (128, 64, 136),
          (129, 256, 257), (255, 1001, 300), (256, 512, 256), (257, 136, 520), (300, 513, 1031), (1000, 264, 776)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(mg, shape, dtype):
    x, wg, wu, dh = inputs(*shape, dtype)
    h, gate, up = check_forward(mg, x, wg, wu, dtype)
    assert torch.equal(check_forward(mg, x, wg, wu, dtype, save=False), h)
    check_backward(mg, x, wg, wu, gate, up, dh, dtype)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens", [1, 16, 200])
def test_activations(mg, act, tokens):
    x, wg, wu, dh = inputs(tokens, 320, 200, "f16", seed=3)
    x = x * 3
    h, gate, up = check_forward(mg, x, wg, wu, "f16", act)
    check_backward(mg, x, wg, wu, gate, up, dh, "f16", act)


@pytest.mark.parametrize("tokens", list(range(1, 20)) + [31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129])
def test_few_tokens(mg, tokens):
    """Every token count around the small kernels' limits; a row does not depend on its neighbours' count."""
    x, wg, wu, dh = inputs(tokens, 1024, 640, "bf16", seed=5)
    h = check_forward(mg, x, wg, wu, "bf16", save=False)
    h3 = check_forward(mg, x, wg, wu, "bf16")
    assert torch.equal(h3[0], h)


@pytest.mark.parametrize("off", [1, 3])
def test_matrices_off_16_byte_boundaries(mg, off):
    for shape in ((5, 64, 24), (130, 256, 264)):
        x, wg, wu, dh = inputs(*shape, "bf16", seed=9, off=off)
        h, gate, up = check_forward(mg, x, wg, wu, "bf16")
        dw = [torch.empty(shape[2] * shape[1] + off, dtype=x.dtype, device="cuda")[off:].view(shape[2], shape[1])
              for _ in range(2)]
        out = check_backward(mg, x, wg, wu, gate, up, dh, "bf16", dw_gate=dw[0], dw_up=dw[1])
        assert out[1] is dw[0] and out[2] is dw[1]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_extreme_pre_activations(mg, act, dtype):
    """Gates at the type's limits give 0 or the gate, gradients 0 or 1, never NaN."""
    big = torch.finfo(DT[dtype]).max
    gate = torch.tensor([[big, -big, 0.0, 40.0, -40.0, 1e-4, -1e-4, 1e4]], dtype=DT[dtype], device="cuda")
    ones = torch.ones_like(gate)
    eye = torch.eye(8, dtype=DT[dtype], device="cuda")
    dx, dwg, dwu = mg.muon_glu_backward(torch.ones(1, 8, dtype=DT[dtype], device="cuda"), eye, eye, gate, ones, ones * 0.5,
                                        act=act)
    G = f64(gate)[0]
    s = np.clip(G, -50, 50)
    da = 0.5 * go.act_grad(s, act)
    a = 0.5 * np.where(np.abs(G) > 50, np.maximum(G, 0), go.act(s, act))
    for got, want in ((f64(dwg)[:, 0], da), (f64(dwu)[:, 0], a)):
        assert np.all(np.abs(got - want) <= ULP[dtype] * 1.01 * np.abs(want) + 1e-7)
    assert np.all(np.isfinite(f64(dx)))


def test_a_token_with_nan_or_inf_stays_its_own_row(mg):
    for tokens in (3, 200):
        x, wg, wu, _ = inputs(tokens, 96, 72, "bf16", seed=11)
        want = mg.muon_glu_forward(x, wg, wu, save=False)
        x[1] = float("nan")
        x[2] = float("inf")
        got = mg.muon_glu_forward(x, wg, wu, save=False)
        keep = [i for i in range(tokens) if i not in (1, 2)]
        assert torch.equal(got[keep], want[keep]) and torch.isnan(got[1]).all()


def test_outputs_left_out(mg):
    x, wg, wu, dh = inputs(40, 64, 48, "bf16", seed=13)
    h, gate, up = mg.muon_glu_forward(x, wg, wu)
    full = mg.muon_glu_backward(x, wg, wu, gate, up, dh)
    part = mg.muon_glu_backward(x, wg, wu, gate, up, dh, need_dx=False)
    assert part[0] is None and torch.equal(part[1], full[1]) and torch.equal(part[2], full[2])
    dx = torch.empty_like(x)
    r = mg.lib().muon_glu_backward(*(t.data_ptr() for t in (x, wg, wu, gate, up, dh, dx)), None, None, 40, 64, 48,
                                   mg.MUON_BF16, 0, torch.cuda.current_stream().cuda_stream)
    assert r == mg.MUON_OK and torch.equal(dx, full[0])


def test_no_tokens(mg):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.randn(32, 64, device="cuda").bfloat16()
    h, gate, up = mg.muon_glu_forward(x, w, w)
    assert h.shape == (0, 32)
    dx, dwg, dwu = mg.muon_glu_backward(x, w, w, gate, up, h)
    assert not bool(dwg.any()) and not bool(dwu.any()) and dx.shape == (0, 64)


def test_repeats_and_other_stream_are_bit_equal(mg):
    x, wg, wu, dh = inputs(700, 520, 1032, "bf16", seed=17)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for stream in (None, s, None):
        h, gate, up = mg.muon_glu_forward(x, wg, wu, stream=stream)
        if stream is not None:
            stream.synchronize()
        outs.append((h, gate, up) + mg.muon_glu_backward(x, wg, wu, gate, up, dh, stream=stream))
        torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_gradient_against_differences_of_the_forward_pass(mg):
    """Directional differences of the library's own forward pass in fp16, steps of
    0.05 standard deviations.  h's rounding (2^-11 |h| at most per entry, of
    either sign) moves a sum over 6144 entries with |dh| near 1/2 by less than
    0.02, the curvature the quotient by (0.05)^2 / 6 of its third derivative,
    and the slopes are near 2: 2 % of the slope's typical size plus the slope."""
    x, wg, wu, dh = inputs(64, 128, 96, "f16", seed=19)
    h, gate, up = mg.muon_glu_forward(x, wg, wu)
    grads = mg.muon_glu_backward(x, wg, wu, gate, up, dh)
    g = torch.Generator(device="cuda").manual_seed(1)
    for k, m in enumerate((x, wg, wu)):
        d = torch.randn(m.shape, device="cuda", generator=g) * m.float().std()
        vals = []
        for sign in (1, -1):
            args = [x, wg, wu]
            args[k] = (m.float() + sign * 0.05 * d).to(m.dtype)
            moved = (args[k].float() - m.float())
            vals.append(((mg.muon_glu_forward(*args, save=False).double() * dh.double()).sum(), moved.double()))
        slope = vals[0][0] - vals[1][0]
        want = (grads[k].double() * (vals[0][1] - vals[1][1])).sum()
        scale = grads[k].double().norm() * (vals[0][1] - vals[1][1]).norm() / (m.numel() ** 0.5)
        assert abs(float(slope - want)) <= 0.02 * float(scale + want.abs())


def test_refusals_on_the_device(mg):
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(32, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(mg.MuonError) as e:
        mg.muon_glu_forward(x.float(), w.float(), w.float())
    assert e.value.status == mg.MUON_EDTYPE
    with pytest.raises(ValueError):
        mg.muon_glu_forward(x, w, w, act="relu")
    with pytest.raises(ValueError):
        mg.muon_glu_forward(x, w, w[:, :32].contiguous())
    with pytest.raises(ValueError):
        mg.muon_glu_forward(x.t(), w, w)
    with pytest.raises(TypeError):
        mg.muon_glu_forward(x, w, w.half())
    h, gate, up = mg.muon_glu_forward(x, w, w)
    with pytest.raises(ValueError):
        mg.muon_glu_backward(x, w, w, gate, up, h[:2])
