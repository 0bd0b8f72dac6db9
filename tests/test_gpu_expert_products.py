"""The experts' products on the GPU against the fp64 oracle, expert by expert.

Bars, as for the dense block.  A product over K terms accumulated in fp32 by the
tensor core (which truncates: at most 2^-23 of the running magnitude per step of
16 terms, 65536 terms of a part at most, then one addition per part) is within
(K/16 + 2) 2^-23 S of the exact one, S the sum of the terms' magnitudes; S is
computed exactly here.  Each result is rounded once: half an ulp of its value.
In the gated backward pass dg and du are rounded to the type as well, which
moves a product by at most half an ulp of each of its terms; the activations and
their gradients carry another 2^-20 of their magnitudes' bound (1.2 + |g|) each.
"""
import numpy as np
import pytest

from oracle import expert_oracle as eo
from oracle import glu_oracle as go

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 1e-37, "f16": 2.0 ** -25}
EPS = 2.0 ** -20
NAN = float("nan")


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def m(shape, std, dtype, seed, off=0):
    n = int(np.prod(shape))
    buf = torch.zeros(n + off + 8, dtype=DT[dtype], device="cuda")
    v = buf[off:off + n].view(shape)                # off != 0: rows off 16-byte boundaries
    v.copy_(torch.randn(shape, generator=gen(seed), device="cuda") * std)
    return v


def ends(counts, tail=0):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda"), int(sum(counts)) + tail


def acc(K, S):
    return (min(K, 65536) / 16 + K / 65536 + 2) * 2.0 ** -23 * S


def close(got, want, err, dtype, what):
    bound = ULP[dtype] * 1.01 * np.abs(want) + TINY[dtype] + err
    d = np.abs(f64(got) - want)
    bad = ~(d <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.nanmax(d - bound), want.shape)


def check_glu(mg, counts, hidden, ffn, dtype, act="silu", tail=0, off=0, bounds=None, rows=None, seed=0):
    """Forward and backward; rows behind the last expert hold NaN in every input."""
    if bounds is None:
        bounds, rows = ends(counts, tail)
    E, B = bounds.numel() - 1, bounds.tolist()
    live = np.zeros(rows, dtype=bool)
    for a, b in eo.segments(B, rows):
        live[a:b] = True
    dead = torch.from_numpy(~live).cuda()
    x, dh = m((rows, hidden), 1.0, dtype, seed + 1, off), m((rows, ffn), 0.5, dtype, seed + 4, off)
    wg, wu = (m((E, ffn, hidden), hidden ** -0.5, dtype, seed + k, off) for k in (2, 3))
    X, D, G, U = f64(x), f64(dh), f64(wg), f64(wu)
    x[dead], dh[dead] = NAN, NAN
    out = mg.muon_expert_glu_forward(x, wg, wu, bounds, act=act)
    alone = mg.muon_expert_glu_forward(x, wg, wu, bounds, act=act, save=False)
    assert mg.muon_sync_status() == mg.MUON_OK and torch.equal(out[0], alone)
    h, gate, up = eo.glu_forward(X, G, U, B, act)
    size = [eo.linear_forward(np.abs(X), np.abs(W), B) for W in (G, U)]
    eg, eu = acc(hidden, size[0]), acc(hidden, size[1])
    close(out[1], gate, eg, dtype, "gate")
    close(out[2], up, eu, dtype, "up")
    eh = np.abs(up) * (1.2 * eg + EPS * np.abs(gate)) + np.abs(go.act(gate, act)) * eu + 1.2 * eg * eu
    close(out[0], h, np.where(live[:, None], eh, 0), dtype, "h")
    gate, up = out[1].clone(), out[2].clone()
    Gt, Up = f64(gate), f64(up)
    gate[dead], up[dead] = NAN, NAN
    dx, dwg, dwu = mg.muon_expert_glu_backward(x, wg, wu, gate, up, dh, bounds, act=act)
    assert mg.muon_sync_status() == mg.MUON_OK
    want = eo.glu_backward(X, G, U, Gt, Up, D, B, act)
    dg, du = np.abs(D * Up * go.act_grad(Gt, act)), np.abs(D * go.act(Gt, act))
    u = ULP[dtype] * 1.01
    e1 = u * dg + TINY[dtype] + np.abs(D * Up) * EPS * (1.2 + np.abs(Gt))
    e2 = u * du + TINY[dtype] + np.abs(D) * EPS * np.abs(Gt)
    ex = np.zeros(X.shape)
    ew = [np.zeros(G.shape), np.zeros(U.shape)]
    for e, (a, b) in enumerate(eo.segments(B, rows)):
        ex[a:b] = e1[a:b] @ np.abs(G[e]) + e2[a:b] @ np.abs(U[e])
        ex[a:b] += acc(2 * ffn, (dg + e1)[a:b] @ np.abs(G[e]) + (du + e2)[a:b] @ np.abs(U[e]))
        for w, d, err in ((ew[0], dg, e1), (ew[1], du, e2)):
            w[e] = err[a:b].T @ np.abs(X[a:b]) + acc(b - a, (d + err)[a:b].T @ np.abs(X[a:b]))
    close(dx, want[0], ex, dtype, "dx")
    close(dwg, want[1], ew[0], dtype, "dw_gate")
    close(dwu, want[2], ew[1], dtype, "dw_up")
    assert not out[0][dead].any() and not dx[dead].any()
    return (x, wg, wu, gate, up, dh, bounds), (dx, dwg, dwu)


def check_linear(mg, counts, cols, outs, dtype, tail=0, off=0, seed=0):
    bounds, rows = ends(counts, tail)
    E, B = len(counts), bounds.tolist()
    x, dy = m((rows, cols), 1.0, dtype, seed + 1, off), m((rows, outs), 0.5, dtype, seed + 2, off)
    w = m((E, outs, cols), cols ** -0.5, dtype, seed + 3, off)
    X, D, W = f64(x), f64(dy), f64(w)
    x[B[-1]:], dy[B[-1]:] = NAN, NAN
    y = mg.muon_expert_linear_forward(x, w, bounds)
    close(y, eo.linear_forward(X, W, B), acc(cols, eo.linear_forward(np.abs(X), np.abs(W), B)), dtype, "y")
    dx, dw = mg.muon_expert_linear_backward(x, w, dy, bounds)
    assert mg.muon_sync_status() == mg.MUON_OK
    want, size = eo.linear_backward(X, W, D, B), eo.linear_backward(np.abs(X), np.abs(W), np.abs(D), B)
    close(dx, want[0], acc(outs, size[0]), dtype, "dx")
    k = np.array([b - a for a, b in eo.segments(B, rows)])[:, None, None]
    close(dw, want[1], (np.minimum(k, 65536) / 16 + k / 65536 + 2) * 2.0 ** -23 * size[1], dtype, "dw")
    return (x, w, dy, bounds), (y, dx, dw)


COUNTS = [[1], [5], [0], [3, 0, 2], [0, 0, 7, 0], [64, 64], [63, 65, 1], [128, 0, 256], [255, 257, 1, 300],
          [300, 31, 33, 0, 129, 700], [1] * 40, [0] * 30 + [9]]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_counts(mg, counts, dtype):
    check_glu(mg, counts, 136, 200, dtype, tail=3)
    check_linear(mg, counts, 200, 136, dtype, tail=3)


@pytest.mark.parametrize("hidden,ffn", [(1, 1), (8, 8), (7, 5), (64, 16), (33, 129), (72, 40), (256, 256), (257, 120),
                                        (512, 264), (1001, 303)])
def test_sizes(mg, hidden, ffn):
    for dtype in ("bf16", "f16"):
        check_glu(mg, [70, 0, 200, 13], hidden, ffn, dtype)
        check_linear(mg, [70, 0, 200, 13], ffn, hidden, dtype)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_activations(mg, act):
    check_glu(mg, [40, 100, 3], 320, 200, "f16", act, tail=5)


@pytest.mark.parametrize("off", [1, 4])
def test_off_16_byte_boundaries(mg, off):
    check_glu(mg, [40, 100, 3], 64, 136, "bf16", tail=5, off=off)
    check_linear(mg, [40, 100, 3], 64, 136, "bf16", tail=5, off=off)


def test_many_experts(mg):
    g = np.random.default_rng(3)
    check_glu(mg, g.integers(0, 4, 1024).tolist(), 24, 40, "bf16", tail=100)
    check_glu(mg, [0] * 1023 + [77], 24, 40, "f16")
    check_linear(mg, g.integers(0, 90, 257).tolist(), 72, 24, "bf16", tail=1)


def test_only_rows_behind_the_last_expert(mg):
    check_glu(mg, [0, 0, 0], 72, 40, "bf16", tail=600)
    check_linear(mg, [0, 0, 0], 72, 300, "bf16", tail=600)


def test_more_tiles_than_clusters(mg):
    check_linear(mg, [1000, 3, 2100, 0, 700], 1032, 2056, "bf16", tail=300)


@pytest.mark.parametrize("B", [[5, 40, 90, 100], [0, 40, 90, 5000], [0, -3, 40, 100], [0, 50, 20, 100], [0, 50, 50, -7]],
                         ids=str)
def test_bounds_no_sort_wrote(mg, B):
    """Offsets are clamped to the matrix; an expert whose end is before its start has no rows."""
    bounds, rows = torch.tensor(B, dtype=torch.int32, device="cuda"), 120
    x, wg, wu = m((rows, 64), 1.0, "bf16", 1), m((3, 72, 64), 0.1, "bf16", 2), m((3, 72, 64), 0.1, "bf16", 3)
    h = mg.muon_expert_glu_forward(x, wg, wu, bounds, save=False)
    dx, dw = mg.muon_expert_linear_backward(x, wg, h, bounds)
    assert mg.muon_sync_status() == mg.MUON_OK
    seen = np.zeros(rows, dtype=int)
    for e, (a, b) in enumerate(eo.segments(B, rows)):
        seen[a:b] += 1
        want = (h[a:b].double().T @ x[a:b].double())
        assert torch.allclose(dw[e].double(), want, rtol=2.0 ** -7, atol=1e-2)
    for e, (a, b) in enumerate(eo.segments(B, rows)):
        once = torch.from_numpy(np.flatnonzero(seen[a:b] == 1) + a).cuda()
        want = torch.nn.functional.silu(x[once].double() @ wg[e].double().T) * (x[once].double() @ wu[e].double().T)
        assert torch.allclose(h[once].double(), want, rtol=2.0 ** -7, atol=1e-2)


def test_an_experts_rows_stay_its_own(mg):
    """Infinities and NaN among one expert's rows change nothing of the others', whose rows share its tiles and
    k-blocks."""
    counts = [70, 59, 1, 130]
    args, want = check_glu(mg, counts, 136, 200, "bf16", tail=9)
    x, wg, wu, gate, up, dh, bounds = args
    wd = m((4, 136, 200), 0.1, "bf16", 9)
    lin = mg.muon_expert_linear_backward(gate, wd, x, bounds)
    y = mg.muon_expert_linear_forward(gate, wd, bounds)
    h = mg.muon_expert_glu_forward(x, wg, wu, bounds, save=False)
    for e in range(4):
        a, b = bounds[e].item(), bounds[e + 1].item()
        bad = [t.clone() for t in (x, gate, up, dh)]
        for t in bad:
            t[a:b:2], t[a + 1:b:2] = float("inf"), NAN
        others = [i for i in range(4) if i != e]
        keep = torch.ones(x.shape[0], dtype=torch.bool, device="cuda")
        keep[a:b] = False
        got = mg.muon_expert_glu_backward(bad[0], wg, wu, bad[1], bad[2], bad[3], bounds)
        assert torch.equal(got[0][keep], want[0][keep])
        assert all(torch.equal(got[k][others], want[k][others]) for k in (1, 2))
        got = mg.muon_expert_linear_backward(bad[1], wd, bad[0], bounds)
        assert torch.equal(got[0][keep], lin[0][keep]) and torch.equal(got[1][others], lin[1][others])
        assert torch.equal(mg.muon_expert_linear_forward(bad[1], wd, bounds)[keep], y[keep])
        assert torch.equal(mg.muon_expert_glu_forward(bad[0], wg, wu, bounds, save=False)[keep], h[keep])


def test_given_and_missing_outputs(mg):
    args, (dx, dwg, dwu) = check_glu(mg, [40, 0, 100], 72, 136, "bf16")
    bufs = [torch.full_like(dwg, NAN) for _ in range(2)]
    out = mg.muon_expert_glu_backward(*args, dw_gate=bufs[0], dw_up=bufs[1], need_dx=False)
    assert out[0] is None and out[1] is bufs[0] and out[2] is bufs[1]
    assert torch.equal(bufs[0], dwg) and torch.equal(bufs[1], dwu)
    largs, (y, dx, dw) = check_linear(mg, [40, 0, 100], 72, 136, "bf16")
    buf = torch.full_like(dw, NAN)
    version = buf._version
    got = mg.muon_expert_linear_backward(*largs, need_dx=False, dw=buf)
    assert got[0] is None and got[1] is buf and torch.equal(buf, dw) and buf._version > version


def test_no_rows(mg):
    bounds = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, w, wd = m((0, 64), 1.0, "bf16", 1), m((2, 40, 64), 1.0, "bf16", 2), m((2, 64, 40), 1.0, "bf16", 3)
    h, gate, up = mg.muon_expert_glu_forward(x, w, w, bounds)
    assert h.shape == (0, 40)
    dx, dwg, dwu = mg.muon_expert_glu_backward(x, w, w, gate, up, h, bounds)
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()
    assert mg.muon_expert_linear_forward(h, wd, bounds).shape == (0, 64)
    assert not mg.muon_expert_linear_backward(h, wd, x, bounds)[1].any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weight_gradients_over_many_rows(mg, dtype):
    """Sums of one sign over more than 65536 rows of an expert, in parts (one ragged, one of whole k-blocks): each at
    most 2^-23 of the sum short per 16 terms, then one rounding."""
    counts, hidden, ffn = [131072 + 77, 5, 65536 + 64], 72, 40
    bounds, rows = ends(counts, tail=7)

    def positive(cols, seed):
        return (0.5 + 0.5 * torch.rand((rows, cols), generator=gen(seed), device="cuda")).to(DT[dtype])

    x, dy = positive(hidden, 1), positive(ffn, 2) * 2.0 ** -9
    w = torch.zeros((3, ffn, hidden), dtype=x.dtype, device="cuda")
    dx, dw = mg.muon_expert_linear_backward(x, w, dy, bounds)
    assert not dx.any()
    for e, (a, b) in enumerate(eo.segments(bounds.tolist(), rows)):
        want = dy[a:b].double().T @ x[a:b].double()
        err = (dw[e].double() / want - 1).abs().max().item()
        assert err <= 4096 * 2.0 ** -23 + ULP[dtype] + 2.0 ** -20, (e, err)


@pytest.mark.parametrize("K", [65536, 65536 + 64, 140001])
def test_long_contractions(mg, K):
    """Sums of one sign over more than 65536 columns: linear forward and dx, gated forward; dx of the gated block
    crosses from dG Wg to dU Wu."""
    counts, n = [3, 130], 40
    bounds, rows = ends(counts, tail=2)

    def positive(shape, seed, scale=1.0):
        return ((0.5 + 0.5 * torch.rand(shape, generator=gen(seed), device="cuda")) * scale).half()

    x, w = positive((rows, K), 1), positive((2, n, K), 2, 2.0 ** -9)
    bar = 4096 * 2.0 ** -23 + 2.0 ** -11 + 2.0 ** -20
    y = mg.muon_expert_linear_forward(x, w, bounds)
    wt = w.transpose(1, 2).contiguous()
    dx, _ = mg.muon_expert_linear_backward(torch.zeros((rows, n), dtype=x.dtype, device="cuda"), wt, x, bounds)
    h, gate, up = mg.muon_expert_glu_forward(x, w, w, bounds)
    # gate = 32: silu(32) = 32, silu'(32) = 1; dg = x / 2, du = 32 x / 64
    c = torch.full_like(x, 32.0)
    dxg, _, _ = mg.muon_expert_glu_backward(torch.zeros((rows, n), dtype=x.dtype, device="cuda"), wt, wt, c,
                                            torch.full_like(x, 32.0), x * 2.0 ** -6, bounds)
    assert mg.muon_sync_status() == mg.MUON_OK
    for e, (a, b) in enumerate(eo.segments(bounds.tolist(), rows)):
        want = x[a:b].double() @ w[e].double().T
        for got, ref in ((y, want), (dx, want), (gate, want), (up, want), (dxg, want)):
            assert ((got[a:b].double() / ref - 1).abs() <= bar).all()


def test_repeats_give_the_same_bytes(mg):
    args, want = check_glu(mg, [300, 31, 0, 129, 700], 512, 264, "bf16")
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(mg.muon_expert_glu_backward(*args), want))


def test_binding_refusals(mg):
    x, w, wd = m((6, 64), 1.0, "bf16", 1), m((2, 40, 64), 1.0, "bf16", 2), m((2, 64, 40), 1.0, "bf16", 3)
    bounds = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    h, gate, up = mg.muon_expert_glu_forward(x, w, w, bounds)
    for call in (lambda: mg.muon_expert_glu_forward(x, w, w[:1], bounds),
                 lambda: mg.muon_expert_glu_forward(x, w[0], w[0], bounds),
                 lambda: mg.muon_expert_glu_forward(x, wd, wd, bounds),
                 lambda: mg.muon_expert_glu_forward(x, w, w, bounds[:2]),
                 lambda: mg.muon_expert_glu_forward(x, w, w, bounds, act="relu"),
                 lambda: mg.muon_expert_glu_forward(x.t(), w, w, bounds),
                 lambda: mg.muon_expert_glu_backward(x, w, w, gate, up, x, bounds),
                 lambda: mg.muon_expert_glu_backward(x, w, w, gate, up, h, bounds, dw_up=wd),
                 lambda: mg.muon_expert_linear_forward(x, wd, bounds),
                 lambda: mg.muon_expert_linear_backward(h, wd, h, bounds),
                 lambda: mg.muon_expert_linear_backward(h, wd, x, bounds, dw=w),
                 lambda: mg.muon_expert_linear_forward(h, wd, bounds.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mg.muon_expert_glu_forward(x.half(), w, w, bounds),
                 lambda: mg.muon_expert_glu_forward(x, w, w, bounds.long()),
                 lambda: mg.muon_expert_linear_backward(h, wd, x.half(), bounds)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(mg.MuonError):
        mg.muon_expert_linear_forward(h.float(), wd.float(), bounds)


def test_scratch(mg):
    """The C call says what it needs, refuses less, and runs with exactly that."""
    import ctypes
    x, w = m((6, 63), 1.0, "bf16", 1), m((2, 40, 63), 1.0, "bf16", 2)
    bounds = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    y = torch.empty((6, 40), dtype=x.dtype, device="cuda")
    need = ctypes.c_int64(0)

    def call(p):
        return mg.lib().muon_expert_linear_forward(x.data_ptr(), w.data_ptr(), bounds.data_ptr(), y.data_ptr(), 6, 2, 63,
                                                   40, mg.MUON_BF16, p, ctypes.byref(need),
                                                   torch.cuda.current_stream().cuda_stream)
    assert call(None) == mg.MUON_ENOMEM
    n = need.value
    assert n >= (6 + 80) * 64 * 2
    guard = torch.full((n + 512,), 7, dtype=torch.uint8, device="cuda")
    need.value = n - 1
    assert call(guard.data_ptr()) == mg.MUON_ENOMEM and need.value == n
    assert call(guard.data_ptr() + 16) == mg.MUON_EINVAL
    assert call(guard.data_ptr()) == mg.MUON_OK
    torch.cuda.synchronize()
    assert (guard[n:] == 7).all()
    assert torch.equal(y, mg.muon_expert_linear_forward(x, w, bounds))


def test_input_gradients_alone(mg):
    """Through the C ABI the weights' gradients may be left out too."""
    import ctypes
    args, (dx, _, _) = check_glu(mg, [40, 0, 100], 72, 136, "bf16", tail=4)
    x, wg, wu, gate, up, dh, bounds = args
    largs, (_, dlx, _) = check_linear(mg, [40, 0, 100], 72, 136, "bf16", tail=4)
    lx, lw, ldy, lbounds = largs
    s = torch.cuda.current_stream().cuda_stream

    def call(name, *a):
        need = ctypes.c_int64(0)
        fn = getattr(mg.lib(), name)
        st = fn(*a, None, ctypes.byref(need), s)
        if st == mg.MUON_ENOMEM:
            scratch = torch.empty(need.value, dtype=torch.uint8, device="cuda")
            st = fn(*a, scratch.data_ptr(), ctypes.byref(need), s)
        assert st == mg.MUON_OK
        torch.cuda.synchronize()
    got = torch.full_like(dx, NAN)
    call("muon_expert_glu_backward", *[t.data_ptr() for t in (x, wg, wu, gate, up, dh, bounds)], got.data_ptr(), None, None,
         144, 3, 72, 136, mg.MUON_BF16, 0)
    assert torch.equal(got, dx)
    got = torch.full_like(dlx, NAN)
    call("muon_expert_linear_backward", *[t.data_ptr() for t in (lx, lw, ldy, lbounds)], got.data_ptr(), None, 144, 3, 72, 136,
         mg.MUON_BF16)
    assert torch.equal(got, dlx)


def test_wide_and_narrow_experts(mg):
    """Column counts around whole blocks of 64 and tiles of 256, where operands are copied in one piece or two."""
    for hidden, ffn in ((64, 320), (320, 64), (448, 128), (127, 192), (192, 65)):
        check_glu(mg, [33, 64, 0, 200], hidden, ffn, "bf16", tail=1)
        check_linear(mg, [33, 64, 0, 200], hidden, ffn, "f16", tail=1)


def test_gradients_alone_of_odd_sizes(mg):
    """Operands of the products that are not asked for are not copied; the others' results stay as they are."""
    import ctypes
    args, (dx, dwg, dwu) = check_glu(mg, [40, 0, 100], 73, 135, "f16", tail=4)
    largs, (_, dlx, dw) = check_linear(mg, [40, 0, 100], 73, 135, "f16", tail=4)
    none, *got = mg.muon_expert_glu_backward(*args, need_dx=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(got, (dwg, dwu)))
    none, got = mg.muon_expert_linear_backward(*largs, need_dx=False)
    assert none is None and torch.equal(got, dw)
    for name, ins, want, rest in (("muon_expert_glu_backward", args, dx, (None, None, 144, 3, 73, 135, mg.MUON_F16, 0)),
                                  ("muon_expert_linear_backward", largs, dlx, (None, 144, 3, 73, 135, mg.MUON_F16))):
        got, need, s = torch.full_like(want, NAN), ctypes.c_int64(0), torch.cuda.current_stream().cuda_stream
        call = [t.data_ptr() for t in ins] + [got.data_ptr(), *rest]
        assert getattr(mg.lib(), name)(*call, None, ctypes.byref(need), s) == mg.MUON_ENOMEM
        scratch = torch.empty(need.value, dtype=torch.uint8, device="cuda")
        assert getattr(mg.lib(), name)(*call, scratch.data_ptr(), ctypes.byref(need), s) == mg.MUON_OK
        torch.cuda.synchronize()
        assert torch.equal(got, want)
