"""Edges of the experts' operators on the GPU: gates far below zero, few rows of many experts, rows that row_of
does not name, the largest sorts of one cluster."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


@pytest.mark.parametrize("act,lowest,step", [("silu", -92.0, 1.0), ("gelu_tanh", -10.1875, 0.0625)])
def test_gates_far_below_zero(mg, act, lowest, step):
    """g sigmoid(z) down to z = -92, far inside bf16's range once it is multiplied by a large value (2^40).

    Gates are exact (one product each).  The sigmoid's e^z has a relative error of |z| 2^-22 from z (GELU's: a few
    roundings of it) and (2 + 1.173 |z|) 2^-23 from the exponential, together below 4 |z| 2^-23 < 2^-14, and e^z and
    g e^z, which may be subnormal (from 1.1e-40 on, steps of 1.4e-45), 2^-17 each: below 2^-13, then the rounding
    to bf16, half a step, 2^-8."""
    gates = torch.arange(lowest, 8.0, step, dtype=torch.float64)
    rows = gates.numel()
    x = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = gates.to(x), 2.0 ** 20
    wg, wu = (torch.zeros(2, 40, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wg[:, :, 0], wu[:, :, 1] = 1.0, 2.0 ** 20
    bounds = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    h, gate, up = mg.muon_expert_glu_forward(x, wg, wu, bounds, act=act)
    assert mg.muon_sync_status() == mg.MUON_OK
    assert (gate.double().cpu() == gates[:, None]).all() and (up == 2.0 ** 40).all()
    z = gates if act == "silu" else 2 * np.sqrt(2 / np.pi) * (gates + 0.044715 * gates ** 3)
    want = (gates / (1 + torch.exp(-z)) * 2.0 ** 40)[:, None]
    assert ((h.double().cpu() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -13)).all()


@pytest.mark.parametrize("seed", [0, 1])
def test_fewer_rows_than_experts(mg, seed):
    """Experts' last k-blocks stand by their first rows then: experts of one row, of whole blocks and one more,
    beside experts without rows."""
    from tests.test_gpu_expert_products import check_glu, check_linear
    g = np.random.default_rng(seed)
    counts = np.zeros(400, dtype=int)
    for n, e in zip((1, 1, 1, 64, 65, 63, 2, 130), g.choice(400, 8, replace=False)):
        counts[e] = n
    check_glu(mg, counts.tolist(), 72, 40, "bf16", tail=3, seed=seed)
    check_linear(mg, counts.tolist(), 136, 72, "f16", tail=3, seed=seed)
    check_linear(mg, counts.tolist(), 73, 41, "bf16", seed=seed)
    check_glu(mg, [0, 0, 1, 0], 64, 64, "f16", seed=seed)


def test_scratch_of_fewer_rows_than_experts(mg):
    """The call stays within the bytes that it asked for."""
    import ctypes
    rows, experts, cols, outs = 70, 500, 72, 200
    g = torch.Generator(device="cuda").manual_seed(2)

    def r(*s):
        return torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    x, dy, w = r(rows, cols), r(rows, outs), r(experts, outs, cols)
    choice = torch.randint(0, experts, (rows, 1), generator=g, device="cuda")
    _, _, bounds = mg.muon_expert_sort(choice, experts)
    want = mg.muon_expert_linear_backward(x, w, dy, bounds)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    need, fn, s = ctypes.c_int64(0), mg.lib().muon_expert_linear_backward, torch.cuda.current_stream().cuda_stream
    args = [t.data_ptr() for t in (x, w, dy, bounds, dx, dw)] + [rows, experts, cols, outs, mg.MUON_BF16]
    assert fn(*args, None, ctypes.byref(need), s) == mg.MUON_ENOMEM
    assert need.value <= rows * 64 * (cols + outs) * 2 + 512
    guard = torch.full((need.value + 4096,), 7, dtype=torch.uint8, device="cuda")
    assert fn(*args, guard.data_ptr(), ctypes.byref(need), s) == mg.MUON_OK
    assert mg.muon_sync_status() == mg.MUON_OK
    assert (guard[need.value:] == 7).all() and torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    for e in torch.unique(choice).tolist():
        a, b = bounds[e].item(), bounds[e + 1].item()
        ref = dy[a:b].double().T @ x[a:b].double()
        size = dy[a:b].double().abs().T @ x[a:b].double().abs()
        assert ((dw[e].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * size + 1e-37).all()
    empty = torch.ones(experts, dtype=torch.bool, device="cuda")
    empty[choice.reshape(-1)] = False
    assert not dw[empty].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("hidden,off", [(64, 0), (33, 1)])
def test_rows_that_are_not_named_stay(mg, hidden, off, dtype):
    """dispatch and combine_backward write the rows that row_of names, and no byte beside them."""
    tokens, k, rows = 5, 2, 10
    row_of = torch.tensor([[0, 7], [-1, 3], [10, 4], [1 << 30, -5], [9, 2]], dtype=torch.int32, device="cuda")
    bounds = torch.tensor([0, 8], dtype=torch.int32, device="cuda")         # row 9 is behind the last expert
    g = torch.Generator(device="cuda").manual_seed(1)

    def r(n):
        return torch.randn(n * hidden + off, generator=g, device="cuda").to(dtype)[off:].view(n, hidden)
    x, ys, w = r(tokens), r(rows), torch.rand(tokens, k, generator=g, device="cuda")
    code = mg.MUON_F32 if dtype is torch.float32 else mg.MUON_BF16
    s = torch.cuda.current_stream().cuda_stream
    bufs = [torch.full((rows * hidden + off + 64,), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    xs, dys = (b[off:off + rows * hidden].view(rows, hidden) for b in bufs)
    dw = torch.full((tokens, k), 7.0, device="cuda")
    assert mg.lib().muon_expert_dispatch(x.data_ptr(), hidden, tokens, k, hidden, code, row_of.data_ptr(),
                                         bounds.data_ptr(), 1, xs.data_ptr(), s) == mg.MUON_OK
    assert mg.lib().muon_expert_combine_backward(x.data_ptr(), hidden, ys.data_ptr(), tokens, k, hidden, code,
                                                 row_of.data_ptr(), bounds.data_ptr(), 1, w.data_ptr(), dys.data_ptr(),
                                                 dw.data_ptr(), s) == mg.MUON_OK
    assert mg.muon_sync_status() == mg.MUON_OK
    for t, j, row in ((0, 0, 0), (0, 1, 7), (1, 1, 3), (2, 1, 4), (4, 1, 2)):
        assert torch.equal(xs[row], x[t]) and torch.equal(dys[row], (x[t].float() * w[t, j]).to(dtype))
    for out, buf in zip((xs, dys), bufs):
        assert not out[9].any() and (out[[1, 5, 6, 8]] == 7).all()
        assert (buf[:off] == 7).all() and (buf[off + rows * hidden:] == 7).all()
    assert not dw[row_of >= 8].any() and not dw[row_of < 0].any()


@pytest.mark.parametrize("slots,experts", [(131072, 1024), (100003, 1000), (131071, 1023), (65537, 1024)])
def test_sort_by_one_cluster_with_the_largest_tables(mg, slots, experts):
    """All sixteen CTAs of a cluster with as many experts as there can be: some empty, some slots without one, all
    slots in one expert, all in the last, none in any."""
    g = torch.Generator(device="cuda").manual_seed(slots)
    e = torch.randint(0, experts, (slots, 1), generator=g, device="cuda")
    lost = torch.rand((slots, 1), generator=g, device="cuda") < 0.1
    few = torch.randint(0, 7, (slots, 1), generator=g, device="cuda", dtype=torch.int32)
    for c in (e, torch.where(lost, torch.full_like(e, experts), e), few, torch.full_like(few, experts - 1),
              torch.zeros_like(few), torch.full_like(few, -1)):
        row_of, slot_of, bounds = mg.muon_expert_sort(c, experts)
        flat = c.reshape(-1).long()
        flat = torch.where(flat < 0, torch.full_like(flat, experts), flat)
        want = torch.argsort(flat, stable=True)
        assert torch.equal(slot_of.long(), want)
        assert torch.equal(row_of.reshape(-1)[want].long(), torch.arange(slots, device="cuda"))
        assert torch.equal(bounds.long(), torch.searchsorted(flat[want].contiguous(), torch.arange(experts + 1, device="cuda")))


def whole(shape, seed, dtype=torch.bfloat16, top=2):
    """Whole numbers, so that sums below 2^24 are exact in fp32 in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


def test_the_most_rows(mg):
    """2^24 rows, one expert with nearly all of them: results are exact whole numbers, rounded once."""
    rows, cols, outs = 1 << 24, 8, 16
    ends = [0, rows - 70100, rows - 100, rows - 100]
    bounds = torch.tensor(ends, dtype=torch.int32, device="cuda")
    x, dy, w = whole((rows, cols), 1), whole((rows, outs), 2), whole((3, outs, cols), 3)
    y = mg.muon_expert_linear_forward(x, w, bounds)
    dx, dw = mg.muon_expert_linear_backward(x, w, dy, bounds)
    assert mg.muon_sync_status() == mg.MUON_OK
    for e in range(3):
        a, b = ends[e], ends[e + 1]
        want = dy[a:b].double().T @ x[a:b].double()
        assert want.numel() == 0 or want.abs().max() < 2 ** 24
        assert torch.equal(dw[e], want.to(dw.dtype))
        for i in range(a, b, 1 << 22):
            s = slice(i, min(b, i + (1 << 22)))
            assert torch.equal(y[s], (x[s].double() @ w[e].double().T).to(y.dtype))
            assert torch.equal(dx[s], (dy[s].double() @ w[e].double()).to(dx.dtype))
    assert not y[ends[3]:].any() and not dx[ends[3]:].any()
    row_of, slot_of, bounds = mg.muon_expert_sort((x[:, 0] + 1).int().reshape(-1, 1), 4)       # -1: no expert
    xs = mg.muon_expert_dispatch(x, row_of, bounds)
    live = int(bounds[-1])
    assert torch.equal(xs[:live], x[slot_of[:live].long()]) and not xs[live:].any()
    weights = whole((rows, 1), 4, torch.float32)
    back = mg.muon_expert_combine(xs, row_of, bounds, weights=weights, residual=x)
    on = (row_of < live).float()
    assert torch.equal(back, (x.float() * (1 + on * weights)).to(x.dtype))
    dys, dweights = mg.muon_expert_combine_backward(x, xs, row_of, bounds, weights)
    assert torch.equal(dys[:live], (x.float() * weights).to(x.dtype)[slot_of[:live].long()]) and not dys[live:].any()
    assert torch.equal(dweights, (x.float() ** 2).sum(1, keepdim=True) * on)


@pytest.mark.parametrize("cols", [40000, 40001])
def test_experts_matrices_beyond_31_bits(mg, cols):
    """Weights of more than 2^31 elements, on 16 bytes and off: the last expert's results."""
    outs, experts, rows = 20001, 3, 70
    w = whole((experts, outs, cols), 1, top=1)
    assert w.numel() > 1 << 31
    x, dy = whole((rows, cols), 2, top=1), whole((rows, outs), 3, top=1)
    ends = [0, 1, 3, rows]
    bounds = torch.tensor(ends, dtype=torch.int32, device="cuda")
    y = mg.muon_expert_linear_forward(x, w, bounds)
    dx, dw = mg.muon_expert_linear_backward(x, w, dy, bounds)
    assert mg.muon_sync_status() == mg.MUON_OK
    for e in range(experts):
        a, b = ends[e], ends[e + 1]
        assert torch.equal(dw[e], (dy[a:b].float().T @ x[a:b].float()).to(dw.dtype))
        for i in range(0, outs, 4000):
            s = slice(i, min(outs, i + 4000))
            assert torch.equal(y[a:b, s], (x[a:b].double() @ w[e, s].double().T).to(y.dtype))
        for i in range(0, cols, 4000):
            s = slice(i, min(cols, i + 4000))
            assert torch.equal(dx[a:b, s], (dy[a:b].double() @ w[e, :, s].double()).to(dx.dtype))
