"""The experts' operators and dropout together, as a block uses them: its results and gradients against fp64 autograd of
the formulas, in graphs, on streams and threads, beside autograd, and in the example's training loop."""
import importlib.util
import os
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(*shape, seed=0, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(dtype)


def problem(tokens, k, experts, hidden, ffn, seed=0, dtype=torch.bfloat16, dropped=0.0):
    choice = torch.topk(torch.rand((tokens, experts), generator=gen(seed), device="cuda"), k, dim=1).indices
    lost = torch.rand((tokens, k), generator=gen(seed + 1), device="cuda") < dropped
    return dict(x=rand(tokens, hidden, seed=seed + 2, dtype=dtype), choice=torch.where(lost, -1, choice),
                weights=torch.rand((tokens, k), generator=gen(seed + 3), device="cuda"),
                wg=rand(experts, ffn, hidden, seed=seed + 4, std=hidden ** -0.5, dtype=dtype),
                wu=rand(experts, ffn, hidden, seed=seed + 5, std=hidden ** -0.5, dtype=dtype),
                wd=rand(experts, hidden, ffn, seed=seed + 6, std=ffn ** -0.5, dtype=dtype),
                dy=rand(tokens, hidden, seed=seed + 7, dtype=dtype), state=torch.tensor([seed + 40, 3], device="cuda"))


def block(mg, p, stream=None, p_drop=0.2):
    """Forward and backward of one block: x + dropout(experts(x)), and everything's gradient."""
    s, E = dict(stream=stream), p["wg"].shape[0]
    row_of, slot_of, bounds = mg.muon_expert_sort(p["choice"], E, **s)
    xs = mg.muon_expert_dispatch(p["x"], row_of, bounds, **s)
    h, gate, up = mg.muon_expert_glu_forward(xs, p["wg"], p["wu"], bounds, **s)
    ys = mg.muon_expert_linear_forward(h, p["wd"], bounds, **s)
    y = mg.muon_expert_combine(ys, row_of, bounds, weights=p["weights"], **s)
    out = mg.muon_dropout(y, p_drop, state=p["state"], residual=p["x"], **s)
    dyd = mg.muon_dropout(p["dy"], p_drop, state=p["state"], **s)
    dys, dweights = mg.muon_expert_combine_backward(dyd, ys, row_of, bounds, p["weights"], **s)
    dh, dwd = mg.muon_expert_linear_backward(h, p["wd"], dys, bounds, **s)
    dxs, dwg, dwu = mg.muon_expert_glu_backward(xs, p["wg"], p["wu"], gate, up, dh, bounds, **s)
    dx = mg.muon_expert_combine(dxs, row_of, bounds, residual=p["dy"], **s)
    return out, dx, dweights, dwg, dwu, dwd, row_of, slot_of, bounds


def plain(mg, p, p_drop=0.2):
    """The same from the definition, in fp64 under autograd; the mask from ones."""
    x, w, wg, wu, wd = (p[n].double().requires_grad_() for n in ("x", "weights", "wg", "wu", "wd"))
    keep = mg.muon_dropout(torch.ones_like(p["x"], dtype=torch.float32), p_drop, state=p["state"]).double()
    y = torch.zeros_like(x)
    for e in range(wg.shape[0]):
        t, j = torch.nonzero(p["choice"] == e, as_tuple=True)
        v = torch.nn.functional.silu(x[t] @ wg[e].t()) * (x[t] @ wu[e].t())
        y = y.index_add(0, t, w[t, j][:, None] * (v @ wd[e].t()))
    out = x + keep * y
    grads = torch.autograd.grad(out, (x, w, wg, wu, wd), p["dy"].double())
    return out.detach(), *grads


def check(mg, p, got=None):
    """Relative 2-norms.  Between the inputs and any result stand at most ten roundings to the type, of half an ulp
    (rms 1/sqrt(3) of that) each and independent of another: 2 sqrt(10 / 3) half ulps, with a factor of two for
    their way through the products."""
    half = torch.finfo(p["x"].dtype).eps / 2
    got = block(mg, p) if got is None else got
    for a, b, name in zip(got, plain(mg, p), ("out", "dx", "dweights", "dw_gate", "dw_up", "dw_down")):
        assert a.shape == b.shape
        err = ((a.double() - b).norm() / b.norm()).item()
        assert err <= 2 * (10 / 3) ** 0.5 * half, (name, err)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(200, 2, 5, 256, 136), (1, 2, 8, 64, 64), (513, 3, 7, 129, 75), (1000, 8, 64, 128, 64),
                                   (300, 1, 1, 72, 200)], ids=str)
def test_block(mg, shape, dtype):
    check(mg, problem(*shape, dtype=dtype))
    check(mg, problem(*shape, seed=50, dtype=dtype, dropped=0.2 if shape[0] > 1 else 0.0))
    assert mg.muon_sync_status() == mg.MUON_OK


def copy_into(dst, src):
    for n in dst:
        dst[n].copy_(src[n])


def test_in_a_graph(mg):
    """Replays follow new inputs, choices (so new bounds), weights and generator states, with nothing on the host."""
    p = problem(300, 3, 9, 200, 137, dropped=0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block(mg, p)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = block(mg, p)
        for seed in (100, 200, 300):
            copy_into(p, problem(300, 3, 9, 200, 137, seed=seed, dropped=0.3))
            graph.replay()
            for a, b in zip([t.clone() for t in out], block(mg, p)):
                assert torch.equal(a, b)
    s.synchronize()
    assert mg.muon_sync_status() == mg.MUON_OK


def test_two_graphs_at_once(mg):
    """Graphs captured on one stream share no scratch: replayed on two streams at the same time they give what each
    gives alone."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ps = [problem(700, 2, 6, 257, 300, seed=k) for k in (1, 2)]     # odd rows: padded copies in the scratch
    graphs, outs, want = [], [], []
    with torch.cuda.stream(s):
        for p in ps:
            want.append([t.clone() for t in block(mg, p)])
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(block(mg, p))
            graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, t in zip(graphs, streams):
            with torch.cuda.stream(t):
                g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_threads_on_separate_streams(mg):
    ps = [problem(*shape, seed=i) for i, shape in enumerate([(300, 2, 5, 256, 136), (64, 3, 7, 129, 75), (900, 4, 16, 128, 64),
                                                              (9, 2, 4, 64, 333)])]
    want = [block(mg, p) for p in ps]
    torch.cuda.synchronize()
    streams, got, errors = [torch.cuda.Stream() for _ in ps], [None] * len(ps), []
    start = threading.Barrier(len(ps))

    def run(i):
        try:
            start.wait(timeout=60)
            got[i] = [block(mg, ps[i], stream=streams[i]) for _ in range(4)]
            streams[i].synchronize()
        except Exception as e:          # noqa: BLE001 - reported on the main thread
            errors.append((i, repr(e)))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(ps))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    assert not any(t.is_alive() for t in threads) and not errors, errors
    torch.cuda.synchronize()
    for rounds, ref in zip(got, want):
        for outs in rounds:
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    assert mg.muon_sync_status() == mg.MUON_OK


def test_beside_autograd(mg):
    """Results carry no graph; a tensor written in place is noticed by a graph that saved it."""
    p = problem(40, 2, 4, 64, 72)
    x = p["x"].clone().requires_grad_()
    row_of, _, bounds = mg.muon_expert_sort(p["choice"], 4)
    assert not mg.muon_expert_dispatch(x, row_of, bounds).requires_grad
    assert not mg.muon_dropout(x, 0.1).requires_grad
    y = x * 1.0
    penalty = (y * y).sum()
    mg.muon_dropout(y.detach(), 0.1, out=y.detach())
    with pytest.raises(RuntimeError, match="inplace"):
        penalty.backward()
    with torch.inference_mode():
        xi = p["x"].clone()
        want = mg.muon_dropout(xi, 0.3, seed=2)
        assert torch.equal(mg.muon_dropout(xi, 0.3, seed=2, out=xi), want) and torch.equal(xi, want)
        block(mg, p)


def test_gradients_where_the_group_reads_them(mg):
    """A Muon step of experts' matrices from the gradients that the backward pass left in the group's tensors is that
    of the same gradients copied there."""
    p = problem(300, 2, 5, 256, 136)
    _, _, _, dwg, dwu, _, _, _, bounds = block(mg, p)
    row_of, _, bounds = mg.muon_expert_sort(p["choice"], 5)
    xs = mg.muon_expert_dispatch(p["x"], row_of, bounds)
    h, gate, up = mg.muon_expert_glu_forward(xs, p["wg"], p["wu"], bounds)
    dh = rand(*h.shape, seed=9)
    results = []
    for in_place in (True, False):
        w = [p["wg"].clone(), p["wu"].clone()]
        g = [torch.zeros_like(t) for t in w]
        group = mg.MuonGroup([m for t in w for m in t], [m for t in g for m in t], [torch.zeros_like(m) for t in w for m in t])
        if in_place:
            mg.muon_expert_glu_backward(xs, p["wg"], p["wu"], gate, up, dh, bounds, dw_gate=g[0], dw_up=g[1])
        else:
            _, a, b = mg.muon_expert_glu_backward(xs, p["wg"], p["wu"], gate, up, dh, bounds)
            g[0].copy_(a)
            g[1].copy_(b)
        group.step(lr=0.02)
        results.append(w)
    assert mg.muon_sync_status() == mg.MUON_OK
    for a, b in zip(*results):
        assert torch.equal(a, b) and not torch.equal(a, p["wg"])


@pytest.fixture(scope="module")
def example(mg):
    spec = importlib.util.spec_from_file_location("post_training", os.path.join(ROOT, "examples", "post_training.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("objective", ["distill", "policy", "preference"])
def test_example_runs(example, objective):
    h = example.train(objective, steps=4, experts=6, choices=2, dropout=0.1)
    assert len(h) == 4 and all(v == v and abs(v) < 1e4 for v in h)


def test_example_gradients(example, mg):
    """Every gradient of the example's model with experts and dropout against fp64 autograd of its formulas, the
    router's choice and the masks taken from the run.  Two layers of about fifteen roundings to bf16 each (2^-8 at
    most, rms 2^-8 / sqrt 3) and a router whose logits are rounded: 2^-8 sqrt(30 / 3) = 0.012, with a factor of
    three for their way through the layers, in relative 2-norms."""
    model = example.Model(503, 128, 96, 2, seed=3, experts=5, choices=2, dropout=0.2)
    tokens = torch.randint(0, 503, (200,), generator=gen(1), device="cuda")
    logits, saved = model.forward(tokens)
    dlogits = rand(*logits.shape, seed=2, std=0.1)
    model.backward(dlogits, saved)

    leaves = [t.double().requires_grad_() for t in model.rest + [w for b in model.blocks for w in b]]
    embed, head, routers, flat = leaves[0], leaves[1], leaves[2:4], leaves[4:]
    x = embed[tokens]
    for i in range(2):
        wg, wu, wd = flat[3 * i:3 * i + 3]
        choice = saved[1][i][2]
        weights = torch.softmax(x @ routers[i].t(), dim=1).gather(1, choice)
        y = torch.zeros_like(x)
        for e in range(5):
            t, j = torch.nonzero(choice == e, as_tuple=True)
            v = torch.nn.functional.silu(x[t] @ wg[e].t()) * (x[t] @ wu[e].t())
            y = y.index_add(0, t, weights[t, j][:, None] * (v @ wd[e].t()))
        keep = mg.muon_dropout(torch.ones(x.shape, device="cuda"), 0.2, 3, offset=i)
        x = x + keep.double() * y
    want = torch.autograd.grad(x @ head.t(), leaves, dlogits.double())
    for k, (a, b) in enumerate(zip(model.rest_grads + model.grads, want)):
        err = ((a.double() - b).norm() / b.norm()).item()
        assert err <= 0.036, (k, err)
