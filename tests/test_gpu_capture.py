"""The losses and the feed-forward block recorded into CUDA graphs: after a first call on the stream that sizes its
workspace, a captured call allocates nothing, its replays give the plain call's results on new inputs, and go on doing
so after larger calls on the stream have taken new workspaces."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


def rand(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ids(*shape, high, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, high, shape, generator=g, device="cuda")


def cases(mg, n):
    """(inputs that change, call) of each operator at a size that grows with n; odd rows need padded copies."""
    V, D, F = 4099, 137, 201
    tok, ent, adv = ids(n, high=V, seed=1), ids(n, 64, high=V, seed=2), rand(n, seed=3, dtype=torch.float32)
    teach = rand(n, 64, seed=4)
    bounds = torch.tensor([0, n // 2, n], device="cuda")
    wg, wu = rand(F, D, seed=5) * 0.1, rand(F, D, seed=6) * 0.1
    gate, up = rand(n, F, seed=7), rand(n, F, seed=8)
    x, logits, dh = rand(n, D, seed=9), rand(n, V, seed=10), rand(n, F, seed=11)
    return {
        "distill": (logits, lambda: mg.muon_distill_loss(logits, ent, teach)),
        "policy": (logits, lambda: mg.muon_policy_loss(logits, tok, adv)),
        "preference": (logits, lambda: mg.muon_preference_loss(logits, tok, bounds)),
        "forward": (x, lambda: mg.muon_glu_forward(x, wg, wu)),
        "backward": (dh, lambda: mg.muon_glu_backward(x, wg, wu, gate, up, dh)),
    }


@pytest.mark.parametrize("name", ["distill", "policy", "preference", "forward", "backward"])
def test_replays_survive_larger_calls(mg, name):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        small, call = cases(mg, 24)[name]
        _, large = cases(mg, 80000)[name]
        call()
        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            out = call()
        large()
        large()
        for seed in (21, 22):
            small.copy_(rand(*small.shape, seed=seed))
            graph.replay()
            got = [t.clone() for t in out]
            large()
            for a, b in zip(got, call()):
                assert torch.equal(a, b)
    s.synchronize()
    assert mg.muon_sync_status() == mg.MUON_OK
