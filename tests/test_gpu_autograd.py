"""The losses and the feed-forward block beside autograd: gradients passed on by hand, and tensors written in place
noticed by a graph that saved them."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


def rand(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def calls(mg):
    tok, adv = torch.arange(4, device="cuda"), rand(4, seed=1)
    return {
        "policy": lambda x, **kw: mg.muon_policy_loss(x, tok, adv, **kw)[-1],
        "distill": lambda x, **kw: mg.muon_distill_loss(x, tok[:, None].contiguous(), adv[:, None].contiguous(), **kw)[-1],
        "preference": lambda x, **kw: mg.muon_preference_loss(x, tok, torch.tensor([0, 2, 4], device="cuda"), **kw)[-1],
    }


@pytest.mark.parametrize("name", ["policy", "distill", "preference"])
def test_gradient_over_saved_logits_is_noticed(mg, name):
    call = calls(mg)[name]
    w = rand(4, 50, seed=2).requires_grad_()
    logits = w * 1.0
    penalty = (logits * logits).sum()               # saves the logits
    before = logits._version
    g = call(logits)
    assert logits._version == before and not g.requires_grad
    call(logits.detach(), grad=logits.detach())
    assert logits._version > before
    with pytest.raises(RuntimeError, match="inplace"):
        penalty.backward()


@pytest.mark.parametrize("name", ["policy", "distill", "preference"])
def test_gradient_passed_on_in_place(mg, name):
    """The product that made the logits does not need them: their gradient may take their place."""
    call = calls(mg)[name]
    x, head = rand(4, 16, seed=3), rand(50, 16, seed=4).requires_grad_()
    logits = x @ head.t()
    g = call(logits.detach())
    want, = torch.autograd.grad(logits, head, g, retain_graph=True)
    logits.backward(call(logits.detach(), grad=logits.detach()))
    assert torch.equal(head.grad, want)


def test_weight_gradients_over_saved_tensors_are_noticed(mg):
    x, wg, wu, dh = (rand(*s, seed=i, dtype=torch.bfloat16) for i, s in enumerate([(6, 64), (32, 64), (32, 64), (6, 32)]))
    h, gate, up = mg.muon_glu_forward(x, wg, wu)
    buf = [rand(32, 64, seed=9, dtype=torch.bfloat16).requires_grad_() * 1.0 for _ in range(2)]
    for k, name in enumerate(("dw_gate", "dw_up")):
        y = (buf[k] * buf[k]).sum()
        mg.muon_glu_backward(x, wg, wu, gate, up, dh, **{name: buf[k].detach()})
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()


def test_inference_tensors_are_written_too(mg):
    with torch.inference_mode():
        x = rand(4, 50, seed=5)
        want = calls(mg)["policy"](x)
        assert torch.equal(calls(mg)["policy"](x, grad=x), want) and torch.equal(x, want)
