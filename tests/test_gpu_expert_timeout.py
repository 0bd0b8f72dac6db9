"""Waits of the experts' products that run out, with no GPU fault.

The test hook muon_debug_arm_stall leaves one stage of CTA 0 unfilled: it issues no
copy for it, the other CTA of the pair fills its half and reports to CTA 0.  So the
issuer's, the producers' and both CTAs' epilogue waits give up after about two
seconds; the odd CTA, some of whose copies the even one does not wait for, then
waits two more, also where its producer had issued all of its copies before.
Each test checks that the status reads MUON_ETIMEOUT once and that the same call
on the same stream then gives the results that it gave before, bit for bit.
"""
import time

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    yield pkg
    pkg.muon_debug_arm_stall(0)


def calls(mg, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, experts, hidden, ffn = 1200, 2, 1024, 768

    def r(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * 0.1).to(dtype)
    x, wg, wu, wd = r(rows, hidden), r(experts, ffn, hidden), r(experts, ffn, hidden), r(experts, hidden, ffn)
    bounds = torch.tensor([0, 600, 1200], dtype=torch.int32, device="cuda")
    h, gate, up = mg.muon_expert_glu_forward(x, wg, wu, bounds)
    return dict(
        glu_forward=lambda: mg.muon_expert_glu_forward(x, wg, wu, bounds),
        linear_forward=lambda: (mg.muon_expert_linear_forward(h, wd, bounds),),
        glu_backward=lambda: mg.muon_expert_glu_backward(x, wg, wu, gate, up, h, bounds),
        linear_backward=lambda: mg.muon_expert_linear_backward(h, wd, x, bounds),
        weights_alone=lambda: mg.muon_expert_linear_backward(h, wd, x, bounds, need_dx=False)[1:],
    )


@pytest.mark.parametrize("stage", [0, 4])
@pytest.mark.parametrize("name", ["linear_forward", "glu_forward", "linear_backward", "glu_backward", "weights_alone"])
def test_wait_runs_out(mg, name, stage):
    """The first stage, and one of the ring's second lap (of the weights' gradients alone: the copied last k-block)."""
    call = calls(mg)[name]
    want = call()
    assert mg.muon_sync_status() == mg.MUON_OK
    mg.muon_debug_arm_stall(mg.STALL_EXPERT, stage)
    try:
        t0 = time.perf_counter()
        call()
        st = mg.muon_sync_status()
        waited = time.perf_counter() - t0
    finally:
        mg.muon_debug_arm_stall(0)
    assert st == mg.MUON_ETIMEOUT, mg.status_str(st)
    assert 3.5 <= waited <= 60.0, waited                  # the waits' limit, and the odd CTA's wait for its copies
    assert mg.muon_sync_status() == mg.MUON_OK            # reading cleared it
    got = call()
    assert mg.muon_sync_status() == mg.MUON_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))
