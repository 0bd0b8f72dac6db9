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
