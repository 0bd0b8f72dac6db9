"""What the experts' products ask for as scratch, over a stand-in for the CUDA runtime."""
import pytest

from tests.fake_cuda import run

ASK = """
def ask(name, *args):
    need = ctypes.c_int64(0)
    st = getattr(L, name)(*args, None, ctypes.byref(need), None)
    assert st in (mg.MUON_OK, mg.MUON_ENOMEM), mg.last_error_message()
    assert (st == mg.MUON_ENOMEM) == (need.value > 0)
    return need.value

def glu_backward(rows, experts, hidden, ffn):
    return ask("muon_expert_glu_backward", *[P] * 10, rows, experts, hidden, ffn, mg.MUON_BF16, 0)

def linear_backward(rows, experts, cols, outs):
    return ask("muon_expert_linear_backward", *[P] * 6, rows, experts, cols, outs, mg.MUON_BF16)

def glu_forward(rows, experts, hidden, ffn):
    return ask("muon_expert_glu_forward", *[P] * 7, rows, experts, hidden, ffn, mg.MUON_BF16, 0)

def linear_forward(rows, experts, cols, outs):
    return ask("muon_expert_linear_forward", *[P] * 4, rows, experts, cols, outs, mg.MUON_BF16)
"""


@pytest.mark.parametrize("rows,experts", [(64, 256), (64, 1024), (1, 1024), (255, 256), (256, 256), (5000, 256)])
def test_last_blocks_of_no_more_experts_than_rows(tmp_path, rows, experts):
    """The backward passes keep 64 rows for each expert that can have any, beside dg and du."""
    out = run(tmp_path, ASK + f"out = [glu_backward({rows}, {experts}, 7168, 2048), linear_backward({rows}, {experts}, 2048, 7168)]")
    blocks = 64 * min(rows, experts)
    assert out == [2 * rows * 2048 * 2 + blocks * (2 * 2048 + 7168) * 2, blocks * (2048 + 7168) * 2]
