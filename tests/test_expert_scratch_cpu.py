"""What the experts' products ask for as scratch, over a stand-in for the CUDA runtime."""
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


def test_last_blocks_of_no_more_experts_than_rows(tmp_path):
    """The backward passes keep 64 rows for each expert that can have any, beside dg and du."""
    calls = [(64, 256), (64, 1024), (1, 1024), (255, 256), (256, 256), (5000, 256)]
    out = run(tmp_path, ASK + f"out = [[glu_backward(r, e, 7168, 2048), linear_backward(r, e, 2048, 7168)] for r, e in {calls}]")
    for (rows, experts), got in zip(calls, out):
        blocks = 64 * min(rows, experts)
        assert got == [2 * rows * 2048 * 2 + blocks * (2 * 2048 + 7168) * 2, blocks * (2048 + 7168) * 2], (rows, experts)


def test_forward_passes_ask_for_running_sums_alone(tmp_path):
    """Aligned forward passes need nothing, and no place to say so, up to 65536 columns; beyond, 128 KB for each of the
    SMs that the launch takes (pairs of them, no more than tiles), and a call without that is refused."""
    out = run(tmp_path, ASK + """
def size(k, rows, outs):
    return [glu_forward(rows, 2, k, outs), linear_forward(rows, 2, k, outs)]
out = dict(short=size(65536, 4, 32), long=size(65536 + 64, 4, 32), many=size(65536 + 8, 100000, 8192))
for k in (65536, 65536 + 64):
    out[k] = [L.muon_expert_glu_forward(*[P] * 7, 4, 2, k, 32, mg.MUON_BF16, 0, None, None, None),
              L.muon_expert_linear_forward(*[P] * 4, 4, 2, k, 32, mg.MUON_BF16, None, None, None)]
out["codes"] = [mg.MUON_OK, mg.MUON_EINVAL]
""")
    ok, refused = out["codes"]
    assert out["short"] == [0, 0] and out["65536"] == [ok, ok]
    # 4 rows to two experts: at most 3 row tiles of one tile of columns
    assert out["long"] == [2 * 3 * 131072] * 2 and out["65600"] == [refused] * 2
    assert out["many"] == [152 * 131072] * 2


def test_backward_passes_count_both_contractions(tmp_path):
    """dx of the gated block contracts 2 ffn columns, the weights' gradients an expert's rows."""
    out = run(tmp_path, ASK + """
out = [linear_backward(64, 1, 64, 65536), linear_backward(64, 1, 64, 65600), glu_backward(64, 1, 64, 32768),
       glu_backward(64, 1, 64, 32832), linear_backward(65536, 1, 64, 64), linear_backward(65537, 1, 64, 64)]
""")

    def rest(rows, columns, glu):
        return (4 * rows * glu) + 64 * columns * 2
    want = [rest(64, 64 + 65536, 0), rest(64, 64 + 65600, 0), rest(64, 64 + 2 * 32768, 32768), rest(64, 64 + 2 * 32832, 32832),
            rest(65536, 128, 0), rest(65537, 128, 0)]
    extra = [a - b for a, b in zip(out, want)]
    assert [e > 0 for e in extra] == [False, True, False, True, False, True]
    assert all(e % (2 * 131072) == 0 for e in extra)
