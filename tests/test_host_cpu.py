"""What the library's host code asks of the CUDA runtime, over a stand-in for it."""
from tests.fake_cuda import run


def test_a_workspace_that_a_graph_holds_outlives_growth(tmp_path):
    """A captured call's launches keep the workspace's address: a larger call on the stream takes a new block and
    leaves that one alone.  Blocks that no graph has seen are freed as before."""
    out = run(tmp_path, """
distill()
first = log("malloc")[-1][1]
distill(rows=20000, k=64)                       # grows: nothing was captured
second = log("malloc")[-1][1]
freed = [f[1] for f in log("free")]
fake.fake_set_capturing(1)
distill()
preference()
fake.fake_set_capturing(0)
distill(rows=60000, k=64)                       # grows past the block a graph holds
third = log("malloc")[-1][1]
kept = [f[1] for f in log("free")]
distill(rows=200000, k=64)
last = [f[1] for f in log("free")]
out = dict(first=first, second=second, third=third, freed=freed, kept=kept, last=last)
""")
    assert out["freed"] == [out["first"]]
    assert out["kept"] == [out["first"]]
    assert out["last"] == [out["first"], out["third"]]


def test_growth_during_capture_leaves_the_block(tmp_path):
    """A call that has to grow the workspace while the stream is captured neither waits for the stream nor frees what
    earlier launches of the graph hold."""
    out = run(tmp_path, """
distill()
fake.fake_set_capturing(1)
distill(rows=20000, k=64)
out = [f[1] for f in log("free")]
""")
    assert out == []


def test_failed_growth_during_capture_keeps_the_workspace(tmp_path):
    out = run(tmp_path, """
import os
distill()
n = len(log("malloc"))
fake.fake_set_capturing(1)
os.environ["MUON_FAIL_ALLOC"] = "1"
ctypes.CDLL(None).setenv(b"MUON_FAIL_ALLOC", b"1", 1)
st = L.muon_distill_loss(P, 8192, 20000, 8192, 0, P, 64, P, 0, 64, None, None, 1.0, P, P, 8192, None)
distill()                                       # the block it has still serves
out = dict(status=st, nomem=mg.MUON_ENOMEM, mallocs=len(log("malloc")) - n, frees=len(log("free")))
""")
    assert out["status"] == out["nomem"] and out["mallocs"] == 0 and out["frees"] == 0
