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


CALLS = """
calls = dict(
    policy=lambda: policy(rows=200, vocab=70001, dtype=1),          # clusters, above 48 KB
    statistics=lambda: preference(rows=200, vocab=70001, dtype=1),
    distill=lambda: distill(rows=200, vocab=70001, dtype=1, k=64),
    wide=lambda: policy(rows=200, vocab=1 << 19),                   # 16 CTAs per row
    few=lambda: forward(5), forward=lambda: forward(500), backward=lambda: backward(500),
    product=lambda: product(128), paired=lambda: product(256),
    small=lambda: step(128, 128),
)
"""


def test_every_device_gets_its_kernels_set_up(tmp_path):
    """Limits of shared memory and cluster size, and how many clusters fit, are per device: a second device of the
    process serves the same calls as the first."""
    out = run(tmp_path, CALLS + """
out = {}
for name, call in calls.items():
    out[name] = []
    for d in (0, 1, 0):
        fake.fake_set_device(d)
        fake.fake_clear()
        try:
            call()
            bad = [l for l in log("launch") if l[5] != "0" or l[0] != str(d)]
            out[name].append([len(log("launch")) > 0, bad, len(log("attribute"))])
        except AssertionError as e:
            out[name].append(str(e))
""")
    for name, (first, second, again) in out.items():
        assert first == [True, [], first[2]] and first[2] > 0, (name, first)
        assert second == first, (name, second)
        assert again == [True, [], 0], (name, again)          # set up once


def test_a_failing_device_leaves_the_others_alone(tmp_path):
    """An error of one device's set-up is neither kept for it nor passed on."""
    out = run(tmp_path, CALLS + """
out = {}
for name, call in calls.items():
    out[name] = []
    for failing, d in ((0, 0), (0, 1), (-1, 0)):
        fake.fake_set_failing(failing)
        fake.fake_set_device(d)
        try:
            call()
            out[name].append("ok")
        except AssertionError:
            out[name].append("error")
""")
    for name, got in out.items():
        assert got == ["error", "ok", "ok"], (name, got)


def test_distillation_plans_with_its_own_shared_memory(tmp_path):
    """How many clusters fit is asked for what a launch takes, to the kilobyte, whatever the teacher's entries: the
    grid is the rows' clusters or all that fit, no fewer and no more."""
    out = run(tmp_path, """
out = []
for vocab, dtype in ((57344, 1), (131072, 0), (1 << 19, 0), (5000, 2)):
    for k in (1, 64, 256, 512, 1024):
        fake.fake_clear()
        distill(rows=9000, vocab=vocab, dtype=dtype, k=k)
        dev, fn, smem, cluster, grid, code = log("launch")[-1]
        asked = [l for l in log("occupancy") if l[1] == fn]
        out.append((vocab, k, int(smem), int(cluster), int(grid), int(code), [int(v) for v in asked[-1][2:]] if asked else None))
""")
    known = {}
    for vocab, k, smem, cluster, grid, code, asked in out:
        assert code == 0
        key = (vocab, cluster, (smem + 1023) // 1024)
        if asked:
            known[key] = asked
        size, width, fits = known[key]
        assert width == cluster and smem <= size < smem + 1024, (vocab, k, smem, known[key])
        assert grid == cluster * min(9000, fits)
