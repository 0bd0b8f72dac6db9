"""Host threads calling the losses and the feed-forward block at the same time, each on its own stream: the bytes of
the same calls made one after another.  The kernels' per-device set-up and occupancies, and the per-stream
workspaces, are shared or raced for."""
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


def jobs(mg):
    """Per thread the calls of one round; sizes grow from call to call, so that workspaces do."""
    g = torch.Generator(device="cuda").manual_seed(7)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    def vocabulary(rows, vocab, dtype):
        x = rand(rows, vocab, dtype=dtype)
        tok = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        ent = torch.randint(0, vocab, (rows, 48), generator=g, device="cuda", dtype=torch.int32)
        adv, teach = rand(rows, dtype=torch.float32), rand(rows, 48, dtype=torch.float32)
        bounds, lse = torch.tensor([0, rows // 3, rows], device="cuda"), adv + 6
        return [lambda s: mg.muon_policy_loss(x, tok, adv, stream=s),
                lambda s: mg.muon_distill_loss(x, ent, teach, teacher_lse=lse, stream=s),
                lambda s: mg.muon_distill_loss(x, ent, teach, stream=s),
                lambda s: mg.muon_preference_loss(x, tok, bounds, stream=s)]

    def block(tokens, hidden, ffn, dtype):
        x, wg, wu = rand(tokens, hidden, dtype=dtype), rand(ffn, hidden, dtype=dtype) * 0.1, rand(ffn, hidden, dtype=dtype)
        dh, gate, up = (rand(tokens, ffn, dtype=dtype) for _ in range(3))
        return [lambda s: mg.muon_glu_forward(x, wg, wu, stream=s),
                lambda s: mg.muon_glu_backward(x, wg, wu, gate, up, dh, stream=s)]

    h, b, f = torch.float16, torch.bfloat16, torch.float32
    return [vocabulary(9, 4099, f) + vocabulary(300, 50257, b), block(3, 72, 40, b) + block(700, 515, 300, b),
            vocabulary(20, 131072, h) + block(64, 256, 512, h), block(130, 264, 1032, h) + vocabulary(2000, 777, f)]


def test_threads_on_separate_streams_match_serial_calls(mg):
    work = jobs(mg)
    torch.cuda.synchronize()
    want = [[call(None) for call in calls] for calls in work]
    torch.cuda.synchronize()
    for _ in range(2):                              # fresh workspaces, then grown ones
        streams = [torch.cuda.Stream() for _ in work]
        got, errors = [None] * len(work), []
        start = threading.Barrier(len(work))

        def run(i):
            try:
                start.wait(timeout=60)
                got[i] = [[call(streams[i]) for call in work[i]] for _ in range(3)]
                streams[i].synchronize()
            except Exception as e:      # noqa: BLE001 - reported on the main thread
                errors.append((i, repr(e)))

        threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
        for th in threads:
            th.start()
        for th in threads:
            th.join(timeout=300)
        assert not any(th.is_alive() for th in threads) and not errors, errors
        torch.cuda.synchronize()
        assert mg.muon_sync_status() == mg.MUON_OK
        for i, rounds in enumerate(got):
            for outs in rounds:
                for j, (a, b) in enumerate(zip(outs, want[i])):
                    assert all(torch.equal(u, v) for u, v in zip(a, b)), (i, j)
