"""The losses at the largest sizes they accept: vocabularies up to 2^19 (a row on 16 CTAs), a thousand teacher entries
on them, in every type and alignment.  Bars as for the smaller sizes."""
import numpy as np
import pytest

from tests.test_gpu_losses import check_distill, check_policy, check_preference, matrix, teacher

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

VOCABS = [400003, (1 << 19) - 5, 1 << 19]


@pytest.fixture(scope="module")
def mg():
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_frobenius_gb300 as pkg
    return pkg


@pytest.mark.parametrize("dtype,layout", [("f32", "plain"), ("f32", "odd"), ("bf16", "odd"), ("f16", "pitch")])
@pytest.mark.parametrize("vocab", VOCABS)
def test_largest_vocabularies(mg, vocab, dtype, layout):
    check_policy(mg, matrix(3, vocab, dtype, vocab, layout), dtype, seed=vocab)
    x = matrix(3, vocab, dtype, vocab + 1, layout)
    for k, tail in ((64, False), (1024, True)):
        idx, t, lse = teacher(x, k, vocab + k, 1.0, tail)
        check_distill(mg, x, idx, t, lse, dtype)
    tok = np.array([0, vocab - 1, vocab // 3])
    check_preference(mg, matrix(3, vocab, dtype, vocab + 2, layout), tok, [0, 1, 3], None, None, dtype)
    assert mg.muon_sync_status() == mg.MUON_OK
