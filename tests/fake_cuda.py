"""The library's host code over a stand-in for the CUDA runtime (fake_cudart.c),
in a child process: no kernel runs, every pointer is a placeholder."""
from __future__ import annotations

import json
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PRELUDE = """
import ctypes, json, sys
import newton_schulz_frobenius_gb300 as mg
L = mg.lib()
fake = ctypes.CDLL(None)
fake.fake_log.restype = ctypes.c_char_p
P = 0x10000000

def log(kind=None):
    lines = [l.split() for l in fake.fake_log().decode().splitlines()]
    return [l[1:] for l in lines if kind is None or l[0] == kind]

def distill(rows=4, vocab=8192, dtype=0, k=8, lse=None, stream=0):
    st = L.muon_distill_loss(P, vocab, rows, vocab, dtype, P, 64, P, 0, k, lse, None, 1.0, P, P, vocab, stream)
    assert st == 0, mg.last_error_message()

def policy(rows=4, vocab=8192, dtype=0, stream=0):
    st = L.muon_policy_loss(P, vocab, rows, vocab, dtype, P, 64, P, None, None, None, 1.0, 0.2, 0.2, 0.0, P, P, P, vocab,
                            stream)
    assert st == 0, mg.last_error_message()

def preference(rows=4, vocab=8192, dtype=0, stream=0):
    st = L.muon_preference_loss(P, vocab, rows, vocab, dtype, P, 64, P, 64, 1, None, None, 0.1, 0.0, 0.0, 0, P, P, P,
                                vocab, stream)
    assert st == 0, mg.last_error_message()

def forward(tokens, hidden=256, ffn=512, stream=0):
    st = L.muon_glu_forward(P, P, P, P, P, P, tokens, hidden, ffn, 1, 0, stream)
    assert st == 0, mg.last_error_message()

def backward(tokens, hidden=256, ffn=512, stream=0):
    st = L.muon_glu_backward(P, P, P, P, P, P, P, P, P, tokens, hidden, ffn, 1, 0, stream)
    assert st == 0, mg.last_error_message()

def product(tile_n, symmetric=0, size=512):
    st = L.muon_debug_gemm(P, P, P, size, size, size, 1, 1, 1, symmetric, 0, 1.0, 0.0, 0.0, 0.0, tile_n, None)
    assert st == 0, mg.last_error_message()

def step(rows, cols):
    one = (ctypes.c_void_p * 1)(P)
    i64 = ctypes.c_int64 * 1
    st = L.muon_step(one, one, one, i64(rows), i64(cols), 1, 1, 1, 0.02, 0.95, 0.1, 1, None)
    assert st == 0, mg.last_error_message()
"""


def run(tmp_path, body, **env):
    """Runs `body` after the prelude; it leaves its result in `out`."""
    from newton_schulz_frobenius_gb300 import _build
    _build.build()
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    so = str(tmp_path / "fake_cudart.so")
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run([cc, "-shared", "-fPIC", "-O1", "-Wall", "-I", os.path.join(home, "include"),
                    os.path.join(ROOT, "tests", "fake_cudart.c"), "-o", so], check=True)
    r = subprocess.run([sys.executable, "-c", PRELUDE + body + "\nprint('OUT' + json.dumps(out))"], cwd=ROOT,
                       env=dict(os.environ, LD_PRELOAD=so, **env), capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    return json.loads(r.stdout.rsplit("OUT", 1)[1])
