"""What the CUDA sources must not hold, read as text."""
from __future__ import annotations

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "newton_schulz_frobenius_gb300", "csrc")


def _sources():
    return sorted(p for e in ("cu", "cuh", "h") for p in glob.glob(os.path.join(CSRC, "*." + e)))


def test_no_multicast_load():
    """No bulk copy of the library delivers to several CTAs of a cluster: the
    library also runs in jobs on several GPUs.  (tcgen05.commit's multicast
    arrive is a signal, not a load.)"""
    for path in _sources():
        text = re.sub(r'"\s*\n\s*"', "", open(path).read())     # adjacent string literals joined
        for ins in re.findall(r"cp\.async\.bulk[^;\"]*", text):
            assert "multicast" not in ins, (path, ins)
        assert "MUON_MC" not in text, path


def test_every_source_counts_for_a_rebuild():
    from newton_schulz_frobenius_gb300 import _build
    assert {os.path.basename(p) for p in os.listdir(CSRC)} <= {os.path.basename(p) for p in _build._deps()}


def test_no_helper_without_a_caller():
    """Every function that the operators' files define is called somewhere."""
    everything = "".join(open(p).read() for p in _sources())
    for name in ("losses.cu", "glu.cu"):
        text = open(os.path.join(CSRC, name)).read()
        defined = set(re.findall(r"__forceinline__ [\w:<>&* ]*?(\w+)\(", text))
        assert len(defined) > 5
        unused = {n for n in defined if len(re.findall(rf"\b{n}\b", everything)) < 2}
        assert not unused, (name, sorted(unused))
