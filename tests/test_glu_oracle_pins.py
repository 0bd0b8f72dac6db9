"""Pins of the feed-forward oracle: activations at known points, gradients
against central differences (step 1e-5 in fp64: about 1e-9 of the scale)."""
import math

import numpy as np
import pytest

from oracle import glu_oracle as go

KINDS = ["silu", "gelu", "gelu_tanh"]


@pytest.mark.parametrize("kind", KINDS)
def test_activation_values(kind):
    assert go.act(np.array(0.0), kind) == 0
    assert abs(go.act(np.array(20.0), kind) - 20) < 1e-6 and abs(go.act(np.array(-20.0), kind)) < 1e-6
    one = {"silu": 1 / (1 + math.exp(-1)), "gelu": 0.841344746068543, "gelu_tanh": 0.841191990608306}[kind]
    assert abs(go.act(np.array(1.0), kind) - one) < 1e-12


@pytest.mark.parametrize("kind", KINDS)
def test_gradients_are_difference_quotients(kind):
    rng = np.random.default_rng(2)
    x, wg, wu = rng.normal(size=(3, 5)), rng.normal(size=(4, 5)), rng.normal(size=(4, 5))
    dh = rng.normal(size=(3, 4))
    h, gate, up = go.forward(x, wg, wu, kind)
    got = go.backward(x, wg, wu, gate, up, dh, kind)
    for k, m in enumerate((x, wg, wu)):
        num = np.zeros_like(m)
        for i in np.ndindex(m.shape):
            out = []
            for e in (1e-5, -1e-5):
                args = [x.copy(), wg.copy(), wu.copy()]
                args[k][i] += e
                out.append((go.forward(*args, kind)[0] * dh).sum())
            num[i] = (out[0] - out[1]) / 2e-5
        assert np.abs(num - got[k]).max() < 1e-7
