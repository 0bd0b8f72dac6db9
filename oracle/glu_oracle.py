"""Plain fp64 CPU oracle of the gated feed-forward block and its gradients.

TEST INFRASTRUCTURE ONLY.  Only ``tests/`` may import this module; the library
never calls it and shares no code with it.  Pinned by
``tests/test_glu_oracle_pins.py`` (differences, closed forms).
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[float])
_erfc = np.vectorize(math.erfc, otypes=[float])


def act(g, kind):
    if kind == "silu":
        return g / (1.0 + np.exp(-g))
    if kind == "gelu":
        return 0.5 * g * _erfc(-g / math.sqrt(2.0))
    return 0.5 * g * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def act_grad(g, kind):
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        return 0.5 * _erfc(-g / math.sqrt(2.0)) + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    th = np.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * k * (1.0 + 3 * 0.044715 * g * g)


def forward(x, wg, wu, kind):
    gate, up = x @ wg.T, x @ wu.T
    return act(gate, kind) * up, gate, up


def backward(x, wg, wu, gate, up, dh, kind, round_to=None):
    """(dx, dw_gate, dw_up); round_to rounds dg and du as the library stores them."""
    dg, du = dh * up * act_grad(gate, kind), dh * act(gate, kind)
    if round_to is not None:
        dg, du = round_to(dg), round_to(du)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x
