"""Plain fp64 CPU oracle of a feed-forward block split over experts, and of dropout.

TEST INFRASTRUCTURE ONLY.  Only ``tests/`` may import this module; the library
never calls it and shares no code with it.  Pinned by
``tests/test_expert_oracle_pins.py`` (hand cases, published vectors, differences).
"""
from __future__ import annotations

import numpy as np

from oracle import glu_oracle as go


def sort(experts, n):
    """(row_of, slot_of, bounds) slot by slot; indices outside [0, n) last."""
    flat = [int(e) for e in np.asarray(experts).reshape(-1)]
    groups = [[] for _ in range(n + 1)]
    for slot, e in enumerate(flat):
        groups[e if 0 <= e < n else n].append(slot)
    slot_of = np.array([s for g in groups for s in g], dtype=np.int64)
    row_of = np.empty(len(flat), dtype=np.int64)
    row_of[slot_of] = np.arange(len(flat))
    bounds = np.concatenate([[0], np.cumsum([len(g) for g in groups[:n]])])
    return row_of.reshape(np.shape(experts)), slot_of, bounds


def dispatch(x, row_of, live):
    tokens, k = row_of.shape
    xs = np.zeros((tokens * k, x.shape[1]))
    for t in range(tokens):
        for j in range(k):
            if row_of[t, j] < live:
                xs[row_of[t, j]] = x[t]
    return xs


def combine(ys, row_of, live, weights=None, residual=None):
    tokens, k = row_of.shape
    y = np.zeros((tokens, ys.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    for t in range(tokens):
        for j in range(k):
            if row_of[t, j] < live:
                y[t] += (1.0 if weights is None else weights[t, j]) * ys[row_of[t, j]]
    return y


def combine_backward(dy, ys, row_of, live, weights):
    dys, dw = np.zeros(ys.shape), np.zeros(row_of.shape)
    for t in range(row_of.shape[0]):
        for j in range(row_of.shape[1]):
            r = row_of[t, j]
            if r < live:
                dys[r] = weights[t, j] * dy[t]
                dw[t, j] = float(dy[t] @ ys[r])
    return dys, dw


M32 = 0xFFFFFFFF


def philox4x32(counter, key, rounds=10):
    """The four words of one counter, in Python integers."""
    c, k = list(counter), list(key)
    for i in range(rounds):
        if i:
            k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & M32, (p >> 32) ^ c[3] ^ k[1], p & M32]
    return c


def drop_bits(n, seed, offset):
    """The 16-bit number of each of n elements."""
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    out = []
    for b in range((n + 7) // 8):
        for w in philox4x32((b & M32, b >> 32, offset & M32, offset >> 32), (seed & M32, seed >> 32)):
            out += [w & 0xFFFF, w >> 16]
    return np.array(out[:n], dtype=np.int64)


def dropout(x, p, seed, offset, residual=None):
    x = np.asarray(x, dtype=np.float64)
    cut = int(np.floor(p * 65536 + 0.5))
    keep = drop_bits(x.size, seed, offset).reshape(x.shape) >= cut
    y = np.zeros(x.shape)
    if cut < 65536:
        y[keep] = x[keep] / (1.0 - cut / 65536.0)
    return y if residual is None else y + residual


def segments(bounds, rows):
    """[first, last) rows of each expert, as the library reads bounds."""
    out = []
    for e in range(len(bounds) - 1):
        first = min(max(0 if e == 0 else int(bounds[e]), 0), rows)
        out.append((first, min(max(int(bounds[e + 1]), first), rows)))
    return out


def glu_forward(x, wg, wu, bounds, kind):
    rows, ffn = x.shape[0], wg.shape[1]
    out = [np.zeros((rows, ffn)) for _ in range(3)]
    for e, (a, b) in enumerate(segments(bounds, rows)):
        for o, v in zip(out, go.forward(x[a:b], wg[e], wu[e], kind)):
            o[a:b] = v
    return out


def glu_backward(x, wg, wu, gate, up, dh, bounds, kind):
    dx, dwg, dwu = np.zeros(x.shape), np.zeros(wg.shape), np.zeros(wu.shape)
    for e, (a, b) in enumerate(segments(bounds, x.shape[0])):
        dx[a:b], dwg[e], dwu[e] = go.backward(x[a:b], wg[e], wu[e], gate[a:b], up[a:b], dh[a:b], kind)
    return dx, dwg, dwu


def linear_forward(x, w, bounds):
    y = np.zeros((x.shape[0], w.shape[1]))
    for e, (a, b) in enumerate(segments(bounds, x.shape[0])):
        y[a:b] = x[a:b] @ w[e].T
    return y


def linear_backward(x, w, dy, bounds):
    dx, dw = np.zeros(x.shape), np.zeros(w.shape)
    for e, (a, b) in enumerate(segments(bounds, x.shape[0])):
        dx[a:b], dw[e] = dy[a:b] @ w[e], dy[a:b].T @ x[a:b]
    return dx, dw
