"""Plain fp64 CPU oracle of the vocabulary losses and their gradients.

TEST INFRASTRUCTURE ONLY.  Only ``tests/`` may import this module; the library
never calls it and shares no code with it.  Pinned by
``tests/test_loss_oracle_pins.py`` (differences, closed forms).

One row at a time, written from the definitions in ``include/muon.h``: z = x / T,
q = softmax(z).  Every function returns its per-row (or per-pair) results and
the dense gradient of the weighted sum of the losses with respect to x.
"""
from __future__ import annotations

import numpy as np


def _log_softmax(z):
    m = z.max()
    return z - (m + np.log(np.exp(z - m).sum()))


def distill(x, idx, t, *, lse=None, weights=None, temperature=1.0):
    rows, vocab = x.shape
    loss, grad = np.zeros(rows), np.zeros((rows, vocab))
    for r in range(rows):
        w = 1.0 if weights is None else float(weights[r])
        if w == 0.0:
            continue
        lq = _log_softmax(x[r] / temperature)
        q = np.exp(lq)
        ok = (idx[r] >= 0) & (idx[r] < vocab)
        ids, zt = idx[r][ok], t[r][ok] / temperature
        if len(ids) == 0:
            lp = np.zeros(0)
        elif lse is None:
            lp = _log_softmax(zt)
        else:
            lp = zt - float(lse[r])
        p = np.exp(lp)
        kl = sum(pj * (lpj - lq[i]) for pj, lpj, i in zip(p, lp, ids) if pj > 0)
        dense = np.zeros(vocab)
        np.add.at(dense, ids, p)
        mass = p.sum()
        dz = mass * q - dense
        if lse is not None:
            outside = np.ones(vocab, bool)
            outside[ids] = False
            pr, qr = max(0.0, 1.0 - mass), q[outside].sum()
            if pr > 0 and qr > 0:
                kl += pr * (np.log(pr) - np.log(qr))
                dz = (mass + pr) * q - dense - np.where(outside, pr * q / qr, 0.0)
        loss[r] = w * temperature ** 2 * kl
        grad[r] = w * temperature * dz
    return loss, grad


def policy(x, tokens, adv, *, old=None, ref=None, weights=None, temperature=1.0, clip_low=0.2, clip_high=0.2, kl=0.0):
    rows, vocab = x.shape
    loss, logp, grad = np.zeros(rows), np.zeros(rows), np.zeros((rows, vocab))
    for r in range(rows):
        w = 1.0 if weights is None else float(weights[r])
        a = int(tokens[r])
        if w == 0.0 or not 0 <= a < vocab:
            continue
        lq = _log_softmax(x[r] / temperature)
        lp = lq[a]
        ratio = 1.0 if old is None else np.exp(lp - float(old[r]))
        clipped = min(max(ratio, 1.0 - clip_low), 1.0 + clip_high)
        A = float(adv[r])
        first = ratio * A <= clipped * A
        L = -(ratio * A if first else clipped * A)
        dl = -ratio * A if first else 0.0
        if kl:
            d = float(ref[r]) - lp
            L += kl * (np.expm1(d) - d)
            dl -= kl * np.expm1(d)
        one = np.zeros(vocab)
        one[a] = 1.0
        loss[r], logp[r] = w * L, lp
        grad[r] = w * dl * (one - np.exp(lq)) / temperature
    return loss, logp, grad


def preference(x, tokens, bounds, *, ref=None, weights=None, beta=0.1, margin=0.0, smoothing=0.0, average=False):
    rows, vocab = x.shape
    pairs = (len(bounds) - 1) // 2
    loss, seq, grad = np.zeros(pairs), np.zeros(2 * pairs), np.zeros((rows, vocab))
    lq = [None] * rows
    count = np.zeros(2 * pairs)
    for s in range(2 * pairs):
        for r in range(int(bounds[s]), int(bounds[s + 1])):
            if 0 <= tokens[r] < vocab:
                lq[r] = _log_softmax(x[r])
                seq[s] += lq[r][int(tokens[r])]
                count[s] += 1
        if average and count[s]:
            seq[s] /= count[s]
    for i in range(pairs):
        w = 1.0 if weights is None else float(weights[i])
        rc, rr = (0.0, 0.0) if ref is None else (float(ref[2 * i]), float(ref[2 * i + 1]))
        h = beta * ((seq[2 * i] - rc) - (seq[2 * i + 1] - rr)) - margin
        nls = np.logaddexp(0.0, -h)          # -log sigmoid(h)
        pls = np.logaddexp(0.0, h)           # -log sigmoid(-h)
        if w == 0.0:
            continue
        loss[i] = w * ((1 - smoothing) * nls + smoothing * pls)
        dh = w * beta * (smoothing * np.exp(-nls) - (1 - smoothing) * np.exp(-pls))
        for s, sign in ((2 * i, 1.0), (2 * i + 1, -1.0)):
            share = 1.0 / count[s] if average and count[s] else 1.0
            for r in range(int(bounds[s]), int(bounds[s + 1])):
                if lq[r] is not None:
                    grad[r] = -np.exp(lq[r]) * (sign * dh * share)
                    grad[r][int(tokens[r])] += sign * dh * share
    return loss, seq, grad
