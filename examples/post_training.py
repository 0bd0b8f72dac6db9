"""A small post-training loop on one GPU: gated feed-forward blocks whose weight
gradients go straight into the Muon group's gradient tensors, a vocabulary
loss that starts the backward pass, AdamW for the embedding and the head.

    python examples/post_training.py [--objective distill|policy|preference]
                                     [--steps N] [--hidden D] [--ffn F] [--vocab V]
                                     [--experts E] [--choices K] [--dropout P]

The model has no attention (each position is read on its own), so that every
step is plain to follow: x = E[token]; x += (act(x Wg^T) * (x Wu^T)) Wd^T per
block; logits = x H^T.  With --experts, each block is E such blocks of which a
router picks K for every token, and with --dropout a block's output is dropped
in part before it joins x.  Data are synthetic.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import newton_schulz_frobenius_gb300 as mg  # noqa: E402


class Model:
    """Weights, their gradients and both optimizers' state, bf16 on the GPU."""

    def __init__(self, vocab, hidden, ffn, layers, seed=0, experts=0, choices=2, dropout=0.0):
        self.experts, self.choices, self.dropout, self.seed = experts, choices, dropout, seed
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols, std):
            return (torch.randn(rows, cols, device="cuda", generator=g) * std).bfloat16()

        self.embed = weight(vocab, hidden, 1.0)
        self.head = weight(vocab, hidden, hidden ** -0.5)
        self.blocks = [(weight(ffn, hidden, hidden ** -0.5), weight(ffn, hidden, hidden ** -0.5),
                        weight(hidden, ffn, ffn ** -0.5)) for _ in range(layers)]
        self.routers = []
        if experts:
            # every expert's matrices one after the other: the products take them as one tensor, the Muon group
            # steps each by itself
            self.blocks = [tuple(torch.stack([weight(*w.shape, w.shape[1] ** -0.5) for _ in range(experts)])
                                 for w in block) for block in self.blocks]
            self.routers = [weight(experts, hidden, hidden ** -0.5) for _ in range(layers)]
        weights = [w for block in self.blocks for w in block]
        self.grads = [torch.zeros_like(w) for w in weights]

        def each(tensors):
            return [m for t in tensors for m in (t if experts else [t])]
        self.matrices = each(weights)
        self.muon = mg.MuonGroup(self.matrices, each(self.grads), [torch.zeros_like(w) for w in self.matrices])
        self.rest = [self.embed, self.head] + self.routers
        self.rest_grads = [torch.zeros_like(w) for w in self.rest]
        self.moments = [[torch.zeros(w.shape, device="cuda") for w in self.rest] for _ in range(2)]
        self.t = 0

    def join(self, x, y, i):
        """x + y, y dropped in part: the same elements in a backward pass before the next step()."""
        if not self.dropout:
            return x + y
        return mg.muon_dropout(y, self.dropout, self.seed, offset=self.t * len(self.blocks) + i, residual=x)

    def forward(self, tokens):
        x = self.embed[tokens]
        kept = []
        for i, (wg, wu, wd) in enumerate(self.blocks):
            if self.experts:
                y, saved = self.experts_forward(i, x)
            else:
                h, gate, up = mg.muon_glu_forward(x, wg, wu)
                y, saved = h @ wd.t(), (x, h, gate, up)
            kept.append(saved)
            x = self.join(x, y, i)
        return x @ self.head.t(), (tokens, kept, x)

    def experts_forward(self, i, x):
        wg, wu, wd = self.blocks[i]
        share = torch.softmax((x @ self.routers[i].t()).float(), dim=1)
        weights, choice = torch.topk(share, self.choices, dim=1)
        row_of, _, bounds = mg.muon_expert_sort(choice, self.experts)
        xs = mg.muon_expert_dispatch(x, row_of, bounds)
        h, gate, up = mg.muon_expert_glu_forward(xs, wg, wu, bounds)
        ys = mg.muon_expert_linear_forward(h, wd, bounds)
        y = mg.muon_expert_combine(ys, row_of, bounds, weights=weights)
        return y, (x, share, choice, weights, row_of, bounds, xs, h, gate, up, ys)

    def experts_backward(self, i, dy, saved):
        wg, wu, wd = self.blocks[i]
        x, share, choice, weights, row_of, bounds, xs, h, gate, up, ys = saved
        dys, dweights = mg.muon_expert_combine_backward(dy, ys, row_of, bounds, weights)
        # the experts' gradients are written where the Muon group reads them
        dh, _ = mg.muon_expert_linear_backward(h, wd, dys, bounds, dw=self.grads[3 * i + 2])
        dxs, _, _ = mg.muon_expert_glu_backward(xs, wg, wu, gate, up, dh, bounds, dw_gate=self.grads[3 * i],
                                                dw_up=self.grads[3 * i + 1])
        dx = mg.muon_expert_combine(dxs, row_of, bounds)
        dshare = torch.zeros_like(share).scatter_(1, choice, dweights)
        dlogits = (share * (dshare - (dshare * share).sum(dim=1, keepdim=True))).to(x.dtype)
        torch.mm(dlogits.t(), x, out=self.rest_grads[2 + i])
        return dx + dlogits @ self.routers[i]

    def backward(self, dlogits, saved):
        tokens, kept, x = saved
        torch.mm(dlogits.t(), x, out=self.rest_grads[1])
        dx = dlogits @ self.head
        for i in reversed(range(len(self.blocks))):
            dy = dx
            if self.dropout:            # the same elements as in the forward pass
                dy = mg.muon_dropout(dx, self.dropout, self.seed, offset=self.t * len(self.blocks) + i)
            if self.experts:
                dx = dx + self.experts_backward(i, dy, kept[i])
                continue
            wg, wu, wd = self.blocks[i]
            x, h, gate, up = kept[i]
            torch.mm(dy.t(), h, out=self.grads[3 * i + 2])
            # the block's two large gradients are written where the Muon group reads them
            dblock, _, _ = mg.muon_glu_backward(x, wg, wu, gate, up, dy @ wd, dw_gate=self.grads[3 * i],
                                                dw_up=self.grads[3 * i + 1])
            dx = dx + dblock
        self.rest_grads[0].zero_().index_add_(0, tokens, dx)

    def step(self, lr, adam_lr):
        self.t += 1
        self.muon.step(lr=lr, beta=0.9, wd=0.0, nesterov=True)
        mg.muon_adamw_step(self.rest, self.rest_grads, *self.moments, lr=adam_lr, step=self.t)


def distill_batch(vocab, rows, k, g):
    """Tokens with, for each, the teacher's k largest logits and its log-sum-exp."""
    tokens = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    idx = (tokens[:, None] * 7 + torch.arange(k, device="cuda") * 13 + 1) % vocab
    logits = 6.0 - 0.3 * torch.arange(k, device="cuda").float().expand(rows, k)
    return tokens, idx.to(torch.int32), logits.contiguous(), torch.logsumexp(logits, 1) + 0.02


#: learning rates (Muon, AdamW): the policy may only move a little per step from the one it sampled with
RATES = {"distill": (0.02, 3e-3), "policy": (0.0005, 1e-4), "preference": (0.001, 1e-4)}


def train(objective="distill", steps=30, vocab=2003, hidden=256, ffn=512, layers=2, rows=512, seed=0, experts=0,
          choices=2, dropout=0.0):
    """Runs `steps` steps and returns the loss of each."""
    lr, adam_lr = RATES[objective]
    model = Model(vocab, hidden, ffn, layers, seed, experts, choices, dropout)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    tokens, idx, teacher, lse = distill_batch(vocab, rows, 16, g)
    weights = torch.full((rows,), 1.0 / rows, device="cuda")
    weights[::8] = 0.0                                          # prompt positions: outside the loss
    labels = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    reference = None
    history = []
    for _ in range(steps):
        logits, saved = model.forward(tokens)
        if objective == "distill":
            loss, dlogits = mg.muon_distill_loss(logits, idx, teacher, teacher_lse=lse, weights=weights, grad=logits)
        elif objective == "policy":
            # reward the sampled labels of even rows, punish those of odd ones
            adv = torch.where(torch.arange(rows, device="cuda") % 2 == 0, 1.0, -1.0)
            if reference is None:       # the sampling policy's log-probabilities
                _, reference, _ = mg.muon_policy_loss(logits, labels, adv)
            loss, logp, dlogits = mg.muon_policy_loss(logits, labels, adv, old_logp=reference, ref_logp=reference,
                                                      weights=weights, kl_coef=0.01, grad=logits)
        else:
            # rows in sequences of 16: chosen and rejected in turn
            bounds = torch.arange(0, rows + 1, 16, device="cuda", dtype=torch.int32)
            pairs = bounds.numel() // 2
            if reference is None:
                _, reference, _ = mg.muon_preference_loss(logits, labels, bounds)
            loss, _, dlogits = mg.muon_preference_loss(
                logits, labels, bounds, ref_logp=reference, beta=0.1, grad=logits,
                weights=torch.full((pairs,), 1.0 / pairs, device="cuda"))
        model.backward(dlogits, saved)
        model.step(lr, adam_lr)
        history.append(loss.sum())
    status = mg.muon_sync_status()
    if status != mg.MUON_OK:
        raise RuntimeError(f"device status {mg.status_str(status)}")
    return [float(v) for v in history]


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--objective", choices=("distill", "policy", "preference"), default="distill")
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--vocab", type=int, default=2003)
    p.add_argument("--hidden", type=int, default=256)
    p.add_argument("--ffn", type=int, default=512)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--rows", type=int, default=512)
    p.add_argument("--experts", type=int, default=0, help="experts per block; 0: one dense block")
    p.add_argument("--choices", type=int, default=2, help="experts of a token")
    p.add_argument("--dropout", type=float, default=0.0)
    a = p.parse_args()
    history = train(a.objective, a.steps, a.vocab, a.hidden, a.ffn, a.layers, a.rows, experts=a.experts,
                    choices=a.choices, dropout=a.dropout)
    for i, v in enumerate(history):
        print(f"step {i + 1:3d}  loss {v:.5f}")


if __name__ == "__main__":
    main()
