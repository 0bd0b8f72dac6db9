"""Cases that time the loss and feed-forward operators, with their plain forms.

``run`` computes one pass: where ``own`` is false in elementary torch
operations on fp32 copies of the inputs, rounded once at the end; where it is
true through the library's entry points.  ``exact`` computes the same outputs
in fp64, one row or one matrix at a time, written from the formulas.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # a short answer distilled in one micro-batch: latency counts
        {"name": "distill_answer_16", "op": "distill", "rows": 16, "vocab": 32000, "k": 32, "dtype": "bf16",
         "tail": False, "temperature": 1.0, "masked": 0.0, "pad": 0},
        # packed fp16 batch, odd vocabulary (rows off 16-byte boundaries), prompts and padding masked
        {"name": "distill_packed_odd", "op": "distill", "rows": 1023, "vocab": 50001, "k": 100, "dtype": "f16",
         "tail": False, "temperature": 2.0, "masked": 0.3, "pad": 0},
        # a long micro-batch against a 128 Ki vocabulary, the teacher's rest kept as one class
        {"name": "distill_long_tail", "op": "distill", "rows": 8192, "vocab": 131072, "k": 64, "dtype": "bf16",
         "tail": True, "temperature": 1.0, "masked": 0.1, "pad": 0},
        # a handful of fp32 rows (a reduced head, a test set-up): the smallest policy call
        {"name": "policy_rows_8_f32", "op": "policy", "rows": 8, "vocab": 32768, "dtype": "f32", "temperature": 1.0,
         "kl": 0.04, "masked": 0.0, "pad": 0},
        # fp32 logits of an odd vocabulary whose last columns are head padding at -inf
        {"name": "policy_odd_f32", "op": "policy", "rows": 2047, "vocab": 100003, "dtype": "f32", "temperature": 0.7,
         "kl": 0.01, "masked": 0.2, "pad": 35},
        # a packed batch of rollouts
        {"name": "policy_rollouts", "op": "policy", "rows": 8192, "vocab": 65536, "dtype": "bf16", "temperature": 1.0,
         "kl": 0.0, "masked": 0.25, "pad": 0},
        # four short pairs
        {"name": "preference_4_pairs", "op": "preference", "pairs": 4, "rows": 600, "vocab": 32000, "dtype": "bf16",
         "average": False, "smoothing": 0.0, "masked": 0.3, "pad": 0},
        # ragged pairs up to a thousand tokens, length-normalised, fp16 logits
        {"name": "preference_ragged", "op": "preference", "pairs": 12, "rows": 8190, "vocab": 65537, "dtype": "f16",
         "average": True, "smoothing": 0.1, "masked": 0.2, "pad": 0},
        # one token through a 4096 x 14336 block: both weights are read once
        {"name": "glu_one_token", "op": "glu_forward", "tokens": 1, "hidden": 4096, "ffn": 14336, "dtype": "bf16",
         "act": "silu", "save": False},
        # a training micro-batch through the same block, pre-activations kept for the backward pass
        {"name": "glu_forward_8192", "op": "glu_forward", "tokens": 8192, "hidden": 4096, "ffn": 14336,
         "dtype": "bf16", "act": "silu", "save": True},
        # odd everything: token count, hidden size and feed-forward size off every tile and 16-byte boundary
        {"name": "glu_backward_odd", "op": "glu_backward", "tokens": 333, "hidden": 1001, "ffn": 2731,
         "dtype": "f16", "act": "gelu"},
        # backward of the 2048 x 8192 block
        {"name": "glu_backward_4096", "op": "glu_backward", "tokens": 4096, "hidden": 2048, "ffn": 8192,
         "dtype": "bf16", "act": "silu"},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm; half of them made odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v | 1 if rng.random() < 0.5 and v < hi else v


def draw(rng):
    op = rng.choice(["distill", "policy", "preference", "glu_forward", "glu_backward"])
    if op.startswith("glu"):
        case = {"op": op, "hidden": _log_int(rng, 32, 4096), "ffn": _log_int(rng, 32, 14336),
                "dtype": rng.choice(["bf16", "f16"]), "act": rng.choice(["silu", "gelu", "gelu_tanh"])}
        # a backward pass has twice the forward's products
        case["tokens"] = _log_int(rng, 1, 8192 if op == "glu_forward" else 4096)
        if op == "glu_forward":
            case["save"] = rng.random() < 0.5
        return case
    dtype = rng.choice(["bf16", "f16", "f32"])
    vocab = _log_int(rng, 1000, 200000)
    # preference reads the logits twice
    most = (8192 * 131072 * 2) // (vocab * ESIZE[dtype] * (2 if op == "preference" else 1))
    rows = _log_int(rng, 8 if op == "preference" else 1, min(8192, most))
    case = {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "masked": rng.choice([0.0, 0.1, 0.5]),
            "pad": rng.choice([0, 0, rng.randint(1, 60)])}
    if op == "distill":
        case.update(k=_log_int(rng, 1, 256), tail=rng.random() < 0.5, temperature=rng.choice([1.0, 1.5, 4.0]))
    elif op == "policy":
        case.update(temperature=rng.choice([1.0, 0.6]), kl=rng.choice([0.0, 0.001, 0.1]))
    else:
        case.update(pairs=rng.randint(1, max(1, min(32, rows // 8))), average=rng.random() < 0.5,
                    smoothing=rng.choice([0.0, 0.05]))
    return case


def work(case):
    if case["op"].startswith("glu"):
        t, d, f, e = case["tokens"], case["hidden"], case["ffn"], ESIZE[case["dtype"]]
        if case["op"] == "glu_forward":
            return {"bytes": e * (t * d + 2 * f * d + (3 if case["save"] else 1) * t * f), "flops": 4.0 * t * d * f}
        return {"bytes": e * (t * d + 2 * f * d + 3 * t * f + t * d + 2 * f * d), "flops": 8.0 * t * d * f}
    # every live row read once, every gradient row written once; small per-row vectors beside them
    row = case["vocab"] * ESIZE[case["dtype"]]
    small = 12.0 * case["k"] if case["op"] == "distill" else 28.0
    return {"bytes": case["rows"] * ((2.0 - case["masked"]) * row + small), "flops": 6.0 * case["rows"] * case["vocab"]}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _bounds(case):
    """Row offsets of the 2 x pairs sequences: ragged, the same for every seed."""
    n = 2 * case["pairs"]
    r = random.Random(case["rows"] * 64 + n)
    share = [r.uniform(0.3, 1.7) for _ in range(n)]
    total, at, out = sum(share), 0.0, [0]
    for s in share:
        at += s
        out.append(int(round(case["rows"] * at / total)))
    out[-1] = case["rows"]
    return out


def _row_losses_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rows, vocab, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    dev = {"device": "cuda", "generator": g}
    logits = torch.randn(rows, vocab, dtype=dt, **dev)
    logits.mul_(2.0)
    if case["pad"]:
        logits[:, vocab - case["pad"]:] = -math.inf      # padded columns of the head
    s = dict(case, logits=logits)
    live = vocab - case["pad"]
    keep = torch.rand(rows, **dev) >= case["masked"]
    if case["op"] == "distill":
        k = min(case["k"], live)
        start = torch.randint(0, live, (rows, 1), **dev)
        step = torch.randint(1, max(2, live // k + 1), (rows, 1), **dev)
        idx = (start + step * torch.arange(k, device="cuda")) % live          # distinct within a row
        t = 14.0 - 3.0 * torch.log1p(torch.arange(k, device="cuda").float()) + torch.randn(rows, k, **dev)
        t = torch.sort(t, dim=1, descending=True).values.to(dt)
        # a student that has learnt part of the teacher
        logits.scatter_(1, idx, (0.8 * t.float() + torch.randn(rows, k, **dev)).to(dt))
        s.update(idx=idx.to(torch.int32), teacher=t, lse=None)
        if case["tail"]:
            mass = 0.6 + 0.39 * torch.rand(rows, **dev)
            s["lse"] = torch.logsumexp(t.float() / case["temperature"], 1) - torch.log(mass)
    else:
        tok = torch.randint(0, live, (rows, 1), **dev)
        # sampled tokens are likely ones
        logits.scatter_add_(1, tok, (10.0 * torch.rand(rows, 1, **dev) + 2.0).to(dt))
        s["tokens"] = tok[:, 0]
    # mean over the live rows; fp16 gradients are loss-scaled to a weight of one
    w = 1.0 if case["dtype"] == "f16" else 1.0 / max(1, rows)
    s["weights"] = keep.float() * w
    if case["op"] == "policy":
        c = 1.0 / case["temperature"]
        logp = torch.empty(rows, device="cuda")
        for a in range(0, rows, 512):
            z = logits[a:a + 512].float() * c
            logp[a:a + 512] = z.gather(1, tok[a:a + 512])[:, 0] - torch.logsumexp(z, 1)
        # ratios around one, some of them beyond the clip range; none sits on its edge, where the
        # derivative jumps
        r = torch.exp(0.15 * torch.randn(rows, **dev))
        for edge in (0.8, 1.28):
            r = torch.where((r - edge).abs() < 2e-3, torch.full_like(r, edge + 4e-3), r)
        s["old"] = logp - torch.log(r)
        s["ref"] = logp + 0.3 * torch.randn(rows, **dev)
        s["adv"] = torch.randn(rows, **dev)
    if case["op"] == "preference":
        s["tokens"] = torch.where(keep, s["tokens"], torch.full_like(s["tokens"], -100))
        b = _bounds(case)
        s["bounds"] = torch.tensor(b, dtype=torch.int32, device="cuda")
        longest = max(y - x for x, y in zip(b, b[1:]))
        s["span"] = longest
        s["weights"] = torch.full((case["pairs"],), 1.0 if case["dtype"] == "f16" else 1.0 / case["pairs"],
                                  device="cuda")
        # the reference model's sequence values, a little off the policy's
        lp = torch.empty(rows, device="cuda")
        for a in range(0, rows, 512):
            z = logits[a:a + 512].float()
            lp[a:a + 512] = z.gather(1, tok[a:a + 512])[:, 0] - torch.logsumexp(z, 1)
        lp = lp * keep
        at = [float(lp[x:y].sum()) / (max(1, int(keep[x:y].sum())) if case["average"] else 1)
              for x, y in zip(b, b[1:])]
        spread = 0.05 if case["average"] else 5.0
        s["ref"] = torch.tensor(at, device="cuda") + spread * torch.randn(2 * case["pairs"], **dev)
        s["beta"] = 2.0 if case["average"] else 0.1
    return s


def prepare(case, seed):
    if not case["op"].startswith("glu"):
        return _row_losses_inputs(case, seed)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    t, d, f, dt = case["tokens"], case["hidden"], case["ffn"], DTYPES[case["dtype"]]

    def normal(*shape, std):
        return torch.randn(*shape, dtype=dt, device="cuda", generator=g).mul_(std)

    s = dict(case, x=normal(t, d, std=1.0), wg=normal(f, d, std=d ** -0.5), wu=normal(f, d, std=d ** -0.5))
    if case["op"] == "glu_backward":
        # what the forward pass kept (pre-activations of unit variance), and the incoming gradient
        s.update(gate=normal(t, f, std=1.0), up=normal(t, f, std=1.0), dh=normal(t, f, std=0.5))
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def _run_own(s):
    import newton_schulz_frobenius_gb300 as mg
    op = s["op"]
    if op == "distill":
        return mg.muon_distill_loss(s["logits"], s["idx"], s["teacher"], teacher_lse=s["lse"], weights=s["weights"],
                                    temperature=s["temperature"])
    if op == "policy":
        return mg.muon_policy_loss(s["logits"], s["tokens"], s["adv"], old_logp=s["old"], ref_logp=s["ref"],
                                   weights=s["weights"], temperature=s["temperature"], clip_low=CLIP_LOW,
                                   clip_high=CLIP_HIGH, kl_coef=s["kl"])
    if op == "preference":
        return mg.muon_preference_loss(s["logits"], s["tokens"], s["bounds"], ref_logp=s["ref"],
                                       weights=s["weights"], beta=s["beta"], label_smoothing=s["smoothing"],
                                       average=s["average"])
    if op == "glu_forward":
        return mg.muon_glu_forward(s["x"], s["wg"], s["wu"], act=s["act"], save=s["save"])
    return mg.muon_glu_backward(s["x"], s["wg"], s["wu"], s["gate"], s["up"], s["dh"], act=s["act"])


def _softmax_parts(z):
    """exp(z - max), its row sums, and max."""
    m = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - m)
    return e, e.sum(dim=1, keepdim=True), m


def _act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * g * g)


def _run_plain(s):
    op = s["op"]
    if op == "glu_forward":
        x = s["x"].float()
        gate, up = x @ s["wg"].float().t(), x @ s["wu"].float().t()
        h = _act(gate, s["act"])[0] * up
        dt = s["x"].dtype
        return (h.to(dt), gate.to(dt), up.to(dt)) if s["save"] else h.to(dt)
    if op == "glu_backward":
        x, dh, dt = s["x"].float(), s["dh"].float(), s["x"].dtype
        a, da = _act(s["gate"].float(), s["act"])
        dg, du = dh * s["up"].float() * da, dh * a
        dx = dg @ s["wg"].float() + du @ s["wu"].float()
        return dx.to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
    logits, w = s["logits"], s["weights"]
    if op == "distill":
        temp = s["temperature"]
        e, total, m = _softmax_parts(logits.float() / temp)
        idx = s["idx"].long()
        zt = s["teacher"].float() / temp
        if s["lse"] is None:
            pe, ps, pm = _softmax_parts(zt)
            p, logp = pe / ps, zt - pm - torch.log(ps)
        else:
            logp = zt - s["lse"][:, None]
            p = torch.exp(logp)
        mass = p.sum(dim=1, keepdim=True)
        zs = logits.gather(1, idx).float() / temp
        logq = zs - m - torch.log(total)
        kl = (p * (logp - logq)).sum(dim=1)
        if s["lse"] is None:
            grad = e * (mass / total)
            grad.scatter_add_(1, idx, -p)
        else:
            inside = torch.exp(zs - m) / total
            rest = 1.0 - mass[:, 0]
            rest = torch.where(rest > 0, rest, torch.zeros_like(rest))
            es = e.scatter(1, idx, 0.0).sum(dim=1)
            qrest = es / total[:, 0]
            ok = (rest > 0) & (qrest > 0)
            one = torch.ones_like(rest)
            kl = kl + torch.where(ok, rest * (torch.log(torch.where(ok, rest, one)) -
                                              torch.log(torch.where(ok, qrest, one))), torch.zeros_like(rest))
            rest = torch.where(ok, rest, torch.zeros_like(rest))
            full = mass + rest[:, None]
            grad = e * ((full[:, 0] - rest / torch.where(ok, qrest, one)) / total[:, 0])[:, None]
            grad.scatter_(1, idx, inside * full - p)
        live = w != 0
        loss = torch.where(live, w * temp * temp * kl, torch.zeros_like(w))
        grad = torch.where(live[:, None], grad * (w * temp)[:, None], torch.zeros_like(grad))
        return loss, grad.to(logits.dtype)
    c = 1.0 / s.get("temperature", 1.0)
    e, total, m = _softmax_parts(logits.float() * c)
    tok = s["tokens"][:, None].clamp(min=0)
    logp = (logits.gather(1, tok).float() * c - m - torch.log(total))[:, 0]
    if op == "policy":
        live = w != 0
        r = torch.exp(logp - s["old"])
        rc = torch.clamp(r, 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
        a = s["adv"]
        x = s["ref"] - logp
        ex = torch.exp(x)
        loss = -torch.minimum(r * a, rc * a) + s["kl"] * (ex - x - 1.0)
        dl = torch.where(r * a <= rc * a, -r * a, torch.zeros_like(r)) + s["kl"] * (1.0 - ex)
        zero = torch.zeros_like(w)
        loss, logp = torch.where(live, w * loss, zero), torch.where(live, logp, zero)
        coef = torch.where(live, w * dl * c, zero)
        grad = e * (-coef[:, None] / total)
        grad.scatter_add_(1, tok, coef[:, None])
        grad = torch.where(live[:, None], grad, torch.zeros_like(grad))
        return loss, logp, grad.to(logits.dtype)
    live = s["tokens"] >= 0
    logp = torch.where(live, logp, torch.zeros_like(logp))
    b = s["bounds"].long()
    at = b[:-1, None] + torch.arange(s["span"], device=b.device)
    inside = at < b[1:, None]
    at = torch.where(inside, at, torch.zeros_like(at))
    seq = torch.where(inside, logp[at], torch.zeros_like(logp[at])).sum(dim=1)
    n = (inside & live[at]).sum(dim=1).float()
    share = torch.where(n > 0, 1.0 / n.clamp(min=1.0), torch.zeros_like(n)) if s["average"] else torch.ones_like(n)
    seq = seq * share
    d = seq - s["ref"]
    h = s["beta"] * (d[0::2] - d[1::2])
    eps = s["smoothing"]
    soft = torch.clamp(-h, min=0) + torch.log1p(torch.exp(-torch.abs(h)))       # -log sigmoid(h)
    loss = w * ((1 - eps) * soft + eps * (soft + h))
    sig = 1.0 / (1.0 + torch.exp(-h))
    dh = w * (sig - (1 - eps))
    coef = torch.stack([dh, -dh], dim=1).reshape(-1) * s["beta"] * share
    which = (torch.arange(logp.numel(), device=b.device)[:, None] >= b[None, 1:-1]).sum(dim=1)
    coef = torch.where(live, coef[which], torch.zeros_like(logp))
    grad = e * (-coef[:, None] / total)
    grad.scatter_add_(1, tok, coef[:, None])
    return loss, seq, torch.where(live[:, None], grad, torch.zeros_like(grad)).to(logits.dtype)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------
# the same outputs in fp64, from the definitions
# ----------------------------------------------------------------------------

def _exact_glu(s):
    x, wg, wu = (s[k].double() for k in ("x", "wg", "wu"))
    if s["op"] == "glu_forward":
        gate, up = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
    else:
        gate, up = s["gate"].double(), s["up"].double()
    if s["act"] == "silu":
        sg = torch.sigmoid(gate)
        a, da = gate * sg, sg + gate * sg * torch.sigmoid(-gate)
    elif s["act"] == "gelu":
        phi = torch.exp(-gate ** 2 / 2) / (2 * math.pi) ** 0.5
        cdf = torch.erfc(-gate / 2 ** 0.5) / 2
        a, da = gate * cdf, cdf + gate * phi
    else:
        k = (2 / math.pi) ** 0.5
        u = k * gate * (1 + 0.044715 * gate ** 2)
        lo = torch.sigmoid(2 * u)                    # (1 + tanh u) / 2
        a, da = gate * lo, lo + gate * 2 * lo * torch.sigmoid(-2 * u) * k * (1 + 0.134145 * gate ** 2)
    if s["op"] == "glu_forward":
        h = a * up
        return (h, gate, up) if s["save"] else h
    dh = s["dh"].double()
    dg, du = dh * up * da, dh * a
    return dg @ wg + du @ wu, torch.einsum("tf,td->fd", dg, x), torch.einsum("tf,td->fd", du, x)


def _log_softmax64(s, rows):
    z = s["logits"][rows].double() / s.get("temperature", 1.0)
    return z - torch.logsumexp(z, dim=1, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("glu"):
        return _exact_glu(s)
    rows, vocab = case["rows"], case["vocab"]
    grad = torch.zeros(rows, vocab, dtype=torch.float64, device="cuda")
    chunks = [slice(a, min(rows, a + 256)) for a in range(0, rows, 256)]
    w = s["weights"].double()
    if case["op"] == "distill":
        temp = case["temperature"]
        loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
        for c in chunks:
            lq = _log_softmax64(s, c)
            n, idx = lq.shape[0], s["idx"][c].long()
            zt = s["teacher"][c].double() / temp
            lp = zt - (torch.logsumexp(zt, 1) if s["lse"] is None else s["lse"][c].double())[:, None]
            p = lp.exp()
            q = lq.exp()
            dense = torch.zeros_like(q).scatter_add_(1, idx, p)
            kl = (p * (lp - lq.gather(1, idx))).sum(1)
            if s["lse"] is None:
                g = q - dense
            else:
                out = torch.ones(n, vocab, dtype=torch.bool, device="cuda").scatter_(1, idx, False)
                rest = (1 - p.sum(1)).clamp(min=0)
                qr = (q * out).sum(1)
                ok = (rest > 0) & (qr > 0)
                kl = kl + torch.where(ok, rest * torch.log(rest.clamp(min=1e-300) / qr.clamp(min=1e-300)), 0.0)
                share = torch.where(ok, rest / qr.clamp(min=1e-300), 0.0)
                full = p.sum(1) + torch.where(ok, rest, 0.0)
                g = q * full[:, None] - dense - q * out * share[:, None]
            loss[c] = w[c] * temp ** 2 * kl
            grad[c] = torch.where(w[c][:, None] != 0, g * (w[c] * temp)[:, None], 0.0)
        return torch.where(w != 0, loss, 0.0), grad
    logp = torch.zeros(rows, dtype=torch.float64, device="cuda")
    tok = s["tokens"].clamp(min=0)[:, None]
    for c in chunks:
        logp[c] = _log_softmax64(s, c).gather(1, tok[c])[:, 0]
    if case["op"] == "policy":
        r = torch.exp(logp - s["old"].double())
        a, ref = s["adv"].double(), s["ref"].double()
        clipped = ((a > 0) & (r > 1 + CLIP_HIGH)) | ((a < 0) & (r < 1 - CLIP_LOW))
        bound = torch.where(a > 0, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW).double()
        loss = -a * torch.where(clipped, bound, r) + case["kl"] * (torch.expm1(ref - logp) - (ref - logp))
        coef = torch.where(clipped, 0.0, -a * r) - case["kl"] * torch.expm1(ref - logp)
        coef = coef * w / case["temperature"]
        loss, logp, coef = (torch.where(w != 0, v, 0.0) for v in (w * loss, logp, coef))
        first = (loss, logp)
    else:
        live = s["tokens"] >= 0
        b = _bounds(case)
        seq, coef = [], torch.zeros(rows, dtype=torch.float64, device="cuda")
        for x, y in zip(b, b[1:]):
            n = max(1, int(live[x:y].sum())) if case["average"] else 1
            seq.append((logp[x:y] * live[x:y]).sum() / n)
            coef[x:y] = live[x:y].double() / n
        seq = torch.stack(seq)
        d = seq - s["ref"].double()
        h = s["beta"] * (d[0::2] - d[1::2])
        eps = case["smoothing"]
        loss = -w * ((1 - eps) * torch.nn.functional.logsigmoid(h) + eps * torch.nn.functional.logsigmoid(-h))
        dh = w * (eps * torch.sigmoid(h) - (1 - eps) * torch.sigmoid(-h)) * s["beta"]
        for i in range(case["pairs"]):
            coef[b[2 * i]:b[2 * i + 1]] *= dh[i]
            coef[b[2 * i + 1]:b[2 * i + 2]] *= -dh[i]
        first = (loss, seq)
    for c in chunks:
        g = -_log_softmax64(s, c).exp() * coef[c][:, None]
        g.scatter_add_(1, tok[c], coef[c][:, None])
        grad[c] = torch.where(coef[c][:, None] != 0, g, 0.0)
    return first + (grad,)
