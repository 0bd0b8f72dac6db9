"""Cases that time the experts' operators and dropout, with their plain forms.

``run`` computes one pass: where ``own`` is false in elementary torch
operations on fp32 copies of the inputs, rounded once at the end; where it is
true through the library's entry points.  ``exact`` computes the same outputs
in fp64, written from the formulas.

Tokens go to experts as slots: slot t k + j is token t's j-th choice.  Sorted
rows are the slots in the order of their experts (equal experts in slot order),
``bounds`` the experts' ends; slots without an expert (dropped ones) come last.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}
PRODUCTS = ("glu_forward", "glu_backward", "linear_forward", "linear_backward")


def listed():
    return [
        # one short answer's tokens to 2 of 8 experts: latency counts
        {"name": "dispatch_few", "op": "dispatch", "tokens": 16, "k": 2, "experts": 8, "hidden": 4096, "dtype": "bf16",
         "dropped": 0.0},
        # a training micro-batch to 8 of 64 experts
        {"name": "dispatch_batch", "op": "dispatch", "tokens": 16384, "k": 8, "experts": 64, "hidden": 2048,
         "dtype": "bf16", "dropped": 0.0},
        # the way back of an odd batch whose experts had a capacity: dropped slots, rows off 16-byte boundaries
        {"name": "combine_odd", "op": "combine", "tokens": 2047, "k": 6, "experts": 160, "hidden": 1001, "dtype": "f32",
         "dropped": 0.1, "residual": True},
        # gradients of the way back for a micro-batch
        {"name": "combine_backward_batch", "op": "combine_backward", "tokens": 8192, "k": 8, "experts": 64,
         "hidden": 2048, "dtype": "bf16", "dropped": 0.0},
        # dropout of a few rows: latency counts
        {"name": "dropout_rows_16", "op": "dropout", "rows": 16, "cols": 4096, "dtype": "bf16", "p": 0.1,
         "residual": False},
        # odd rows in fp32, as a backward pass (no residual) sees them
        {"name": "dropout_odd_f32", "op": "dropout", "rows": 4097, "cols": 5003, "dtype": "f32", "p": 0.25,
         "residual": False},
        # a block's output joined to the residual stream
        {"name": "dropout_residual", "op": "dropout", "rows": 16384, "cols": 4096, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # a handful of tokens: the chosen experts' weights are read once
        {"name": "glu_forward_few", "op": "glu_forward", "tokens": 8, "k": 2, "experts": 8, "hidden": 2048, "ffn": 8192,
         "dtype": "bf16", "act": "silu", "save": False, "dropped": 0.0},
        # a micro-batch through 8 experts of 4096 x 14336, pre-activations kept for the backward pass
        {"name": "glu_forward_8", "op": "glu_forward", "tokens": 8192, "k": 2, "experts": 8, "hidden": 4096,
         "ffn": 14336, "dtype": "bf16", "act": "silu", "save": True, "dropped": 0.0},
        # backward through many small experts
        {"name": "glu_backward_64", "op": "glu_backward", "tokens": 4096, "k": 8, "experts": 64, "hidden": 2048,
         "ffn": 1024, "dtype": "bf16", "act": "silu", "dropped": 0.0},
        # the projection back, every size off its tile and off 16-byte boundaries
        {"name": "linear_forward_odd", "op": "linear_forward", "tokens": 1023, "k": 6, "experts": 20, "hidden": 1001,
         "ffn": 2731, "dtype": "f16", "dropped": 0.05},
        # backward of the 4096 x 14336 experts' projection back
        {"name": "linear_backward_8", "op": "linear_backward", "tokens": 8192, "k": 2, "experts": 8, "hidden": 4096,
         "ffn": 14336, "dtype": "bf16", "dropped": 0.0},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm; half of them made odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v | 1 if rng.random() < 0.5 and v < hi else v


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_backward", "dropout"] + list(PRODUCTS))
    if op == "dropout":
        cols = _log_int(rng, 1, 16384)
        return {"op": op, "rows": _log_int(rng, 1, min(16384, 16384 * 4096 // cols)), "cols": cols,
                "dtype": rng.choice(["bf16", "f16", "f32"]), "p": rng.choice([0.05, 0.1, 0.5]),
                "residual": rng.random() < 0.5}
    experts = _log_int(rng, 2, 256)
    k = rng.randint(1, min(8, experts))
    case = {"op": op, "k": k, "experts": experts, "dropped": rng.choice([0.0, 0.0, 0.1])}
    if op in PRODUCTS:
        case.update(hidden=_log_int(rng, 32, 4096), ffn=_log_int(rng, 32, 14336), dtype=rng.choice(["bf16", "f16"]))
        # the weights of all experts within the largest listed case's, the products too
        case["experts"] = experts = max(k, min(experts, 8 * 4096 * 14336 // (case["hidden"] * case["ffn"])))
        case["tokens"] = _log_int(rng, 1, 8192 if experts <= 8 else 4096)
        if op.startswith("glu"):
            case["act"] = rng.choice(["silu", "gelu", "gelu_tanh"])
        if op == "glu_forward":
            case["save"] = rng.random() < 0.5
        dense = case["tokens"] * k * case["hidden"] * case["ffn"] * (2 if op == "glu_backward" else 1)
        if dense > 16384 * 4096 * 14336:
            case["tokens"] = max(1, int(case["tokens"] * 16384 * 4096 * 14336 / dense))
        return case
    case.update(hidden=_log_int(rng, 16, 8192), dtype=rng.choice(["bf16", "f16", "f32"]))
    most = 8192 * 8 * 2048 * 2 // (case["hidden"] * k * ESIZE[case["dtype"]])
    case["tokens"] = _log_int(rng, 1, max(1, min(32768, most)))
    if op == "combine":
        case["residual"] = rng.random() < 0.5
    return case


def work(case):
    op, e = case["op"], ESIZE[case["dtype"]]
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": n * e * (3 if case["residual"] else 2), "flops": 2.0 * n}
    t, d, slots = case["tokens"], case["hidden"], case["tokens"] * case["k"]
    live = slots * (1.0 - case["dropped"])
    if op == "dispatch":
        return {"bytes": (t + slots) * d * e + 12.0 * slots, "flops": 0.0}
    if op == "combine":
        return {"bytes": (live + (2 if case["residual"] else 1) * t) * d * e + 8.0 * slots, "flops": 2.0 * live * d}
    if op == "combine_backward":
        return {"bytes": (t + live + slots) * d * e + 12.0 * slots, "flops": 3.0 * live * d}
    # experts that some token chose, in the mean of even choices: only their weights are read
    n, f = case["experts"], case["ffn"]
    hit = n * (1.0 - (1.0 - case["k"] / n) ** t)
    if op == "glu_forward":
        return {"bytes": e * (slots * d + 2 * hit * f * d + (3 if case["save"] else 1) * slots * f),
                "flops": 4.0 * live * d * f}
    if op == "glu_backward":
        return {"bytes": e * (slots * (2 * d + 3 * f) + 2 * (hit + n) * f * d),
                "flops": 8.0 * live * d * f}
    if op == "linear_forward":
        return {"bytes": e * (slots * (d + f) + hit * f * d), "flops": 2.0 * live * d * f}
    return {"bytes": e * (slots * (d + 2 * f) + (hit + n) * f * d), "flops": 4.0 * live * d * f}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, dtype=dt, device="cuda", generator=g).mul_(std)

    op, s = case["op"], dict(case)
    if op == "dropout":
        s["x"] = normal(case["rows"], case["cols"])
        s["add"] = normal(case["rows"], case["cols"]) if case["residual"] else None
        # (seed, offset) of the generator, as a program keeps them on the device
        s["state"] = torch.tensor([(int(seed) * 2654435761 + 12345) % (1 << 62), (1 << 32) + int(seed) % 1000],
                                  dtype=torch.int64, device="cuda")
        return s
    t, k, n, d = case["tokens"], case["k"], case["experts"], case["hidden"]
    # a router's choice: experts of different popularity, k different ones per token
    taste = 0.5 * torch.randn(1, n, device="cuda", generator=g)
    u = torch.rand(t, n, device="cuda", generator=g).clamp(1e-6, 1 - 1e-6)
    score, choice = torch.topk(taste - torch.log(-torch.log(u)), k, dim=1)
    if case["dropped"]:
        lost = torch.rand(t, k, device="cuda", generator=g) < case["dropped"]
        choice = torch.where(lost, torch.full_like(choice, -1), choice)
    s["choice"] = choice.to(torch.int32)
    if op == "dispatch":
        s["x"] = normal(t, d)
        return s
    s["row_of"], s["slot_of"], s["bounds"] = _sort(s["choice"], n)
    s["ends"] = s["bounds"].tolist()
    total = s["ends"][-1]
    if op in ("combine", "combine_backward"):
        e = torch.exp(score - score.max(dim=1, keepdim=True).values)
        s["weights"] = e / e.sum(dim=1, keepdim=True)
        s["ys"] = normal(t * k, d)
        s["ys"][total:] = 0.0
        s["add"] = normal(t, d) if case.get("residual") else None
        if op == "combine_backward":
            s["dy"] = normal(t, d, std=0.5)
        return s
    f, r = case["ffn"], t * k

    def rows(cols, std=1.0):
        v = normal(r, cols, std=std)
        v[total:] = 0.0
        return v

    if op.startswith("glu"):
        s.update(x=rows(d), wg=normal(n, f, d, std=d ** -0.5), wu=normal(n, f, d, std=d ** -0.5))
        if op == "glu_backward":
            # what the forward pass kept (pre-activations of unit variance), and the incoming gradient
            s.update(gate=rows(f), up=rows(f), dh=rows(f, 0.5))
    else:
        s.update(h=rows(f), w=normal(n, d, f, std=f ** -0.5))
        if op == "linear_backward":
            s["dy"] = rows(d, 0.5)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _run_own(s):
    import newton_schulz_frobenius_gb300 as mg
    op = s["op"]
    if op == "dispatch":
        row_of, slot_of, bounds = mg.muon_expert_sort(s["choice"], s["experts"])
        return mg.muon_expert_dispatch(s["x"], row_of, bounds), row_of, slot_of, bounds
    if op == "combine":
        return mg.muon_expert_combine(s["ys"], s["row_of"], s["bounds"], weights=s["weights"], residual=s["add"])
    if op == "combine_backward":
        return mg.muon_expert_combine_backward(s["dy"], s["ys"], s["row_of"], s["bounds"], s["weights"])
    if op == "dropout":
        return mg.muon_dropout(s["x"], s["p"], state=s["state"], residual=s["add"])
    if op == "glu_forward":
        return mg.muon_expert_glu_forward(s["x"], s["wg"], s["wu"], s["bounds"], act=s["act"], save=s["save"])
    if op == "glu_backward":
        return mg.muon_expert_glu_backward(s["x"], s["wg"], s["wu"], s["gate"], s["up"], s["dh"], s["bounds"],
                                           act=s["act"])
    if op == "linear_forward":
        return mg.muon_expert_linear_forward(s["h"], s["w"], s["bounds"])
    return mg.muon_expert_linear_backward(s["h"], s["w"], s["dy"], s["bounds"])


def _sort(choice, experts):
    """(row of each slot, slot of each row, experts' ends) in int32."""
    e = choice.reshape(-1)
    e = torch.where((e >= 0) & (e < experts), e, torch.full_like(e, experts))
    slot_of = torch.argsort(e, stable=True)
    row_of = torch.empty_like(slot_of)
    row_of[slot_of] = torch.arange(e.numel(), device=e.device)
    each = torch.zeros(experts + 2, dtype=torch.int64, device=e.device)
    each.index_add_(0, e.long() + 1, torch.ones_like(slot_of))
    return row_of.view(choice.shape).int(), slot_of.int(), torch.cumsum(each, 0)[:-1].int()


PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)


def _mul32(a, m):
    """High and low words of the product of 32-bit a (in int64) and m."""
    lo = (a & 0xFFFF) * m
    hi = (a >> 16) * m + (lo >> 16)
    return hi >> 16, ((hi & 0xFFFF) << 16) | (lo & 0xFFFF)


def _drop(n, state):
    """16 random bits for each of n elements: Philox4x32-10, eight elements to a counter."""
    m32 = 0xFFFFFFFF
    b = torch.arange((n + 7) // 8, dtype=torch.int64, device=state.device)
    key = [state[0] & m32, (state[0] >> 32) & m32]
    c = [b & m32, b >> 32, (state[1] & m32).expand_as(b), ((state[1] >> 32) & m32).expand_as(b)]
    for _ in range(10):
        h0, l0 = _mul32(c[0], PHILOX_M[0])
        h1, l1 = _mul32(c[2], PHILOX_M[1])
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + PHILOX_W[0]) & m32, (key[1] + PHILOX_W[1]) & m32]
    half = [v for w in c for v in (w & 0xFFFF, w >> 16)]
    return torch.stack(half, dim=1).reshape(-1)[:n]


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
    if op == "dropout":
        x = s["x"]
        cut = int(math.floor(s["p"] * 65536 + 0.5))
        keep = (_drop(x.numel(), s["state"]) >= cut).view(x.shape)
        y = torch.where(keep, x.float() * (65536.0 / (65536 - cut)), torch.zeros((), device=x.device))
        return (y if s["add"] is None else s["add"].float() + y).to(x.dtype)
    if op == "dispatch":
        row_of, slot_of, bounds = _sort(s["choice"], s["experts"])
        xs = s["x"][slot_of.long() // s["k"]]
        live = torch.arange(slot_of.numel(), device=xs.device) < bounds[-1]
        return torch.where(live[:, None], xs, torch.zeros_like(xs)), row_of, slot_of, bounds
    if op in ("combine", "combine_backward"):
        at = s["row_of"].long()
        live = (s["row_of"] < s["bounds"][-1])[:, :, None]
        part = s["ys"][at].float()
        part = torch.where(live, part, torch.zeros_like(part))
        w = s["weights"][:, :, None]
        if op == "combine":
            y = (part * w).sum(dim=1)
            return (y if s["add"] is None else y + s["add"].float()).to(s["ys"].dtype)
        dy = s["dy"].float()[:, None, :]
        dw = (part * dy).sum(dim=2)
        dslot = torch.where(live, dy * w, torch.zeros_like(part)).to(s["ys"].dtype)
        dys = torch.empty_like(s["ys"])
        dys[at.reshape(-1)] = dslot.reshape(-1, dslot.shape[2])
        return dys, dw
    # the experts' products, one expert after the other
    ends = s["ends"]
    first = s["x"] if op.startswith("glu") else s["h"]
    dt, n, d, f = first.dtype, s["experts"], s["hidden"], s["ffn"]

    def zeros(*shape):
        return torch.zeros(*shape, dtype=dt, device=first.device)

    r = first.shape[0]
    if op == "glu_forward":
        out = [zeros(r, f) for _ in range(3 if s["save"] else 1)]
    elif op == "glu_backward":
        out = [zeros(r, d), zeros(n, f, d), zeros(n, f, d)]
    elif op == "linear_forward":
        out = [zeros(r, d)]
    else:
        out = [zeros(r, f), zeros(n, d, f)]
    for e in range(n):
        c = slice(ends[e], ends[e + 1])
        if c.start == c.stop:
            continue
        if op == "glu_forward":
            x = s["x"][c].float()
            gate, up = x @ s["wg"][e].float().t(), x @ s["wu"][e].float().t()
            got = (_act(gate, s["act"])[0] * up, gate, up)
            for o, v in zip(out, got):
                o[c] = v.to(dt)
        elif op == "glu_backward":
            x, dh = s["x"][c].float(), s["dh"][c].float()
            a, da = _act(s["gate"][c].float(), s["act"])
            dg, du = dh * s["up"][c].float() * da, dh * a
            out[0][c] = (dg @ s["wg"][e].float() + du @ s["wu"][e].float()).to(dt)
            out[1][e], out[2][e] = (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
        elif op == "linear_forward":
            out[0][c] = (s["h"][c].float() @ s["w"][e].float().t()).to(dt)
        else:
            dy = s["dy"][c].float()
            out[0][c] = (dy @ s["w"][e].float()).to(dt)
            out[1][e] = (dy.t() @ s["h"][c].float()).to(dt)
    return out[0] if len(out) == 1 else tuple(out)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------
# the same outputs in fp64, from the definitions
# ----------------------------------------------------------------------------

def _exact_dropout(s):
    n = s["x"].numel()
    seed, offset = (int(v) & 0xFFFFFFFFFFFFFFFF for v in s["state"].tolist())
    block = np.arange((n + 7) // 8, dtype=np.uint64)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    a, b = block & low, block >> half
    c = np.full_like(block, offset & 0xFFFFFFFF)
    d = np.full_like(block, offset >> 32)
    for i in range(10):
        p, q = a * np.uint64(PHILOX_M[0]), c * np.uint64(PHILOX_M[1])
        k0 = np.uint64(((seed & 0xFFFFFFFF) + i * PHILOX_W[0]) & 0xFFFFFFFF)
        k1 = np.uint64(((seed >> 32) + i * PHILOX_W[1]) & 0xFFFFFFFF)
        a, b, c, d = (q >> half) ^ b ^ k0, q & low, (p >> half) ^ d ^ k1, p & low
    words = np.stack([a, b, c, d], axis=1).astype("<u4")
    bits = torch.from_numpy(words.view("<u2").astype(np.int32).reshape(-1)[:n]).to("cuda").view(s["x"].shape)
    cut = round(s["p"] * 65536)
    y = torch.where(bits >= cut, s["x"].double() / (1 - cut / 65536), 0.0)
    return y if s["add"] is None else y + s["add"].double()


def _act64(gate, kind):
    if kind == "silu":
        sg = torch.sigmoid(gate)
        return gate * sg, sg + gate * sg * torch.sigmoid(-gate)
    if kind == "gelu":
        cdf = torch.erfc(-gate / 2 ** 0.5) / 2
        return gate * cdf, cdf + gate * torch.exp(-gate ** 2 / 2) / (2 * math.pi) ** 0.5
    k = (2 / math.pi) ** 0.5
    u = k * gate * (1 + 0.044715 * gate ** 2)
    lo = torch.sigmoid(2 * u)                    # (1 + tanh u) / 2
    return gate * lo, lo + gate * 2 * lo * torch.sigmoid(-2 * u) * k * (1 + 0.134145 * gate ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        return _exact_dropout(s)
    k, n = case["k"], case["experts"]
    if op == "dispatch":
        # counted on the host, slot by slot
        each = [[] for _ in range(n + 1)]
        for i, e in enumerate(s["choice"].reshape(-1).tolist()):
            each[e if 0 <= e < n else n].append(i)
        order = [i for group in each for i in group]
        ends = np.cumsum([0] + [len(group) for group in each[:n]]).tolist()
        slot_of = torch.tensor(order, device="cuda")
        row_of = torch.zeros_like(slot_of)
        row_of[slot_of] = torch.arange(len(order), device="cuda")
        xs = s["x"].double()[slot_of // k]
        xs[ends[-1]:] = 0.0
        bounds = torch.tensor(ends, dtype=torch.int32, device="cuda")
        return xs, row_of.view(-1, k).int(), slot_of.int(), bounds
    total = s["ends"][-1]
    if op in ("combine", "combine_backward"):
        ys, w = s["ys"].double(), s["weights"].double()
        t, d = case["tokens"], case["hidden"]
        y = torch.zeros(t, d, dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()
        dys, dw = torch.zeros_like(ys), torch.zeros_like(w)
        for j in range(k):
            row = s["row_of"][:, j].long()
            on = torch.nonzero(row < total)[:, 0]
            y[on] += w[on, j, None] * ys[row[on]]
            if op == "combine_backward":
                dy = s["dy"].double()[on]
                dys[row[on]] = w[on, j, None] * dy
                dw[on, j] = torch.einsum("td,td->t", dy, ys[row[on]])
        return y if op == "combine" else (dys, dw)
    r, d, f = case["tokens"] * k, case["hidden"], case["ffn"]
    out = []
    for e, (b, c) in enumerate(zip(s["ends"], s["ends"][1:])):
        if op.startswith("glu"):
            x, wg, wu = s["x"][b:c].double(), s["wg"][e].double(), s["wu"][e].double()
            if op == "glu_forward":
                gate, up = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
                h = _act64(gate, case["act"])[0] * up
                out.append((h, gate, up) if case["save"] else (h,))
                continue
            a, da = _act64(s["gate"][b:c].double(), case["act"])
            dh = s["dh"][b:c].double()
            dg, du = dh * s["up"][b:c].double() * da, dh * a
            out.append((dg @ wg + du @ wu, torch.einsum("tf,td->fd", dg, x), torch.einsum("tf,td->fd", du, x)))
        else:
            h, w = s["h"][b:c].double(), s["w"][e].double()
            if op == "linear_forward":
                out.append((torch.einsum("tf,df->td", h, w),))
            else:
                dy = s["dy"][b:c].double()
                out.append((dy @ w, torch.einsum("td,tf->df", dy, h)))
    cols = list(zip(*out))
    whole = []
    for i, parts in enumerate(cols):
        if op.endswith("forward") or i == 0:
            v = torch.cat(parts)
            whole.append(torch.cat([v, torch.zeros(r - total, v.shape[1], dtype=v.dtype, device="cuda")]))
        else:
            whole.append(torch.stack(parts))
    return whole[0] if len(whole) == 1 else tuple(whole)
