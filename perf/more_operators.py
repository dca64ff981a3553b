"""Workloads of the router's scored selection and of the 4-bit weights: the
choice of experts from logits (softmax or sigmoid scores, a bias for balance,
groups, top-k, renormalised weights) and its gradient, the quantisation of
weights to 4 bits with group scales and the way back, the product of a few
rows with such weights, and the experts' products with them.

``listed()`` names the cases, ``draw`` makes more of the same ranges,
``prepare`` makes a case's inputs, ``run`` computes one pass: in plain torch
operations, or (``own``) through the library. ``exact`` gives the results in
64 bits and ``work`` the bytes and operations a pass cannot do without.
"""
from __future__ import annotations

import math

import torch

own = False

BF16 = torch.bfloat16
NEG_INF = float("-inf")


# ------------------------------------------------------------------ cases --
def _select(name, op, T, E, k, score, **kw):
    c = {"name": name, "op": op, "T": T, "E": E, "k": k, "score": score, "groups": 1,
         "topk_groups": 1, "group_rank": 2, "renormalise": True, "scale": 1.0, "balance": False}
    c.update(kw)
    return c


def _weights(name, op, E, K, N, kind, group, **kw):
    c = {"name": name, "op": op, "E": E, "K": K, "N": N, "kind": kind, "group": group}
    c.update(kw)
    return c


def _experts(name, T, d, f, E, k, kind, group, **kw):
    c = {"name": name, "op": "experts", "T": T, "d": d, "f": f, "E": E, "k": k, "S": 0,
         "kind": kind, "group": group, "clamped": False}
    c.update(kw)
    return c


def listed():
    out = []
    # one token's choice while decoding: nothing but latency
    out.append(_select("select_one", "select", 1, 256, 8, "sigmoid", groups=8, topk_groups=4,
                       scale=2.5, balance=True))
    # a training batch of 4 x 4096 tokens, experts in groups, a bias for balance
    out.append(_select("select_groups", "select", 16384, 256, 8, "sigmoid", groups=8,
                       topk_groups=4, scale=2.5, balance=True))
    # many small experts, plain softmax scores with a bias for balance, kept unnormalised
    out.append(_select("select_softmax", "select", 8192, 512, 10, "softmax", renormalise=False,
                       balance=True))
    # the gradients of the two batches: of sigmoid scores, which touches the chosen experts
    # alone, and of unnormalised softmax scores, which touches every expert
    out.append(_select("select_groups_bwd", "select_bwd", 16384, 256, 8, "sigmoid", groups=8,
                       topk_groups=4, scale=2.5, balance=True))
    out.append(_select("select_softmax_bwd", "select_bwd", 8192, 512, 10, "softmax",
                       renormalise=False, balance=True))
    # a checkpoint's experts on their way into 4 bits and back: a layer's down projections,
    # and one matrix of odd sizes
    out.append(_weights("quantise_layer", "quantise", 32, 2880, 2880, "fp4", 32))
    out.append(_weights("quantise_odd", "quantise", 1, 1096, 648, "int4", 64))
    # the projection in front of attention, for one token and for a batch of drafts
    out.append(_weights("linear_one", "linear", 1, 2880, 5120, "fp4", 32, T=1))
    out.append(_weights("linear_batch", "linear", 1, 4096, 2880, "int4", 128, T=40))
    # one user's next token through many small experts
    out.append(_experts("experts_one", 1, 2048, 768, 128, 8, "int4", 64))
    # a serving batch of single tokens: every expert read, a few rows each
    out.append(_experts("experts_batch", 64, 2880, 2880, 32, 4, "fp4", 32, clamped=True))
    # a chunk of prompts, a shared expert beside the routed ones
    out.append(_experts("experts_chunk", 2048, 2048, 768, 128, 8, "int4", 32, S=1))
    return out


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top_flops = max(work(c)["flops"] for c in listed())
    top_bytes = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["select", "select", "select_bwd", "quantise", "linear", "linear",
                         "experts", "experts", "experts"])
        kind, group = rng.choice(["int4", "fp4"]), rng.choice([32, 64, 128])
        if op in ("select", "select_bwd"):
            E = rng.choice([8, 20, 32, 60, 64, 128, 160, 256, 384, 512, 1024])
            groups = rng.choice([1, 1] + [n for n in (2, 4, 5, 8, 16) if E % n == 0 and E // n >= 2])
            tg = rng.randint(1, groups)
            k = min(rng.choice([1, 2, 4, 6, 8, 10, 16, 32]), tg * (E // groups))
            c = _select("", op, _log_int(rng, 1, 16384), E, k, rng.choice(["softmax", "sigmoid"]),
                        groups=groups, topk_groups=tg, group_rank=rng.choice([1, 2]),
                        renormalise=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                        balance=rng.random() < 0.6)
        elif op == "quantise":
            c = _weights("", op, _log_int(rng, 1, 32), 8 * _log_int(rng, 4, 512),
                         8 * _log_int(rng, 4, 512), kind, group)
        elif op == "linear":
            c = _weights("", op, 1, 8 * _log_int(rng, 16, 1024), 8 * _log_int(rng, 16, 1024), kind,
                         group, T=_log_int(rng, 1, 2048))
        else:
            d, f, E, k = rng.choice([(2048, 768, 128, 8), (2880, 2880, 32, 4), (2560, 640, 512, 10),
                                     (1024, 512, 64, 6), (520, 392, 8, 3), (1288, 1000, 20, 2)])
            c = _experts("", _log_int(rng, 1, 2048), d, f, E, k, kind, group,
                         S=rng.choice([0, 0, 1, 2]), clamped=rng.random() < 0.4)
        del c["name"]
        w = work(c)
        if w["flops"] <= top_flops and w["bytes"] <= top_bytes:
            return c


# ------------------------------------------------------------------ inputs --
# kind -> the values of the codes 0 .. 15: two's complement, or sign, two bits of
# exponent, one of mantissa
VALUES = {"int4": [0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1],
          "fp4": [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]}
ACT = (7.0, 1.702, 1.0)      # limit, alpha, offset of the clamped activation


def _group_max(w, group):
    """The largest magnitude of every group of rows: [E, ceil(K / group), N]."""
    E, K, N = w.shape
    pad = -K % group
    a = torch.nn.functional.pad(w.abs(), (0, 0, 0, pad))
    return a.view(E, (K + pad) // group, group, N).amax(2)


def _scales(amax, kind):
    """A group's scale from its largest magnitude, in 32 bits. int4: a seventh, its
    significand rounded up to five bits; fp4: the least power of two that keeps the
    group within 6. Either times a code is a bf16 value."""
    if kind == "int4":
        # (by a tensor: a division by a number is a product with its rounded inverse)
        bits = (amax / torch.full_like(amax, 7.0)).view(torch.int32)
        s = ((bits + 0x7FFFF) & ~0x7FFFF).view(torch.float32)
    else:
        m = torch.frexp(amax).mantissa                # amax = m 2^e, m in [1/2, 1)
        s = amax / m * torch.where(m > 0.75, 0.25, 0.125)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _quantise(w, kind, group):
    """(codes uint8 [E, K, N], scales bf16 [E, groups, N]) of weights [E, K, N]: the
    code of the nearest value, halves to the even code."""
    s = _scales(_group_max(w.float(), group), kind)
    per_row = s.repeat_interleave(group, 1)[:, :w.shape[1]]
    q = torch.where(per_row > 0, w.float() / per_row, torch.zeros_like(per_row))
    if kind == "int4":
        return (q.round().to(torch.int8) & 15).to(torch.uint8), s.to(BF16)
    a = q.abs()
    # steps of 1/2 up to 2, of 1 up to 4, of 2 beyond; the codes count the steps
    n = torch.where(a < 2, (2 * a).round(), torch.where(a < 4, a.round() + 2, (a / 2).round() + 4))
    return (n.to(torch.uint8) | (torch.signbit(q) & (n > 0)).to(torch.uint8) << 3), s.to(BF16)


def _codes(E, K, N, kind, group, gen):
    """A weight matrix in hand as codes and scales: N(0, 1/sqrt(K)) weights."""
    dev = gen.device
    codes = torch.empty(E, K, N, dtype=torch.uint8, device=dev)
    scales = torch.empty(E, -(-K // group), N, dtype=BF16, device=dev)
    for e in range(E):
        w = (torch.randn(1, K, N, generator=gen, device=dev) / math.sqrt(K)).to(BF16)
        codes[e:e + 1], scales[e:e + 1] = _quantise(w, kind, group)
    return codes, scales


def prepare(case, seed):
    """Inputs on the GPU: logits and upstream gradients, weights, or codes and
    scales with the rows they are applied to and the routing of those; with ``own``
    also the library's objects."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("select", "select_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        # experts that differ in how often they are wanted, and a bias that makes up for part of it
        lean = torch.randn(E, generator=gen, device=dev)
        st["logits"] = 1.5 * torch.randn(T, E, generator=gen, device=dev) + lean
        st["balance"] = -0.1 * lean * (1.0 if case["score"] == "sigmoid" else 4.0 / E)
        st["balance"] = st["balance"] if case["balance"] else None
        if op == "select_bwd":
            st["dw"] = torch.randn(T, k, generator=gen, device=dev)
            st["idx"] = _plain_choice(st)
    elif op == "quantise":
        E, K, N = case["E"], case["K"], case["N"]
        # columns of different size, as trained weights have them
        size = torch.exp(0.5 * torch.randn(E, 1, N, generator=gen, device=dev)) / math.sqrt(K)
        st["w"] = torch.randn(E, K, N, generator=gen, device=dev).mul_(size).to(BF16)
    elif op == "linear":
        st["codes"], st["scales"] = _codes(1, case["K"], case["N"], case["kind"], case["group"], gen)
        st["x"] = torch.randn(case["T"], case["K"], generator=gen, device=dev).to(BF16)
    else:
        T, d, f, E, k, S = (case[n] for n in ("T", "d", "f", "E", "k", "S"))
        for name, (K, N) in (("gate", (d, f)), ("up", (d, f)), ("down", (f, d))):
            st[name] = _codes(E + S, K, N, case["kind"], case["group"], gen)
        st["x"] = torch.randn(T, d, generator=gen, device=dev).to(BF16)
        logits = torch.randn(T, E, generator=gen, device=dev)
        logits += 0.5 * torch.randn(E, generator=gen, device=dev)
        top = torch.topk(logits, k, dim=1)
        st["idx"] = top.indices.to(torch.int32)
        st["w"] = torch.softmax(top.values, dim=1)
    if own:
        from mixture_experts_routed_softmax_gb300 import router, w4
        if op in ("select", "select_bwd"):
            st["router"] = router.Router(
                E, k, score=case["score"], n_groups=case["groups"], topk_groups=case["topk_groups"],
                group_rank=case["group_rank"], renormalise=case["renormalise"],
                scale=case["scale"], balance=st["balance"])
            st["buf"] = st["router"].buffers(T, backward=op == "select_bwd")
            if op == "select_bwd":
                st["buf"].topk_idx.copy_(st["idx"])
        elif op == "quantise":
            st["w4"] = w4.Weights4.empty(E, K, N, kind=case["kind"], group=case["group"])
            st["values"] = torch.empty_like(st["w"])
        elif op == "linear":
            st["layer"] = w4.Linear4(w4.Weights4.from_codes(
                st["codes"], st["scales"], kind=case["kind"], group=case["group"]))
            st["buf"] = st["layer"].buffers(case["T"])
        else:
            st["layer"] = w4.Experts4(
                *(w4.Weights4.from_codes(*st[n], kind=case["kind"], group=case["group"])
                  for n in ("gate", "up", "down")), k=k, E=E, act=ACT if case["clamped"] else None)
            st["buf"] = st["layer"].buffers(T)
    return st


# --------------------------------------------------------------- plain form --
def _plain_scores(st):
    """Scores in 64 bits: what lies next to a border decides which expert is taken."""
    l = st["logits"].double()
    if st["case"]["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    p = torch.exp(l - l.amax(1, keepdim=True))
    return p / p.sum(1, keepdim=True)


def _plain_choice(st):
    case = st["case"]
    T, E, n = case["T"], case["E"], case["groups"]
    c = _plain_scores(st)
    if st["balance"] is not None:
        c = c + st["balance"].double()
    if n > 1:
        best = torch.sort(c.view(T, n, E // n), dim=2, descending=True).values
        rank = best[:, :, :case["group_rank"]].sum(2)
        kept = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        drop = torch.ones(T, n, dtype=torch.bool, device=c.device).scatter_(1, kept, False)
        c = c.masked_fill(drop.repeat_interleave(E // n, 1), NEG_INF)
    return torch.sort(c, dim=1, descending=True, stable=True).indices[:, :case["k"]].to(torch.int32)


def _plain_select(st):
    case = st["case"]
    idx = _plain_choice(st)
    s = _plain_scores(st).gather(1, idx.long())
    w = s / s.sum(1, keepdim=True) if case["renormalise"] else s
    return {"idx": idx, "w": (w * case["scale"]).float()}


def _plain_select_bwd(st):
    """The chain rule from the weights to the scores to the logits."""
    case = st["case"]
    idx, g = st["idx"].long(), st["dw"].double() * case["scale"]
    p = _plain_scores(st)
    s = p.gather(1, idx)
    if case["renormalise"]:
        total = s.sum(1, keepdim=True)
        g = (g - (g * s).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(p).scatter_(1, idx, g)
    if case["score"] == "sigmoid":
        return {"d_logits": (ds * p * (1.0 - p)).float()}
    return {"d_logits": (p * (ds - (ds * p).sum(1, keepdim=True))).float()}


def _plain_values(codes, scales, case, values):
    """The weights that codes [.., K, N] and scales stand for, in 32 bits."""
    per_row = scales.float().repeat_interleave(case["group"], -2)[..., :codes.shape[-2], :]
    return values[codes.long()] * per_row


def _table(case, dev):
    return torch.tensor(VALUES[case["kind"]], dtype=torch.float32, device=dev)


def _plain_act(case, G, U):
    if not case["clamped"]:
        return G / (1.0 + torch.exp(-G)) * U
    limit, alpha, offset = ACT
    G = G.clamp(max=limit)
    return G / (1.0 + torch.exp(-alpha * G)) * (U.clamp(-limit, limit) + offset)


def _plain_experts(st):
    """Every expert's rows side by side, padded to the longest expert's."""
    case = st["case"]
    T, E, k, S, d = (case[n] for n in ("T", "E", "k", "S", "d"))
    dev = st["x"].device
    values = _table(case, dev)
    pair_e = torch.cat([st["idx"].long().reshape(-1),
                        torch.arange(E, E + S, device=dev).repeat_interleave(T)])
    pair_t = torch.cat([torch.arange(T, device=dev).repeat_interleave(k),
                        torch.arange(T, device=dev).repeat(S)])
    pair_w = torch.cat([st["w"].reshape(-1), torch.ones(S * T, device=dev)])
    order = torch.argsort(pair_e, stable=True)
    used, slot, counts = torch.unique(pair_e[order], return_inverse=True, return_counts=True)
    first = torch.cumsum(counts, 0) - counts
    at = torch.arange(order.numel(), device=dev) - first[slot]
    rows = torch.zeros(used.numel(), int(counts.max()), d, device=dev)
    rows[slot, at] = st["x"].float()[pair_t[order]]
    G, U = (torch.bmm(rows, _plain_values(c[used], s[used], case, values))
            for c, s in (st["gate"], st["up"]))
    c, s = st["down"]
    Y = torch.bmm(_plain_act(case, G, U), _plain_values(c[used], s[used], case, values))
    parts = torch.zeros(order.numel(), d, device=dev)
    parts[order] = Y[slot, at] * pair_w[order, None]
    y = parts[:T * k].view(T, k, d).sum(1) + parts[T * k:].view(S, T, d).sum(0)
    return {"y": y.to(BF16)}


def run(state):
    """One pass through the case's operator and its outputs."""
    st, op = state, state["case"]["op"]
    if own:
        if op == "select":
            st["router"].select(st["logits"], st["buf"])
            return {"idx": st["buf"].topk_idx, "w": st["buf"].topk_w}
        if op == "select_bwd":
            return {"d_logits": st["router"].select_bwd(st["dw"], st["logits"], st["buf"])}
        if op == "quantise":
            st["w4"].quantise_from(st["w"])
            return {"values": st["w4"].dequantise(st["values"])}
        if op == "linear":
            return {"y": st["layer"].apply(st["x"], st["buf"])}
        return {"y": st["layer"].forward(st["x"], st["idx"], st["w"], st["buf"])}
    if op == "select":
        return _plain_select(st)
    if op == "select_bwd":
        return _plain_select_bwd(st)
    case = st["case"]
    if op == "quantise":
        codes, scales = _quantise(st["w"], case["kind"], case["group"])
        return {"values": _plain_values(codes, scales, case, _table(case, codes.device)).to(BF16)}
    if op == "linear":
        W = _plain_values(st["codes"][0], st["scales"][0], case, _table(case, st["x"].device))
        return {"y": (st["x"].float() @ W).to(BF16)}
    return _plain_experts(st)


# ---------------------------------------------------------------- 64 bits --
def _decoded(codes, scales, kind, group):
    """Weights [K, N] in 64 bits, from the codes' bits."""
    c = codes.long()
    if kind == "int4":
        v = (c - 16 * (c >= 8)).double()
    else:
        e, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e > 0, (1 + m / 2) * (1 << e) / 2, m / 2)
        v = torch.where(c >= 8, -v, v)
    rows = torch.arange(c.shape[0], device=c.device) // group
    return v * scales.double()[rows]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("select", "select_bwd"):
        l = st["logits"].double()
        log_s = (torch.nn.functional.logsigmoid(l) if case["score"] == "sigmoid"
                 else torch.log_softmax(l, 1))
    if op == "select":
        chosen = log_s.gather(1, _plain_choice(st).long())
        if case["renormalise"]:
            chosen = chosen - torch.logsumexp(chosen, 1, keepdim=True)
        return {"idx": None, "w": case["scale"] * torch.exp(chosen)}
    if op == "select_bwd":
        # the gradient through the logarithms of the scores
        idx, dw = st["idx"].long(), st["dw"].double()
        chosen = log_s.gather(1, idx)
        if case["renormalise"]:
            chosen = chosen - torch.logsumexp(chosen, 1, keepdim=True)
        h = dw * case["scale"] * torch.exp(chosen)               # to the weight's logarithm
        if case["renormalise"]:
            h = h - torch.exp(chosen) * h.sum(1, keepdim=True)   # to the score's logarithm
        out = torch.zeros_like(l)
        rows = torch.arange(case["T"], device=l.device)
        for j in range(case["k"]):
            out[rows, idx[:, j]] += h[:, j]
        if case["score"] == "sigmoid":
            out = out * torch.exp(torch.nn.functional.logsigmoid(-l))
        else:
            out = out - torch.exp(log_s) * h.sum(1, keepdim=True)
        return {"d_logits": out}
    if op == "quantise":
        out = torch.empty(st["w"].shape, dtype=torch.float64, device=st["w"].device)
        grid = torch.tensor(sorted(set(abs(v) for v in VALUES[case["kind"]] if v != -8)),
                            dtype=torch.float64, device=out.device)
        # borders between neighbouring magnitudes; a value on one goes to the even code
        mid, even = (grid[1:] + grid[:-1]) / 2, torch.arange(1, len(grid), device=out.device) % 2
        for e in range(case["E"]):
            for r in range(0, case["K"], case["group"]):
                w = st["w"][e, r:r + case["group"]].double()
                top = w.abs().amax(0)
                if case["kind"] == "int4":
                    # top <= 7 lead n for the least whole n of five bits
                    lead = top / torch.frexp(top).mantissa / 256
                    n = torch.ceil(top / (7 * lead))
                    s = lead * torch.where(n > 32, 2 * torch.ceil(top / (14 * lead)), n)
                else:
                    s = top / torch.frexp(top).mantissa / 8
                    s = torch.where(top > 6 * s, 2 * s, s)
                a = torch.where(top > 0, w.abs() / s, torch.zeros_like(w))
                n = torch.zeros_like(a, dtype=torch.long)
                for b in range(len(mid)):
                    n += (a > mid[b]) | ((a == mid[b]) & (even[b] == 0))
                out[e, r:r + case["group"]] = torch.where(top > 0, torch.sign(w) * grid[n] * s,
                                                          torch.zeros_like(w))
        return {"values": out}
    if op == "linear":
        W = _decoded(st["codes"][0], st["scales"][0], case["kind"], case["group"])
        return {"y": st["x"].double() @ W}
    # expert by expert
    E, k, S = case["E"], case["k"], case["S"]
    x, y = st["x"].double(), torch.zeros(case["T"], case["d"], dtype=torch.float64, device=st["x"].device)
    idx = st["idx"].cpu()
    for e in range(E + S):
        if e < E:
            t, j = (v.to(x.device) for v in torch.nonzero(idx == e, as_tuple=True))
            w = st["w"].double()[t, j]
        else:
            t = torch.arange(case["T"], device=x.device)
            w = torch.ones(case["T"], dtype=torch.float64, device=x.device)
        if t.numel():
            W = [_decoded(st[n][0][e], st[n][1][e], case["kind"], case["group"])
                 for n in ("gate", "up", "down")]
            G, U = x[t] @ W[0], x[t] @ W[1]
            if case["clamped"]:
                G, U = torch.clamp(G, max=ACT[0]), torch.clamp(U, -ACT[0], ACT[0]) + ACT[2]
            A = G * torch.sigmoid((ACT[1] if case["clamped"] else 1.0) * G) * U
            y.index_add_(0, t, (A @ W[2]) * w[:, None])
    return {"y": y}


def work(case):
    op = case["op"]
    if op in ("select", "select_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        dense = case["score"] == "softmax" and not case["renormalise"]
        if op == "select":
            return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["balance"] else 0),
                    "flops": 4 * T * E}
        # only the chosen experts' logits are needed where the others' gradients are zero
        return {"bytes": 4 * T * E * (2 if dense else 1) + (8 if dense else 12) * T * k,
                "flops": 4 * T * (E if dense else k)}
    per = 0.5 + 2.0 / case["group"]                     # bytes of a weight with its scale
    if op == "quantise":
        n = case["E"] * case["K"] * case["N"]
        return {"bytes": int(n * (4 + 2 * per)), "flops": 4 * n}
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": int(K * N * per) + 2 * T * (K + N), "flops": 2 * T * K * N}
    T, d, f, E, k, S = (case[n] for n in ("T", "d", "f", "E", "k", "S"))
    used = E * (1 - (1 - k / E) ** T) + S               # experts that a routing of this size wants
    return {"bytes": int(3 * used * d * f * per) + 4 * T * d + 8 * T * k,
            "flops": 6 * T * (k + S) * d * f}
