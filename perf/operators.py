"""Workloads of the attention operators: the rotary positions, the append to a
paged cache of keys and values, and the attention of new tokens over it.

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
def _case(name, op, Hq, Hkv, D, page, q_lens, kv_lens, **kw):
    """A ragged batch: sequence b has q_lens[b] new tokens, the last ones of
    its kv_lens[b] tokens. Lengths are kept as text so a case stays plain."""
    c = {"name": name, "op": op, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
         "q_lens": " ".join(map(str, q_lens)), "kv_lens": " ".join(map(str, kv_lens)),
         "window": 0, "sinks": False, "rd": D, "interleaved": False, "axes": 1,
         "transpose": False}
    c.update(kw)
    return c


def _spread(n, lo, hi):
    """n lengths spread over [lo, hi] (in their logarithm), in a mixed order."""
    v = [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]
    return [v[(i * 37 + 11) % n] for i in range(n)]


def listed():
    out = []
    # one user's next token early in a chat: nothing but latency
    out.append(_case("attn_decode_one", "attn", 64, 8, 64, 16, [1], [613], sinks=True))
    # a serving batch of chats of every length, one token each
    out.append(_case("attn_decode_batch", "attn", 64, 8, 64, 16, [1] * 64,
                     _spread(64, 17, 16384), sinks=True))
    # the same heads in a sliding-window layer: little to read, many sequences
    out.append(_case("attn_decode_window", "attn", 64, 8, 64, 16, [1] * 128,
                     _spread(128, 3, 8000), sinks=True, window=128))
    # a few users with long documents: one token each over a long cache
    out.append(_case("attn_decode_long", "attn", 32, 4, 128, 64, [1] * 4,
                     [131071, 90001, 120000, 65537]))
    # drafts of five tokens verified at once, pages that no tile divides
    out.append(_case("attn_verify", "attn", 32, 4, 128, 24, [5] * 32, _spread(32, 400, 9000)))
    # a training-sized batch of prompts from scratch: 4 x 4096 tokens
    out.append(_case("attn_prefill", "attn", 64, 8, 64, 64, [4096] * 4, [4096] * 4, sinks=True))
    # a chunk of a long prompt over what is cached already
    out.append(_case("attn_chunk_long", "attn", 32, 4, 128, 32, [2048], [31017]))
    # decodes and one prompt chunk in one call, five queries per key head, D = 80
    out.append(_case("attn_mixed", "attn", 20, 4, 80, 48, [1] * 31 + [777],
                     _spread(31, 30, 5000) + [2500]))
    # the append of a decode step
    out.append(_case("append_decode", "append", 32, 4, 128, 16, [1] * 64, _spread(64, 17, 16384)))
    # the append of a batch of prompts, rotary over time, height and width
    out.append(_case("append_prefill", "append", 64, 8, 64, 64, [4096, 5000, 3000, 4288],
                     [4096, 5000, 3000, 4288], axes=3))
    # a few tokens of images: rotation alone, neighbouring pairs
    out.append(_case("rope_small", "rope", 32, 4, 128, 16, [8], [8], axes=3, interleaved=True))
    # the rotation's backward pass in training, 4 x 4096 tokens
    out.append(_case("rope_train_bwd", "rope", 64, 8, 64, 16, [16384], [16384], axes=3,
                     transpose=True))
    return out


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top_flops = max(work(c)["flops"] for c in listed())
    top_bytes = max(work(c)["bytes"] for c in listed())
    while True:
        D = rng.choice([64, 64, 128, 128, 80, 72, 40, 112])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 5, 7, 8, 16])
        page = rng.choice([16, 16, 32, 64, 128, 24, 48, 13])
        op = rng.choice(["attn", "attn", "attn", "append", "rope"])
        kind = rng.choice(["decode", "verify", "chunk", "mixed"])
        kw = {}
        if op == "attn":
            B = _log_int(rng, 1, 128) if kind != "chunk" else rng.choice([1, 2, 3, 4])
            kv = [_log_int(rng, 1, 131072 if B <= 4 else 16384) for _ in range(B)]
            if kind == "decode":
                ql = [1] * B
            elif kind == "verify":
                n = rng.randint(2, 9)
                ql = [min(n, k) for k in kv]
            elif kind == "chunk":
                ql = [min(_log_int(rng, 60, 4096), k) for k in kv]
            else:
                ql = [1] * B
                ql[rng.randrange(B)] = _log_int(rng, 60, 2048)
                kv = [max(k, q) for k, q in zip(kv, ql)]
            kw = {"window": rng.choice([0, 0, 0, 128, rng.randint(1, 3000)]),
                  "sinks": rng.random() < 0.4}
        else:
            T = _log_int(rng, 1, 16384)
            B = min(T, _log_int(rng, 1, 64)) if op == "append" else 1
            ql = [T // B] * B
            ql[-1] += T - sum(ql)
            kv = [q + (rng.randint(0, 4000) if op == "append" else 0) for q in ql]
            rd = rng.choice([D, D, D // 2])
            kw = {"rd": rd - rd % 2, "interleaved": rng.random() < 0.4,
                  "axes": rng.choice([1, 3, 3]),
                  "transpose": op == "rope" and rng.random() < 0.5}
        c = _case("", op, Hkv * G, Hkv, D, page, ql, kv, **kw)
        del c["name"]
        w = work(c)
        if w["flops"] <= top_flops and w["bytes"] <= top_bytes and sum(ql) * Hkv * G <= (1 << 20):
            return c


def _lens(case):
    return [int(v) for v in case["q_lens"].split()], [int(v) for v in case["kv_lens"].split()]


# ------------------------------------------------------------------ inputs --
BASE = 150000.0


def _axis_of_pair(case):
    """Which position axis turns each pair: all the first, or time, height
    and width taken in sections of about a quarter, 3/8 and 3/8."""
    n = case["rd"] // 2
    if case["axes"] == 1:
        return [0] * n
    a = max(1, n // 4)
    h = (n - a) // 2
    return [0 if i < a else 1 if i < a + h else 2 for i in range(n)]


def prepare(case, seed):
    """Inputs on the GPU: queries from one projection's output, keys and values as
    views of another's, a cache whose pages lie in a random order, the batch's lengths and
    page table, positions, sinks; with ``own`` also the library's objects."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    Hq, Hkv, D, ps = case["Hq"], case["Hkv"], case["D"], case["page"]
    ql, kv = _lens(case)
    T, B = sum(ql), len(ql)
    st = {"case": case, "ql": ql, "kv": kv, "T": T}
    st["q"] = torch.randn(T, Hq, D, generator=gen, device=dev).to(BF16)
    kv_proj = torch.randn(T, 2 * Hkv * D, generator=gen, device=dev).to(BF16)
    st["k"] = kv_proj[:, :Hkv * D].view(T, Hkv, D)
    st["v"] = kv_proj[:, Hkv * D:].view(T, Hkv, D)
    # image tokens count rows and columns; text tokens move all axes together
    n_ax = case["axes"]
    if case["op"] != "attn":
        base_pos = torch.cat([torch.arange(k - q, k) for q, k in zip(ql, kv)])
        pos = torch.stack([base_pos] * n_ax)
        if n_ax == 3:
            img = torch.rand(T, generator=cpu) < 0.5
            pos[1] = torch.where(img, base_pos // 32 % 32 + 7, pos[1])
            pos[2] = torch.where(img, base_pos % 32 + 7, pos[2])
        # far positions too: a sequence deep into a long context
        pos = pos + int(torch.randint(0, 100000, (1,), generator=cpu))
        st["pos"] = pos.to(torch.int32).to(dev)
    if case["op"] != "rope":
        n_pp = [(k + ps - 1) // ps for k in kv]
        n_pages = sum(n_pp) + 3
        order = torch.randperm(n_pages, generator=cpu).to(torch.int32)
        table = torch.full((B, max(n_pp) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(n_pp):
            table[b, :n] = order[at:at + n]
            at += n
        st["table"] = table.to(dev)
        shape = (n_pages, Hkv, ps, D)
        st["k_cache"] = torch.randn(shape, generator=gen, device=dev, dtype=BF16)
        st["v_cache"] = torch.randn(shape, generator=gen, device=dev, dtype=BF16)
        st["cu_q"] = torch.tensor([0] + [sum(ql[:i + 1]) for i in range(B)], dtype=torch.int32,
                                  device=dev)
        st["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    st["sinks"] = (torch.randn(Hq, generator=gen, device=dev) if case["sinks"] else None)
    st["inv_freq"] = BASE ** (-torch.arange(0, case["rd"], 2, dtype=torch.float64, device=dev)
                              / case["rd"])
    st["axis"] = torch.tensor(_axis_of_pair(case), dtype=torch.int64, device=dev)
    if own:
        from mixture_experts_routed_softmax_gb300 import attention as A
        if case["op"] != "attn":
            st["rope"] = A.Rope.from_base(case["rd"], BASE, axis=_axis_of_pair(case),
                                          n_axes=case["axes"], interleaved=case["interleaved"],
                                          device=dev)
        if case["op"] == "rope":
            st["q_out"] = torch.empty(T, Hq, D, dtype=BF16, device=dev)
            st["k_out"] = torch.empty(T, Hkv, D, dtype=BF16, device=dev)
        else:
            st["layer"] = A.PagedAttention(st["k_cache"], st["v_cache"], Hq,
                                           rope=st.get("rope"), window=case["window"],
                                           sinks=st["sinks"])
            st["buf"] = st["layer"].buffers(T)
            st["batch"] = A.KVBatch(st["cu_q"], st["kv_len"], st["table"], T, max(ql))
    return st


# --------------------------------------------------------------- plain form --
def _plain_rotate(st, x):
    """R x, or R^T x for the backward pass: angles in 64 bits, the products in 32."""
    case = st["case"]
    rd = case["rd"]
    ang = st["pos"].double()[st["axis"]].T * st["inv_freq"]          # [T, rd/2]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    if case["transpose"]:
        sin = -sin
    xf = x.float()
    y = xf.clone()
    if case["interleaved"]:
        a, b = xf[..., 0:rd:2], xf[..., 1:rd:2]
        y[..., 0:rd:2], y[..., 1:rd:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = xf[..., :rd // 2], xf[..., rd // 2:rd]
        y[..., :rd // 2], y[..., rd // 2:rd] = a * cos - b * sin, b * cos + a * sin
    return y.to(BF16)


def _plain_append(st):
    ps = st["case"]["page"]
    pages, slots = [], []
    for b, (nq, n) in enumerate(zip(st["ql"], st["kv"])):
        c = torch.arange(n - nq, n, device=st["table"].device)
        pages.append(st["table"][b].long()[c // ps])
        slots.append(c % ps)
    pages, slots = torch.cat(pages), torch.cat(slots)
    st["k_cache"][pages, :, slots] = _plain_rotate(st, st["k"])
    st["v_cache"][pages, :, slots] = st["v"]
    return {"q": _plain_rotate(st, st["q"]), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_attn(st):
    case = st["case"]
    Hq, Hkv, D, ps, win = (case[n] for n in ("Hq", "Hkv", "D", "page", "window"))
    G = Hq // Hkv
    out = torch.zeros(st["T"], Hq, D, dtype=BF16, device=st["q"].device)
    t0 = 0
    for b, (nq, n) in enumerate(zip(st["ql"], st["kv"])):
        np_ = (n + ps - 1) // ps
        pages = st["table"][b, :np_].long()
        K = st["k_cache"][pages].float().transpose(0, 1).reshape(Hkv, np_ * ps, D)[:, :n]
        V = st["v_cache"][pages].float().transpose(0, 1).reshape(Hkv, np_ * ps, D)[:, :n]
        step = max(1, (1 << 28) // (Hq * n))
        for i0 in range(0, nq, step):
            i1 = min(nq, i0 + step)
            q = st["q"][t0 + i0:t0 + i1].float().reshape(i1 - i0, Hkv, G, D)
            q = q.permute(1, 0, 2, 3).reshape(Hkv, (i1 - i0) * G, D)
            s = torch.matmul(q, K.transpose(1, 2)) * (1.0 / math.sqrt(D))
            c = torch.arange(n - nq + i0, n - nq + i1, device=s.device)[:, None]
            j = torch.arange(n, device=s.device)[None]
            hide = (j > c) | (j <= c - win) if win else j > c
            s = s.view(Hkv, i1 - i0, G, n).masked_fill(hide[None, :, None], NEG_INF)
            m = s.amax(-1, keepdim=True)
            if st["sinks"] is not None:
                sink = st["sinks"].view(Hkv, 1, G, 1)
                m = torch.maximum(m, sink)
            p = torch.exp(s - m)
            l = p.sum(-1, keepdim=True)
            if st["sinks"] is not None:
                l = l + torch.exp(sink - m)
            o = torch.matmul(p.view(Hkv, -1, n), V).view(Hkv, i1 - i0, G, D) / l
            out[t0 + i0:t0 + i1] = o.permute(1, 0, 2, 3).reshape(i1 - i0, Hq, D).to(BF16)
        t0 += nq
    return {"out": out}


def run(state):
    """One pass through the case's operator and its outputs."""
    op = state["case"]["op"]
    if own:
        if op == "attn":
            return {"out": state["layer"].attend(state["q"], state["batch"], state["buf"])}
        if op == "append":
            q = state["layer"].append(state["k"], state["v"], state["batch"], q=state["q"],
                                      q_out=state["buf"].q, pos=state["pos"])
            return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
        state["rope"].apply(state["q"], state["pos"], state["q_out"], k=state["k"],
                            k_out=state["k_out"], transpose=state["case"]["transpose"])
        return {"q": state["q_out"], "k": state["k_out"]}
    if op == "attn":
        return _plain_attn(state)
    if op == "append":
        return _plain_append(state)
    return {"q": _plain_rotate(state, state["q"]), "k": _plain_rotate(state, state["k"])}


# ---------------------------------------------------------------- 64 bits --
def _turn(x, pos, case, sign):
    """Rotation pair by pair as a complex product, in 64 bits."""
    rd, T = case["rd"], x.shape[0]
    z = x.double().clone()
    axis = _axis_of_pair(case)
    for i in range(rd // 2):
        w = math.exp(-2.0 * i / rd * math.log(BASE))
        e = torch.polar(torch.ones(T, dtype=torch.float64, device=x.device),
                        sign * w * pos[axis[i]].double())[:, None]
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rd // 2)
        r = torch.complex(x[..., lo].double(), x[..., hi].double()) * e
        z[..., lo], z[..., hi] = r.real, r.imag
    return z


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    sign = -1.0 if case["transpose"] else 1.0
    if op == "rope":
        return {"q": _turn(st["q"], st["pos"], case, sign),
                "k": _turn(st["k"], st["pos"], case, sign)}
    ps, D, G = case["page"], case["D"], case["Hq"] // case["Hkv"]
    table = st["table"].cpu().tolist()
    if op == "append":
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        k = _turn(st["k"], st["pos"], case, sign)
        page, slot = [], []
        for b, (nq, n) in enumerate(zip(st["ql"], st["kv"])):
            for c in range(n - nq, n):
                page.append(table[b][c // ps])
                slot.append(c % ps)
        page = torch.tensor(page, device=kc.device)
        slot = torch.tensor(slot, device=kc.device)
        for h in range(case["Hkv"]):
            kc[page, h, slot] = k[:, h]
            vc[page, h, slot] = st["v"][:, h].double()
        return {"q": _turn(st["q"], st["pos"], case, sign), "k_cache": kc, "v_cache": vc}
    # attention: head by head, weights as exp(s - logsumexp)
    out = torch.zeros(st["T"], case["Hq"], D, dtype=torch.float64, device=st["q"].device)
    start = 0
    for b, (nq, n) in enumerate(zip(st["ql"], st["kv"])):
        pages = torch.tensor(table[b][:(n + ps - 1) // ps], device=out.device)
        for h in range(case["Hq"]):
            K = st["k_cache"][pages, h // G].reshape(-1, D)[:n].double()
            V = st["v_cache"][pages, h // G].reshape(-1, D)[:n].double()
            for i0 in range(0, nq, 1024):
                i1 = min(nq, i0 + 1024)
                where = torch.arange(n - nq + i0, n - nq + i1, device=out.device).unsqueeze(1)
                age = where - torch.arange(n, device=out.device).unsqueeze(0)
                seen = age >= 0
                if case["window"]:
                    seen &= age < case["window"]
                s = st["q"][start + i0:start + i1, h].double() @ K.T / math.sqrt(D)
                s = torch.where(seen, s, torch.full_like(s, NEG_INF))
                z = torch.logsumexp(s, dim=1, keepdim=True)
                if st["sinks"] is not None:
                    z = torch.logaddexp(z, st["sinks"][h].double())
                out[start + i0:start + i1, h] = torch.exp(s - z) @ V
        start += nq
    return {"out": out}


def work(case):
    ql, kv = _lens(case)
    Hq, Hkv, D, win = case["Hq"], case["Hkv"], case["D"], case["window"]
    T = sum(ql)
    if case["op"] == "rope":
        el = T * (Hq + Hkv) * D
        return {"bytes": 4 * el + 4 * T * case["axes"], "flops": 3 * T * (Hq + Hkv) * case["rd"]}
    if case["op"] == "append":
        return {"bytes": 4 * T * (Hq + 2 * Hkv) * D + 4 * T * case["axes"],
                "flops": 3 * T * (Hq + Hkv) * case["rd"]}
    pairs = keys = 0
    for nq, n in zip(ql, kv):
        first = n - nq
        keys += n - max(0, first - win + 1) if win else n
        if win:
            for c in range(first, n):
                pairs += min(c + 1, win)
        else:
            pairs += nq * first + nq * (nq + 1) // 2
    return {"bytes": 4 * T * Hq * D + 4 * keys * Hkv * D, "flops": 4 * D * Hq * pairs}
