"""Plain 64-bit forms of the attention operators, and the bounds the kernels'
outputs are held to.

Bounds, from the arithmetic (u = 2^-8, half a step of bf16; fp32 terms in
multiples of 2^-24):
  * rotation: two products and a sum in fp32 of values |x1| + |x2|, sine and
    cosine within 2^-21 (the angle's 2^-32 turns fraction held in 24 bits, and
    the function's own error), then one rounding to bf16:
      |got - ref| <= u |ref| + 2^-20 m (|x1| + |x2|)    (m the scale, at least 1)
    (the second term also covers u times the first error);
  * attention, with A = sum_j p_j |v_j| / l: each weight is rounded to bf16 for
    the product with V, the output is rounded once, and a score is off by at
    most e = (D + 16) 2^-23 max_j scale sum_d |q_d k_jd| + 2^-20, which moves a
    weight by that ratio, in the numerator and the denominator:
      |got - ref| <= u |ref| + (u + 2 e + 2^-14) (1 + u) A
    (2^-14: sums of up to 2^10 fp32 terms of one sign per accumulator, joined);
  * log-sum-exp: |got - ref| <= e + 2^-20 (1 + |ref|).
"""
import math

import torch

U = torch.finfo(torch.bfloat16).eps / 2


def rotate(x, pos, inv_freq, axis, interleaved=False, transpose=False, scale=1.0):
    """x [T, H, D] -> (R x, bound of the error), float64; pos [n_axes, T]."""
    x = x.double()
    rd = 2 * len(inv_freq)
    w = torch.tensor(inv_freq, dtype=torch.float64, device=x.device)
    ang = pos.double()[torch.tensor(axis, device=x.device)].T * w
    c, s = ang.cos()[:, None] * scale, ang.sin()[:, None] * scale
    if transpose:
        s = -s
    y, mag = x.clone(), torch.zeros_like(x)
    i1 = slice(0, rd, 2) if interleaved else slice(0, rd // 2)
    i2 = slice(1, rd, 2) if interleaved else slice(rd // 2, rd)
    a, b = x[..., i1], x[..., i2]
    y[..., i1], y[..., i2] = a * c - b * s, b * c + a * s
    mag[..., i1] = mag[..., i2] = (a.abs() + b.abs()) * max(1.0, abs(scale))
    return y, U * y.abs() + 2.0 ** -20 * mag


def slots(cu_q, kv_len, table, page_size):
    """(row, page, slot) of every token of the batch."""
    rows = []
    for b in range(len(kv_len)):
        nq = cu_q[b + 1] - cu_q[b]
        for i in range(nq):
            c = kv_len[b] - nq + i
            rows.append((cu_q[b] + i, int(table[b][c // page_size]), c % page_size))
    return rows


def attention(q, kc, vc, cu_q, kv_len, table, scale, causal=True, window=0, sinks=None):
    """q [T, Hq, D], kc and vc [pages, Hkv, page_size, D] -> out, its bound, lse,
    its bound, all float64. Keys a row does not see are left out of its sums, so
    what they hold does not matter. Rows of no sequence are NaN."""
    T, Hq, D = q.shape
    Hkv, ps = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    dev = q.device
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64, device=dev)
    tol, lse, lse_tol = out.clone(), out[..., 0].clone(), out[..., 0].clone()
    for b in range(len(kv_len)):
        s0, nq, n = cu_q[b], cu_q[b + 1] - cu_q[b], kv_len[b]
        if nq == 0:
            continue
        pages = torch.tensor([int(table[b][i]) for i in range((n + ps - 1) // ps)],
                             dtype=torch.long, device=dev)
        c = (torch.arange(nq, device=dev) + n - nq)[:, None]
        j = torch.arange(n, device=dev)[None]
        see = (j <= c) if causal else torch.ones(nq, n, dtype=torch.bool, device=dev)
        if window:
            see = see & (j > c - window)
        for h in range(Hq):
            K = kc[pages, h // G].reshape(-1, D)[:n].double()
            V = vc[pages, h // G].reshape(-1, D)[:n].double()
            x = q[s0:s0 + nq, h].double()
            s = torch.where(see, (x @ K.nan_to_num(0.0, 0.0, 0.0).T) * scale, -math.inf)
            mag = (x.abs() @ K.nan_to_num(0.0, 0.0, 0.0).abs().T) * scale
            mag = torch.where(see, mag, torch.zeros_like(mag))
            sink = -math.inf if sinks is None else float(sinks[h])
            m = s.amax(1, keepdim=True) if n else torch.full((nq, 1), -math.inf,
                                                             dtype=torch.float64, device=dev)
            m = torch.clamp(m, min=sink)
            ref = torch.where(m.isinf(), torch.zeros_like(m), m)
            p = torch.exp(s - ref)
            l = p.sum(1, keepdim=True) + torch.exp(sink - ref)
            # 0 * NaN is left out: only seen keys enter
            bad = ~V.isfinite()
            Vz = V.masked_fill(bad, 0.0)
            o, a = p @ Vz, p @ Vz.abs()
            if bad.any():
                hit = see.double() @ bad.double() > 0
                o = torch.where(hit, torch.full_like(o, math.nan), o)
            o = torch.where(l > 0, o / l, torch.zeros_like(o))
            a = torch.where(l > 0, a / l, torch.zeros_like(a))
            e = (D + 16) * 2.0 ** -23 * (mag.amax(1, keepdim=True) if n else 0.0) + 2.0 ** -20
            out[s0:s0 + nq, h] = o
            tol[s0:s0 + nq, h] = U * o.abs() + (U + 2 * e + 2.0 ** -14) * (1 + U) * a
            L = ref + torch.log(l)
            lse[s0:s0 + nq, h] = L[:, 0]
            lse_tol[s0:s0 + nq, h] = (e + 2.0 ** -20 * (1 + L.abs()))[:, 0]
    return out, tol, lse, lse_tol
