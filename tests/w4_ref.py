"""4-bit weights in 64 bits: codes, scales, products and the experts' forward from
the formulas of include/moe.h (moe_w4), with bounds of the kernels' error.

Bounds. A product of code and x is exact in fp32; the matrix unit adds sixteen of
them to an accumulator and may cut each addition at its last place (2^-23 of the
magnitudes so far), scales and warps add a multiplication and an addition each:
``sums`` counts those. A bf16 result is off by half a step, 2^-8 of itself."""
import numpy as np

FP4 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
BF16_MAX = 2.0 ** 128 - 2.0 ** 120
U_BF16, CUT = 2.0 ** -8, 2.0 ** -23


def values(codes, kind):
    c = np.asarray(codes).astype(np.int64) & 15
    if kind == "int4":
        return np.where(c >= 8, c - 16, c).astype(np.float64)
    return np.where(c >= 8, -1.0, 1.0) * FP4[c & 7]


def weights(codes, scales, kind, group):
    """[.., K, N] in 64 bits of codes and scales [.., ceil(K/group), N]."""
    K = codes.shape[-2]
    s = np.repeat(np.asarray(scales, dtype=np.float64), group, axis=-2)[..., :K, :]
    return values(codes, kind) * s


def scale_of(a, kind):
    """A group's scale from its largest magnitude."""
    if not np.isfinite(a):
        return np.nan
    if a < 2.0 ** -120:
        return 0.0
    if kind == "int4":
        # the least s = n 2^e, n of five bits, with 7 s >= a
        e = np.floor(np.log2(a / 7)) - 4
        n = np.ceil(a / 7 / 2.0 ** e)
        return n * 2.0 ** e
    e = -130.0
    e = np.floor(np.log2(a)) - 3
    while 6 * 2.0 ** e < a:
        e += 1
    return 2.0 ** e


def quantise(w, kind, group):
    """(codes, scales) of w [K, N], a value at a time."""
    K, N = w.shape
    G = -(-K // group)
    codes, scales = np.zeros((K, N), dtype=np.uint8), np.zeros((G, N))
    for n in range(N):
        for g in range(G):
            col = w[g * group:(g + 1) * group, n].astype(np.float64)
            a = np.abs(col).max() if np.isfinite(col).all() else np.nan
            s = scales[g, n] = scale_of(a, kind)
            if not s > 0:
                continue
            q = col / s
            grid = np.arange(8.0) if kind == "int4" else FP4
            d = np.abs(np.abs(q)[:, None] - grid)
            best = d.min(1, keepdims=True)
            # the nearest value; halves to the even code; one that bf16 holds
            c = np.array([max(np.nonzero(r)[0], key=lambda i: (i % 2 == 0, i))
                          for r in d == best])
            c = np.where(grid[c] * s > BF16_MAX, c - 1, c)
            if kind == "int4":
                c = np.where(q < 0, -c, c) & 15
            else:
                c = np.where((q < 0) & (c > 0), c + 8, c)
            codes[g * group:(g + 1) * group, n] = c
    return codes, scales


def sums(K):
    """Additions that a sum over K goes through, each cut at 2^-23 of the magnitudes."""
    return K / 16 + 2 * (K / 32) + 40


def linear_bound(x, W, out_bf16=True):
    """(exact product, bound of the error) of x W."""
    ref = x @ W
    return ref, sums(x.shape[1]) * CUT * (np.abs(x) @ np.abs(W)) + out_bf16 * U_BF16 * np.abs(ref)


def experts(x, idx, w, gate, up, down, E, act=None, rounded=0.0, a_rounded=U_BF16):
    """(y, bound) of the experts' forward; weights [E+S, .., ..] in 64 bits. rounded: how far
    code * scale may be rounded in the products, relative (2^-8 where scales have many bits);
    a_rounded: how far A is."""
    limit, alpha, off = act if act is not None else (np.inf, 1.0, 0.0)
    T, d = x.shape
    S = gate.shape[0] - E
    y, err, mag = np.zeros((T, d)), np.zeros((T, d)), np.zeros((T, d))
    for e in range(E + S):
        if e < E:
            t, j = np.nonzero(idx == e)
            we = w[t, j]
        else:
            t, we = np.arange(T), np.ones(T)
        if not len(t):
            continue
        xe, cut = x[t], sums(d) * CUT + rounded
        G, U = xe @ gate[e], xe @ up[e]
        eG, eU = (cut * (np.abs(xe) @ np.abs(m[e])) for m in (gate, up))
        Gc, Uc = np.minimum(G, limit), np.clip(U, -limit, limit)
        sig = 1 / (1 + np.exp(-alpha * Gc))
        A = Gc * sig * (Uc + off)
        # |h'| <= 1.1 for every alpha; exp and quotient: 2^-20 (1 + |alpha G|)
        eA = (1.1 * np.abs(Uc + off) * eG + np.abs(Gc * sig) * eU + 1.1 * eG * eU
              + np.abs(A) * (a_rounded + 2.0 ** -20 * (1 + np.abs(alpha * Gc))))
        Y = A @ down[e]
        absY = (np.abs(A) + eA) @ np.abs(down[e])
        eY = eA @ np.abs(down[e]) + (sums(down.shape[1]) * CUT + rounded) * absY
        np.add.at(y, t, we[:, None] * Y)
        np.add.at(err, t, np.abs(we)[:, None] * eY)
        np.add.at(mag, t, np.abs(we)[:, None] * absY)
    slots = idx.shape[1] + S
    return y, err + slots * CUT * mag + U_BF16 * (np.abs(y) + err)


def assert_within(name, got, ref, bound):
    worst = float((np.abs(got - ref) / (bound + 1e-30)).max()) if ref.size else 0.0
    assert worst <= 1.0, f"{name}: worst |diff| / bound = {worst:.3f}"
    return worst
