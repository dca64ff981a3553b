"""The attention operators on the GPU against plain 64-bit forms
(tests/attention_ref.py, where the tolerances are derived): rotary positions,
the append to a paged cache, and attention over it — head layouts, ragged
lengths from none to chunks, page sizes a tile does not divide, strides, masks
that leave rows without keys, and infinities and NaN in every masked place."""
import math

import pytest
import torch

import attention_ref as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
NAN = float("nan")


def _mod():
    from mixture_experts_routed_softmax_gb300.build import build
    build()
    from mixture_experts_routed_softmax_gb300 import attention
    return attention


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """A ragged batch over a shuffled cache. Everything outside the sequences'
    own slots is NaN: the rest of last pages, other pages, and the bytes
    between strided rows."""

    def __init__(self, Hq, Hkv, D, ps, ql, kv, seed=0, heads_first=True, pad=0, extra_rows=0,
                 spare=3):
        A = _mod()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.ps, self.ql, self.kv = Hq, Hkv, D, ps, ql, kv
        self.cu = [0]
        for n in ql:
            self.cu.append(self.cu[-1] + n)
        self.T = self.cu[-1] + extra_rows
        npp = [(n + ps - 1) // ps for n in kv]
        n_pages = sum(npp) + spare
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        width = max(npp + [1]) + 1
        self.table, at = [], 0
        for n in npp:
            self.table.append(order[at:at + n] + [-7] * (width - n))
            at += n
        shape = (n_pages, Hkv, ps, D + pad) if heads_first else (n_pages, ps, Hkv, D + pad)
        kc = torch.full(shape, NAN, dtype=BF16, device="cuda")
        vc = torch.full(shape, NAN, dtype=BF16, device="cuda")
        self.k_cache, self.v_cache = kc[..., :D], vc[..., :D]
        sw = (lambda t: t) if heads_first else (lambda t: t.transpose(1, 2))  # noqa: E731
        self.kn, self.vn = sw(self.k_cache), sw(self.v_cache)   # [pages, heads, slots, D]
        for b, n in enumerate(kv):
            for i in range(npp[b]):
                m = min(ps, n - i * ps)
                pg = self.table[b][i]
                self.kn[pg, :, :m] = torch.randn(Hkv, m, D, generator=g, device="cuda").to(BF16)
                self.vn[pg, :, :m] = torch.randn(Hkv, m, D, generator=g, device="cuda").to(BF16)
        qp = torch.full((self.T, Hq * D + 8), NAN, dtype=BF16, device="cuda")
        self.q = qp[:, :Hq * D].view(self.T, Hq, D) if self.T else qp[:, :Hq * D].reshape(0, Hq, D)
        self.q.copy_(torch.randn(self.T, Hq, D, generator=g, device="cuda"))
        self.batch = A.KVBatch(_i32(self.cu), _i32(kv), _i32(self.table), self.T, max(ql + [0]))
        self.heads_first = heads_first

    def attend(self, lse=True, max_q=None, **kw):
        A = _mod()
        layer = A.PagedAttention(self.k_cache, self.v_cache, self.Hq,
                                 heads_first=self.heads_first, **kw)
        b = layer.buffers(self.T, lse=lse)
        b.out.fill_(NAN)
        if lse:
            b.lse.fill_(NAN)
        b.ws.fill_(255)                 # its contents need no initialisation
        if max_q is not None:
            self.batch.args.max_q = max_q
        layer.attend(self.q, self.batch, b)
        assert layer.status() == 0
        return layer, b

    def check(self, **kw):
        layer, b = self.attend(**kw)
        kw.pop("max_q", None)
        sinks = kw.get("sinks")
        out, tol, lse, ltol = R.attention(self.q, self.kn, self.vn, self.cu, self.kv, self.table,
                                          layer.scale, kw.get("causal", True),
                                          kw.get("window", 0), sinks)
        _same(b.out, out, tol, "out")
        _same(b.lse, lse, ltol, "lse")
        return b


def _same(got, ref, tol, name):
    """Within tol where ref is finite; NaN where it is NaN; equal infinities."""
    got = got.double()
    nan = ref.isnan()
    assert bool((got.isnan() | got.isinf())[nan].all()), f"{name}: a value where none belongs"
    fin = ref.isfinite()
    assert torch.equal(got[~fin & ~nan], ref[~fin & ~nan]), f"{name}: infinities differ"
    assert bool(got[fin].isfinite().all()), f"{name}: a masked value reached a row"
    if fin.any():
        ratio = float(((got - ref).abs()[fin] / (tol[fin] + 1e-37)).max())
        assert ratio <= 1.0, f"{name}: error / bound = {ratio:.3f}"


LAYOUTS = [(8, 8, 64, 16), (16, 2, 64, 16), (6, 1, 128, 32), (10, 2, 80, 24), (14, 2, 40, 13),
           (3, 3, 8, 1), (32, 4, 128, 64), (16, 1, 112, 128), (40, 2, 72, 5), (64, 1, 16, 8)]


@pytest.mark.parametrize("Hq,Hkv,D,ps", LAYOUTS)
def test_single_tokens(Hq, Hkv, D, ps):
    kv = [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 500, 1111]
    Case(Hq, Hkv, D, ps, [1] * len(kv), kv).check()


@pytest.mark.parametrize("Hq,Hkv,D,ps", LAYOUTS)
def test_ragged_chunks(Hq, Hkv, D, ps):
    ql = [0, 1, 5, 130, 3, 0, 257, 64]
    kv = [9, 700, 5, 130, 77, 0, 600, 321]
    Case(Hq, Hkv, D, ps, ql, kv, seed=1).check()


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 130, 5000])
@pytest.mark.parametrize("ps", [16, 13])
def test_windows(window, ps):
    c = Case(8, 2, 64, ps, [1, 7, 300, 1], [1000, 45, 450, 3], seed=2)
    c.check(window=window)
    c.check(window=window, causal=False)


@pytest.mark.parametrize("D,ps", [(64, 16), (128, 24), (80, 7)])
def test_without_the_causal_mask(D, ps):
    Case(12, 4, D, ps, [1, 9, 200], [333, 9, 250], seed=3).check(causal=False)


@pytest.mark.parametrize("ql", [[1] * 5, [4, 40, 1, 200, 9]])
def test_sinks(ql):
    c = Case(16, 2, 64, 16, ql, [300, 40, 1, 260, 77], seed=4)
    sinks = torch.linspace(-30, 30, 16, device="cuda")
    c.check(sinks=sinks)
    c.check(sinks=torch.full((16,), -math.inf, device="cuda"))


@pytest.mark.parametrize("sinks", [False, True])
def test_rows_without_keys(sinks):
    # more new tokens than the sequence has: the first rows see nothing
    c = Case(8, 2, 64, 16, [5, 300, 1, 2], [2, 120, 0, 0], seed=5)
    kw = {"sinks": torch.randn(8, device="cuda")} if sinks else {}
    b = c.check(**kw)
    assert bool((b.out[:3] == 0).all()) and bool((b.out[305:] == 0).all())


def test_rows_of_no_sequence_stay():
    c = Case(8, 2, 64, 16, [3, 4], [30, 4], seed=6, extra_rows=5)
    _, b = c.attend()
    assert bool(b.out[7:].isnan().all()) and bool(b.lse[7:].isnan().all())
    assert bool(b.out[:7].isfinite().all())


def test_no_tokens_and_no_sequences():
    A = _mod()
    c = Case(8, 2, 64, 16, [0, 0], [5, 0])
    c.attend()
    e = A.KVBatch(_i32([0]), torch.empty(0, dtype=torch.int32, device="cuda"),
                  torch.empty(0, 1, dtype=torch.int32, device="cuda"), 0)
    layer = A.PagedAttention(c.k_cache, c.v_cache, 8)
    layer.attend(torch.empty(0, 8, 64, dtype=BF16, device="cuda"), e, layer.buffers(0))
    assert layer.status() == 0


@pytest.mark.parametrize("heads_first", [True, False])
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("ql,kv", [([1, 1, 1], [100, 7, 640]), ([140, 20], [300, 20])])
def test_cache_layouts(heads_first, pad, ql, kv):
    Case(8, 2, 128, 16, ql, kv, seed=7, heads_first=heads_first, pad=pad).check()


@pytest.mark.parametrize("max_q", [0, 1, 4, 300, 1 << 20])
def test_the_hint_changes_nothing(max_q):
    Case(16, 4, 64, 16, [1, 300, 5], [900, 400, 5], seed=8).check(max_q=max_q)


@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf, -3.3895313892515355e38])
@pytest.mark.parametrize("D,ps,ql,kv", [(64, 16, [40], [90]), (128, 32, [200], [333]),
                                        (80, 13, [50], [50]), (128, 16, [2], [70])])
def test_values_in_masked_places(bad, D, ps, ql, kv):
    """A key or value a row does not see, in a token later in the chunk or
    behind the window, reaches only the rows that see it."""
    c = Case(8, 2, D, ps, ql, kv, seed=9)
    n, nq = kv[0], ql[0]
    where = [n - 1, n - nq // 2]
    for j in where:
        pg, sl = c.table[0][j // ps], j % ps
        c.vn[pg, 0, sl, 3] = bad
        c.vn[pg, 1, sl] = bad
    layer, b = c.attend()
    out, tol, _, _ = R.attention(c.q, c.kn, c.vn, c.cu, c.kv, c.table, layer.scale)
    first = min(where) - (n - nq)
    _same(b.out[:first], out[:first], tol[:first], "rows that see no such value")
    # and keys: rows before the first bad key are untouched
    c = Case(8, 2, D, ps, ql, kv, seed=10)
    for j in where:
        c.kn[c.table[0][j // ps], :, j % ps, 1] = bad
    layer, b = c.attend()
    out, tol, _, _ = R.attention(c.q, c.kn, c.vn, c.cu, c.kv, c.table, layer.scale)
    _same(b.out[:first], out[:first], tol[:first], "rows that see no such key")


@pytest.mark.parametrize("D,ps,nq,n,window", [(64, 16, 64, 300, 40), (128, 16, 3, 300, 100),
                                              (128, 13, 150, 400, 90)])
def test_values_behind_the_window(D, ps, nq, n, window):
    c = Case(8, 2, D, ps, [nq], [n], seed=11)
    first_key = n - nq - window + 1           # of the chunk's first row
    cut = first_key + nq // 2                 # rows past the middle do not see it
    for j in range(cut + 1):
        c.vn[c.table[0][j // ps], :, j % ps] = NAN
        c.kn[c.table[0][j // ps], :, j % ps] = NAN
    layer, b = c.attend(window=window)
    out, tol, _, _ = R.attention(c.q, c.kn, c.vn, c.cu, c.kv, c.table, layer.scale, window=window)
    rows = slice(nq // 2 + 1, nq)
    _same(b.out[rows], out[rows], tol[rows], "rows whose window starts later")


def test_pages_before_the_window_are_not_touched():
    # a server frees them: their table entries may be anything
    c = Case(8, 2, 64, 16, [1, 40], [400, 300], seed=12)
    t = c.batch.page_table
    t[0, :(400 - 128) // 16] = -1
    t[1, :(300 - 40 + 1 - 128) // 16] = 1 << 30
    c.check(window=128)


def test_large_scores_and_lowest_values():
    c = Case(8, 2, 64, 16, [1, 100], [300, 300], seed=13)
    c.q.mul_(60.0)
    c.check()
    c.kn[c.table[0][3], :, 5] = -3.3895313892515355e38     # a score near -inf: weight 0
    layer, b = c.attend()
    assert bool(b.out[1:].isfinite().all())


def test_offsets_past_32_bits():
    A = _mod()
    Hq, Hkv, D, ps, n = 8, 2, 64, 16, 200
    c = Case(Hq, Hkv, D, ps, [1, 30], [n, 90], seed=14)
    stride = 1 << 28                            # elements between pages
    n_pages = c.k_cache.shape[0]
    big = torch.empty(stride * (n_pages - 1) + Hkv * ps * D * 2, dtype=BF16, device="cuda")
    assert big.numel() > 1 << 32
    kc = big.as_strided((n_pages, Hkv, ps, D), (stride, ps * D, D, 1), 0)
    vc = big.as_strided((n_pages, Hkv, ps, D), (stride, ps * D, D, 1), Hkv * ps * D)
    kc.copy_(c.k_cache)
    vc.copy_(c.v_cache)
    layer = A.PagedAttention(kc, vc, Hq)
    b = layer.buffers(c.T)
    layer.attend(c.q, c.batch, b)
    _, b0 = c.attend(lse=False)
    assert torch.equal(b.out, b0.out)
    # the append reaches the same far slots
    k = torch.randn(c.T, Hkv, D, device="cuda").to(BF16)
    layer.append(k, k, c.batch)
    for row, page, slot in R.slots(c.cu, c.kv, c.table, ps):
        assert torch.equal(kc[page, :, slot], k[row])
        assert torch.equal(vc[page, :, slot], k[row])
    assert layer.status() == 0


def test_twice_the_same_bits_and_another_stream():
    c = Case(32, 4, 128, 16, [1] * 20 + [200], list(range(50, 2050, 100)) + [900], seed=15)
    layer, b = c.attend()
    one, lse = b.out.clone(), b.lse.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.out.fill_(NAN)
    s.wait_stream(torch.cuda.current_stream())
    layer.attend(c.q, c.batch, b, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(b.out, one) and torch.equal(b.lse, lse)


def test_captured_into_a_graph_lengths_change():
    """Lengths, tables and queries are read on the device: a captured step serves
    the next one after they change in place."""
    c = Case(16, 2, 64, 16, [1, 1, 1], [200, 30, 7], seed=16)
    layer, b = c.attend()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.attend(c.q, c.batch, b)
    c.kv = [190, 20, 1]
    c.batch.kv_len.copy_(_i32(c.kv))
    c.q.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    out, tol, lse, ltol = R.attention(c.q, c.kn, c.vn, c.cu, c.kv, c.table, layer.scale)
    _same(b.out, out, tol, "out")
    _same(b.lse, lse, ltol, "lse")


def test_many_sequences():
    """More sequences than a block has threads; empty ones in between."""
    kv = [(i * 37) % 50 for i in range(700)]
    ql = [1 if n and i % 3 else 0 for i, n in enumerate(kv)]
    Case(4, 2, 64, 16, ql, kv, seed=17).check()


@pytest.mark.parametrize("what", ["page", "length", "negative length", "rows"])
def test_bad_device_data_is_reported(what):
    A = _mod()
    c = Case(8, 2, 64, 16, [1, 20, 1], [90, 33, 8], seed=18)
    layer = A.PagedAttention(c.k_cache, c.v_cache, 8)
    b = layer.buffers(c.T)
    layer.attend(c.q, c.batch, b)
    assert layer.status() == 0
    good = b.out.clone()
    if what == "page":
        c.batch.page_table[1, 0] = c.k_cache.shape[0]
    elif what == "length":
        c.batch.kv_len[1] = 1 << 30
    elif what == "negative length":
        c.batch.kv_len[1] = -5
    else:
        c.batch.cu_q[3] = 5000
    layer.attend(c.q, c.batch, b)
    from mixture_experts_routed_softmax_gb300 import _lib
    assert layer.status() == _lib.MOE_ERR_DEVICE_INDEX
    assert layer.status() == 0
    assert torch.equal(b.out[0], good[0])       # the other sequences are as before


# ------------------------------------------------------------------ rotation --
ROT = [(64, 64, False, 1), (128, 128, True, 3), (80, 80, False, 3), (128, 32, False, 1),
       (72, 36, False, 3), (40, 20, True, 1), (8, 2, True, 1), (64, 24, True, 3), (24, 24, False, 2)]


def _rot(rd, interleaved, n_axes, base=150000.0, scale=1.0):
    A = _mod()
    w = [base ** (-2.0 * i / rd) for i in range(rd // 2)]
    axis = [i * n_axes // (rd // 2) for i in range(rd // 2)]
    if interleaved and n_axes > 1:
        axis = [i % n_axes for i in range(rd // 2)]
    return A.Rope(w, axis=axis, n_axes=n_axes, interleaved=interleaved, scale=scale), w, axis


@pytest.mark.parametrize("D,rd,interleaved,n_axes", ROT)
@pytest.mark.parametrize("T", [1, 37, 2500])
@pytest.mark.parametrize("transpose", [False, True])
def test_rope(D, rd, interleaved, n_axes, T, transpose):
    rope, w, axis = _rot(rd, interleaved, n_axes, scale=1.25)
    g = torch.Generator(device="cuda").manual_seed(T)
    Hq, Hk = 5, 2
    proj = torch.randn(T, (Hq + Hk) * D + 16, generator=g, device="cuda").to(BF16)
    q = proj[:, :Hq * D].view(T, Hq, D)
    k = proj[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    pos = torch.randint(-1000, 2_000_000, (n_axes, T), generator=g, device="cuda").int()
    pos[:, 0] = 2 ** 31 - 1
    qo, ko = torch.full_like(q.contiguous(), NAN), torch.full_like(k.contiguous(), NAN)
    rope.apply(q, pos, qo, k=k, k_out=ko, transpose=transpose)
    for got, x in ((qo, q), (ko, k)):
        ref, tol = R.rotate(x, pos, w, axis, interleaved, transpose, 1.25)
        # the reference's own angle is a rounded double: |angle| 2^-53 off
        tol = tol + 2.0 ** -21 * x.double().abs().amax(-1, keepdim=True)
        _same(got, ref, tol, "rope")
        assert torch.equal(got[..., rd:], x[..., rd:])
    # q alone, in place
    qi = q.clone()
    rope.apply(qi, pos, qi, transpose=transpose)
    assert torch.equal(qi, qo)


def test_rope_gradient():
    """<g, R x>'s gradient is R^T g: against the formula, and against central
    differences of the 64-bit rotation."""
    T, H, D = 3, 2, 16
    rope, w, axis = _rot(D, False, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, D, generator=g, device="cuda").to(BF16)
    dy = torch.randn(T, H, D, generator=g, device="cuda").to(BF16)
    pos = torch.randint(0, 5000, (2, T), generator=g, device="cuda").int()
    dx = torch.empty_like(x)
    rope.apply(dy, pos, dx, transpose=True)
    f = lambda z: float((R.rotate(z, pos, w, axis)[0] * dy.double()).sum())  # noqa: E731
    _, tol = R.rotate(dy, pos, w, axis, transpose=True)
    h = 1e-4
    for t in range(T):
        for i in range(D):
            e = torch.zeros(T, H, D, dtype=torch.float64, device="cuda")
            e[t, 1, i] = h
            num = (f(x.double() + e) - f(x.double() - e)) / (2 * h)
            assert abs(float(dx[t, 1, i]) - num) <= float(tol[t, 1, i]) + 1e-8


def test_rope_no_tokens():
    rope, _, _ = _rot(16, False, 1)
    q = torch.empty(0, 2, 16, dtype=BF16, device="cuda")
    rope.apply(q, torch.empty(1, 0, dtype=torch.int32, device="cuda"), q)


# -------------------------------------------------------------------- append --
@pytest.mark.parametrize("D,rd,interleaved,n_axes", ROT)
@pytest.mark.parametrize("ps,ql", [(16, [1, 1, 1, 1]), (5, [3, 0, 40, 7]), (64, [2, 3000, 1, 9])])
@pytest.mark.parametrize("heads_first", [True, False])
def test_append(D, rd, interleaved, n_axes, ps, ql, heads_first):
    A = _mod()
    rope, w, axis = _rot(rd, interleaved, n_axes)
    kv = [q + e for q, e in zip(ql, [0, 33, 5, 90])]
    c = Case(6, 2, D, ps, ql, kv, seed=20, heads_first=heads_first, extra_rows=2)
    g = torch.Generator(device="cuda").manual_seed(21)
    k = torch.randn(c.T, 2, D, generator=g, device="cuda").to(BF16)
    v = torch.randn(c.T, 2, D, generator=g, device="cuda").to(BF16)
    pos = torch.randint(0, 300_000, (n_axes, c.T), generator=g, device="cuda").int()
    layer = A.PagedAttention(c.k_cache, c.v_cache, 6, rope=rope, heads_first=heads_first)
    before_k, before_v = c.kn.clone(), c.vn.clone()
    qo = torch.full((c.T, 6, D), NAN, dtype=BF16, device="cuda")
    layer.append(k, v, c.batch, q=c.q, q_out=qo, pos=pos)
    assert layer.status() == 0
    qr, qt = R.rotate(c.q, pos, w, axis, interleaved)
    _same(qo, qr, qt, "q")
    kr, kt = R.rotate(k, pos, w, axis, interleaved)
    where = R.slots(c.cu, c.kv, c.table, ps)
    rows = torch.tensor([x[0] for x in where], device="cuda")
    pg = torch.tensor([x[1] for x in where], device="cuda")
    sl = torch.tensor([x[2] for x in where], device="cuda")
    _same(c.kn[pg, :, sl], kr[rows], kt[rows], "k")
    assert torch.equal(c.vn[pg, :, sl], v[rows])
    # nothing else changed, NaN and all
    before_k[pg, :, sl] = c.kn[pg, :, sl]
    before_v[pg, :, sl] = v[rows]
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(c.kn), bits(before_k)) and torch.equal(bits(c.vn), bits(before_v))


def test_append_positions_default_to_the_cache():
    A = _mod()
    rope, w, axis = _rot(64, False, 1)
    c = Case(4, 2, 64, 16, [1, 30, 2], [500, 30, 77], seed=22)
    k = torch.randn(c.T, 2, 64, device="cuda").to(BF16)
    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(c.ql, c.kv)]).int().cuda()
    layer = A.PagedAttention(c.k_cache, c.v_cache, 4, rope=rope)
    q1, q2 = torch.empty_like(c.q.contiguous()), torch.empty_like(c.q.contiguous())
    layer.append(k, k, c.batch, q=c.q, q_out=q1)
    k1 = c.k_cache.clone().view(torch.int16)
    layer.append(k, k, c.batch, q=c.q, q_out=q2, pos=pos)
    assert torch.equal(q1, q2) and torch.equal(k1, c.k_cache.view(torch.int16))
    # without a rotation: copies
    plain = A.PagedAttention(c.k_cache, c.v_cache, 4)
    plain.append(k, k, c.batch, q=c.q, q_out=q2)
    assert torch.equal(q2, c.q)
    for row, page, slot in R.slots(c.cu, c.kv, c.table, 16):
        assert torch.equal(c.kn[page, :, slot], k[row])


def test_append_bad_pages_are_reported():
    A = _mod()
    from mixture_experts_routed_softmax_gb300 import _lib
    c = Case(4, 2, 64, 16, [1, 3, 1], [40, 20, 9], seed=23)
    layer = A.PagedAttention(c.k_cache, c.v_cache, 4)
    before = c.k_cache.clone().view(torch.int16)
    k = torch.randn(c.T, 2, 64, device="cuda").to(BF16)
    c.batch.page_table[0, 2] = -1
    c.batch.kv_len[1] = 1 << 29
    c.batch.page_table[2, 0] = c.k_cache.shape[0]
    layer.append(k, k, c.batch)
    assert layer.status() == _lib.MOE_ERR_DEVICE_INDEX
    assert torch.equal(before, c.k_cache.view(torch.int16))


def test_forward_is_append_then_attend():
    """One serving step: the new tokens see the cache and themselves."""
    A = _mod()
    rope, w, axis = _rot(64, False, 3)
    c = Case(8, 2, 64, 16, [1, 50, 1], [300, 50, 17], seed=24)
    g = torch.Generator(device="cuda").manual_seed(25)
    k = torch.randn(c.T, 2, 64, generator=g, device="cuda").to(BF16)
    v = torch.randn(c.T, 2, 64, generator=g, device="cuda").to(BF16)
    pos = torch.randint(0, 9000, (3, c.T), generator=g, device="cuda").int()
    layer = A.PagedAttention(c.k_cache, c.v_cache, 8, rope=rope)
    b = layer.buffers(c.T)
    layer.forward(c.q, k, v, c.batch, b, pos=pos)
    assert layer.status() == 0
    out, tol, _, _ = R.attention(b.q, c.kn, c.vn, c.cu, c.kv, c.table, layer.scale)
    _same(b.out, out, tol, "out")


# ------------------------------------------------- schedules, references, joins --
@pytest.mark.parametrize("D,ps,ql,kv", [(64, 16, [1, 3], [700, 400]), (128, 16, [1, 2], [500, 90]),
                                        (80, 13, [1, 9], [300, 250]), (64, 64, [300], [700]),
                                        (128, 24, [200, 40], [900, 300]), (40, 16, [90], [2000])])
def test_references_move_on_the_way(D, ps, ql, kv):
    """Scores that keep growing by far more than 2^16 in weight: sums, accumulators
    and weights already rounded are rescaled between and inside tiles. A weight so
    is rounded up to twice: twice the bound."""
    c = Case(8, 2, D, ps, ql, kv, seed=30)
    for b, n in enumerate(kv):
        for j in range(n):
            grow = 1.0 + 40.0 * j / n if j % 97 else 1.0 + 60.0 * j / n
            c.kn[c.table[b][j // ps], :, j % ps] *= grow
    sinks = torch.linspace(-5, 60, 8, device="cuda")
    for s in (None, sinks):
        layer, b = c.attend(sinks=s)
        out, tol, lse, ltol = R.attention(c.q, c.kn, c.vn, c.cu, c.kv, c.table, layer.scale,
                                          sinks=s)
        _same(b.out, out, 2 * tol, "out")
        _same(b.lse, lse, ltol, "lse")


@pytest.mark.parametrize("D,ps,nq", [(64, 16, 1), (128, 64, 1), (128, 13, 3), (128, 8, 9),
                                     (64, 24, 11), (128, 64, 7)])
def test_one_long_sequence_in_many_parts(D, ps, nq):
    c = Case(8, 2, D, ps, [nq], [30011], seed=31)
    c.check()
    c.check(sinks=torch.linspace(-3, 9, 8, device="cuda"), causal=False)


@pytest.mark.parametrize("D,G,nq,window", [(64, 2, 1, 0), (64, 8, 2, 100), (40, 2, 3, 17),
                                           (64, 1, 16, 90), (128, 2, 1, 100)])
def test_many_short_units(D, G, nq, window):
    """More uncut units than warps that work on them, empty ones in between."""
    B = 90
    kv = [(i * 53) % 240 for i in range(B)] if not window else [(i * 997) % 3000 for i in range(B)]
    ql = [min(nq, n) if i % 7 else 0 for i, n in enumerate(kv)]
    c = Case(8 * G, 8, D, 16, ql, kv, seed=32)
    c.check(window=window, sinks=torch.linspace(-4, 4, 8 * G, device="cuda"))


@pytest.mark.parametrize("D", [64, 128])
def test_long_stretches(D):
    """Enough units that cuts near a unit's end move there."""
    c = Case(64, 16, D, 64, [1024, 700, 901, 1100], [1024, 1500, 901, 1111], seed=33)
    c.check()
    c = Case(16, 8, D, 16, [1] * 130, [(i * 211) % 3000 + 1 for i in range(130)], seed=34)
    c.check()


def test_a_captured_chunk_follows_its_lengths():
    c = Case(16, 2, 64, 16, [100, 1, 60], [200, 80, 300], seed=35)
    layer, b = c.attend()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.attend(c.q, c.batch, b)
    c.kv = [150, 77, 60]
    c.batch.kv_len.copy_(_i32(c.kv))
    c.cu = [0, 90, 120, 161]
    c.batch.cu_q.copy_(_i32(c.cu))
    g.replay()
    torch.cuda.synchronize()
    out, tol, lse, ltol = R.attention(c.q, c.kn, c.vn, c.cu, c.kv, c.table, layer.scale)
    _same(b.out, out, tol, "out")
    _same(b.lse, lse, ltol, "lse")


def test_tokens_in_front_of_the_first_sequence_are_refused():
    A = _mod()
    from mixture_experts_routed_softmax_gb300 import _lib
    c = Case(4, 2, 64, 16, [3, 2], [40, 20], seed=36)
    layer = A.PagedAttention(c.k_cache, c.v_cache, 4)
    c.batch.cu_q[0] = 2                    # rows 0 and 1 are no sequence's
    k = torch.randn(c.T, 2, 64, device="cuda").to(BF16)
    before = c.kn.clone()
    layer.append(k, k, c.batch)
    assert layer.status() == _lib.MOE_ERR_DEVICE_INDEX
    for j in (37, 38):
        assert torch.equal(c.kn[c.table[0][j // 16], :, j % 16],
                           before[c.table[0][j // 16], :, j % 16])
    assert torch.equal(c.kn[c.table[0][2], :, 39 % 16], k[2])


def test_shapes_that_do_not_fit_are_refused():
    A = _mod()
    c = Case(8, 2, 64, 16, [1, 1], [40, 20], seed=37)
    layer = A.PagedAttention(c.k_cache, c.v_cache, 8)
    b = layer.buffers(2, lse=True)
    for q in (c.q[:1], c.q[:, :4], c.q.float(), c.q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            layer.attend(q, c.batch, b)
    with pytest.raises(ValueError):
        layer.attend(c.q, c.batch, layer.buffers(3, lse=True))
    with pytest.raises(ValueError):
        layer.append(c.q, c.q, c.batch)
    with pytest.raises(ValueError):
        layer.append(c.q[:, :2], c.q[:, :2], c.batch, q=c.q)
    with pytest.raises(ValueError):
        layer.append(c.q[:, :2], c.q[:, :2], c.batch, pos=_i32([0, 0]))
    with pytest.raises(ValueError):
        A.PagedAttention(c.k_cache, c.v_cache, 7)
    with pytest.raises(ValueError):
        A.KVBatch(c.batch.cu_q[:2], c.batch.kv_len, c.batch.page_table, 2)
    rope = A.Rope.from_base(64, 10000.0)
    with pytest.raises(ValueError):
        rope.apply(c.q, _i32([0, 1, 2]), torch.empty_like(c.q))


def test_a_block_of_attention_and_experts():
    """examples/serve_block.py on a small shape: prompts in one ragged step, then
    captured single-token steps; each step's attention against the 64-bit form
    over the cache it left, the block against its parts."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "serve_block.py")
    spec = importlib.util.spec_from_file_location("serve_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    _mod()
    ql = [70, 3, 200]
    blk = m.Block(d=256, Hq=8, Hkv=2, D=64, f=136, E=8, k=2, page_size=16, max_pages=20, B=3,
                  window=90, seed=1)
    x = torch.randn(sum(ql), 256, generator=torch.Generator(device="cuda").manual_seed(2),
                    device="cuda").to(BF16)
    last = blk.prefill(x, ql)
    assert last.shape == (3, 256) and bool(last.isfinite().all())
    dec = m.Decoder(blk, last)
    assert torch.equal(dec.x, last) and blk.kv_len.tolist() == ql
    lens = list(ql)
    for _ in range(4):
        before = dec.x.clone()
        row = dec.step()
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        assert blk.kv_len.tolist() == lens
        # the same step without the graph, part by part: its append writes the
        # same keys and values to the same slots
        batch = blk.batch([1] * 3)
        ab, mb = blk.buffers(3)
        y = blk.step(before, batch, (ab, mb))
        assert torch.equal(row, y)
        a = blk.attn
        out, tol, _, _ = R.attention(ab.q, a.k_cache, a.v_cache, [0, 1, 2, 3], lens,
                                     blk.table.tolist(), a.scale, window=90, sinks=a.sinks)
        _same(ab.out, out, tol, "out")
    assert blk.attn.status() == 0


@pytest.mark.parametrize("D,ps,ql,kv,window", [
    (64, 13, [700, 1, 300], [2000, 90, 310], 0), (128, 5, [900], [3000], 0),
    (80, 1, [400, 50], [4000, 50], 77), (40, 100, [5, 1500], [700, 1500], 0),
    (128, 13, [60] * 12, [900 + 31 * i for i in range(12)], 0)])
def test_chunks_over_odd_pages(D, ps, ql, kv, window):
    """Enough rows and keys for the chunk kernel to read pages no box fits."""
    c = Case(16, 2, D, ps, ql, kv, seed=38)
    c.check(window=window)
    c.check(window=window, causal=False, sinks=torch.linspace(-4, 9, 16, device="cuda"))


def test_odd_pages_that_do_not_exist_are_reported():
    A = _mod()
    from mixture_experts_routed_softmax_gb300 import _lib
    c = Case(16, 2, 64, 13, [600, 500], [2000, 1900], seed=39)
    layer = A.PagedAttention(c.k_cache, c.v_cache, 16)
    b = layer.buffers(c.T)
    layer.attend(c.q, c.batch, b)
    assert layer.status() == 0
    good = b.out.clone()
    c.batch.page_table[0, 7] = c.k_cache.shape[0]
    c.batch.page_table[0, 9] = -1
    layer.attend(c.q, c.batch, b)
    assert layer.status() == _lib.MOE_ERR_DEVICE_INDEX
    assert torch.equal(b.out[600:], good[600:])


# ------------------------------------------- small shapes on the chunk kernel --
class WideCase(Case):
    """A page table far wider than the sequences need and a large hint: what a
    call of much work looks like to the choice of a kernel."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        A = _mod()
        width = (1 << 27) // (max(self.T, 1) * self.Hq * self.ps) + 2
        t = torch.full((len(self.kv), max(width, len(self.table[0]) if self.table else 1)), -7,
                       dtype=torch.int32)
        for b, row in enumerate(self.table):
            t[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
        self.batch = A.KVBatch(_i32(self.cu), _i32(self.kv), t.cuda(), self.T, 1 << 28)


SMALL = ([(test_ragged_chunks, a) for a in LAYOUTS] +
         [(test_windows, (w, ps)) for w in (1, 2, 16, 63, 64, 65, 130, 5000) for ps in (16, 13)] +
         [(test_without_the_causal_mask, a) for a in ((64, 16), (128, 24), (80, 7))] +
         [(test_sinks, ([4, 40, 1, 200, 9],)), (test_rows_without_keys, (False,)),
          (test_rows_without_keys, (True,)), (test_rows_of_no_sequence_stay, ())] +
         [(test_cache_layouts, (h, p, [140, 20], [300, 20])) for h in (True, False)
          for p in (0, 8)] +
         [(test_values_in_masked_places, (bad, D, ps, ql, kv))
          for bad in (NAN, math.inf, -math.inf, -3.3895313892515355e38)
          for D, ps, ql, kv in ((64, 16, [40], [90]), (128, 32, [200], [333]),
                                (80, 13, [50], [50]))] +
         [(test_values_behind_the_window, a) for a in ((64, 16, 64, 300, 40),
                                                       (128, 13, 150, 400, 90))] +
         [(test_pages_before_the_window_are_not_touched, ()),
          (test_large_scores_and_lowest_values, ()), (test_offsets_past_32_bits, ()),
          (test_twice_the_same_bits_and_another_stream, ()),
          (test_a_captured_chunk_follows_its_lengths, ())] +
         [(test_references_move_on_the_way, a)
          for a in ((64, 64, [300], [700]), (128, 24, [200, 40], [900, 300]),
                    (40, 16, [90], [2000]), (80, 13, [60], [250]))] +
         [(test_bad_device_data_is_reported, (w,)) for w in ("page", "negative length", "rows")])


@pytest.mark.parametrize("i", range(len(SMALL)),
                         ids=[f"{t.__name__[5:]}-{i}" for i, (t, _) in enumerate(SMALL)])
def test_small_shapes_on_the_chunk_kernel(i, monkeypatch):
    test, args = SMALL[i]
    monkeypatch.setitem(globals(), "Case", WideCase)
    test(*args)
