"""4-bit weights on the GPU against 64 bits (w4_ref.py): quantisation and its way
back (equal), the linear layer, the experts' forward and the layer in front of it,
with bounds derived there before the first run."""
import numpy as np
import pytest
import torch

import w4_ref as W

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _codes(rng, E, K, N, kind, group, wide=False):
    """Random codes (all sixteen) and scales; wide: scales of eight significant bits."""
    codes = rng.integers(0, 16, (E, K, N)).astype(np.uint8)
    G = -(-K // group)
    s = torch.tensor(np.exp(0.5 * rng.standard_normal((E, G, N))) / np.sqrt(K) / 4)
    if not wide:                       # five bits
        m, e = torch.frexp(s)
        s = torch.ldexp((m * 32).round() / 32, e)
    return codes, s.to(BF16)


def _weights4(codes, scales, kind, group):
    from mixture_experts_routed_softmax_gb300.w4 import Weights4
    return Weights4.from_codes(torch.tensor(codes).cuda(), scales.cuda(), kind, group)


def _np(t):
    return t.detach().cpu().double().numpy()


def _status(lib):
    return lib.moe_status(torch.cuda.current_stream().cuda_stream)


# ------------------------------------------------------------ quantisation --
@pytest.mark.parametrize("kind", ["int4", "fp4"])
@pytest.mark.parametrize("E,K,N,group", [(1, 8, 8, 32), (2, 136, 72, 32), (1, 64, 16, 64),
                                         (3, 200, 24, 128), (1, 392, 136, 64), (1, 1000, 8, 32)])
def test_quantise(kind, E, K, N, group):
    from mixture_experts_routed_softmax_gb300.w4 import Weights4
    rng = np.random.default_rng(K + N)
    w = torch.tensor(rng.standard_normal((E, K, N)) * np.exp(2 * rng.standard_normal((E, 1, N))))
    w = w.to(BF16)
    w[0, :, 0] = 0.0                                     # a column of zeros
    w[0, :4, 1] = torch.tensor([7., -3.5, 2.5, 0.5]).to(BF16)      # halves
    w[-1, 5, 3] = 3.0e38
    w[-1, 6, 4] = 1e-38                                  # (alone in its group where K allows)
    q = Weights4.quantise(w.cuda(), kind, group)
    got = _np(q.dequantise())
    for e in range(E):
        codes, scales = W.quantise(w[e].double().numpy(), kind, group)
        np.testing.assert_array_equal(got[e], W.weights(codes, scales, kind, group))
    assert _status(q.lib) == 0


def test_quantise_keeps_what_is_not_finite():
    from mixture_experts_routed_softmax_gb300.w4 import Linear4, Weights4
    w = torch.ones(1, 128, 16, dtype=BF16)
    w[0, 3, 2], w[0, 70, 5] = float("inf"), float("nan")
    w[0, :, 9] = 1e-39                                   # below 2^-120: zeros
    q = Weights4.quantise(w.cuda(), "fp4", 64)
    got = q.dequantise().cpu()[0]
    bad = torch.zeros(128, 16, dtype=torch.bool)
    bad[:64, 2] = True
    bad[64:, 5] = True
    assert torch.equal(torch.isnan(got), bad)
    assert not got[:, 9].any() and bool((got[~bad.clone()].reshape(-1) >= 0).all())
    lin = Linear4(q)
    y = lin.apply(torch.ones(3, 128, dtype=BF16, device="cuda"), lin.buffers(3))
    assert torch.isnan(y[:, [2, 5]]).all() and torch.isfinite(y[:, [0, 1, 3, 4, 9]]).all()


@pytest.mark.parametrize("kind", ["int4", "fp4"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("wide", [False, True])
def test_pack_and_back(kind, group, wide):
    rng = np.random.default_rng(group)
    codes, scales = _codes(rng, 2, 328, 88, kind, group, wide)
    got = _np(_weights4(codes, scales, kind, group).dequantise())
    want = W.weights(codes, scales.double().numpy(), kind, group)
    # rounded to bf16 once (the product is exact in fp32), exact for scales of five bits
    np.testing.assert_array_equal(got, _np(torch.tensor(want).float().to(BF16)))
    if not wide:
        np.testing.assert_array_equal(got, want)


# ------------------------------------------------------------------ linear --
@pytest.mark.parametrize("kind", ["int4", "fp4"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,K,N", [(1, 8, 8), (1, 2880, 520), (3, 136, 72), (8, 1024, 96),
                                   (9, 200, 40), (17, 640, 264), (33, 392, 16), (70, 1288, 136),
                                   (300, 520, 392)])
def test_linear(kind, group, T, K, N):
    from mixture_experts_routed_softmax_gb300.w4 import Linear4
    rng = np.random.default_rng(T + K + N)
    codes, scales = _codes(rng, 1, K, N, kind, group)
    q = _weights4(codes, scales, kind, group)
    x = torch.tensor(rng.standard_normal((T, K))).to(BF16)
    Wd = W.weights(codes, scales.double().numpy(), kind, group)[0]
    for dtype in (BF16, torch.float32):
        lin = Linear4(q, out_dtype=dtype)
        ref, bound = W.linear_bound(x.double().numpy(), Wd, dtype is BF16)
        # rows of a wider array, in and out; what lies beside them stays
        xs = torch.full((T, K + 24), float("nan"), dtype=BF16, device="cuda")
        xs[:, 8:8 + K] = x.cuda()
        ys = torch.full((T, N + 5), 7.0, dtype=dtype, device="cuda")
        b = lin.buffers(T)
        lin.apply(xs[:, 8:8 + K], b, out=ys[:, 2:2 + N])
        W.assert_within("y", _np(ys[:, 2:2 + N]), ref, bound)
        assert bool((ys[:, :2] == 7).all()) and bool((ys[:, 2 + N:] == 7).all())
        y = lin.apply(x.cuda(), b)
        assert torch.equal(y, ys[:, 2:2 + N])            # the same bits
    assert _status(q.lib) == 0


@pytest.mark.parametrize("kind,group", [("int4", 32), ("int4", 128), ("fp4", 64)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,K,N", [(9, 8200, 4808), (40, 4096, 2880), (257, 1288, 1096),
                                   (300, 1032, 1128), (700, 8, 65536), (1900, 136, 1400)])
def test_linear_many_rows(kind, group, wide, T, K, N):
    """Work enough for tensor memory: K in one run and in several, whose sums meet."""
    from mixture_experts_routed_softmax_gb300.w4 import Linear4
    rng = np.random.default_rng(T + K + N)
    codes, scales = _codes(rng, 1, K, N, kind, group, wide)
    q = _weights4(codes, scales, kind, group)
    x = torch.tensor(rng.standard_normal((T, K))).to(BF16)
    x[T // 2, K - 1] = float("nan")
    clean = torch.nan_to_num(x).double().numpy()
    Wd = W.weights(codes, scales.double().numpy(), kind, group)[0]
    for dtype in (BF16, torch.float32):
        lin = Linear4(q, out_dtype=dtype)
        ref, bound = W.linear_bound(clean, Wd, dtype is BF16)
        if wide:                       # code * scale rounded to bf16
            bound = bound + W.U_BF16 * (np.abs(clean) @ np.abs(Wd))
        xs = torch.full((T, K + 24), float("nan"), dtype=BF16, device="cuda")
        xs[:, 8:8 + K] = x.cuda()
        ys = torch.full((T, N + 5), 7.0, dtype=dtype, device="cuda")
        b = lin.buffers(T)
        b.ws.fill_(255)
        lin.apply(xs[:, 8:8 + K], b, out=ys[:, 2:2 + N])
        got = ys[:, 2:2 + N]
        keep = [t for t in range(T) if t != T // 2]
        W.assert_within("y", _np(got[keep]), ref[keep], bound[keep])
        assert bool(torch.isnan(got[T // 2]).all())
        assert bool((ys[:, :2] == 7).all()) and bool((ys[:, 2 + N:] == 7).all())
        y = lin.apply(x.cuda(), b)
        assert torch.equal(y[keep], got[keep])           # the same bits
        short = lin.buffers(T)
        if short.ws.numel() > 256:
            short.ws = short.ws[:-256]
            with pytest.raises(RuntimeError):
                lin.apply(x.cuda(), short)
    assert _status(q.lib) == 0


def test_weights_cannot_be_replaced():
    q = _weights4(*_codes(np.random.default_rng(0), 1, 64, 16, "int4", 32), "int4", 32)
    for name in ("codes", "scales"):
        with pytest.raises(AttributeError):
            setattr(q, name, getattr(q, name).clone())


@pytest.mark.parametrize("T,K,N", [(97, 8, 8), (130, 128, 24), (2050, 136, 72), (60, 3200, 16)])
def test_linear_many_rows_of_small_matrices(T, K, N):
    from mixture_experts_routed_softmax_gb300.w4 import Linear4
    rng = np.random.default_rng(T)
    codes, scales = _codes(rng, 1, K, N, "int4", 64)
    x = torch.tensor(rng.standard_normal((T, K))).to(BF16)
    lin = Linear4(_weights4(codes, scales, "int4", 64))
    b = lin.buffers(T)
    b.ws.fill_(255)
    ref, bound = W.linear_bound(x.double().numpy(),
                                W.weights(codes, scales.double().numpy(), "int4", 64)[0])
    W.assert_within("y", _np(lin.apply(x.cuda(), b)), ref, bound)


def test_linear_any_scales_and_rows():
    """Scales of eight bits; infinities and NaN stay in their rows; no rows at all."""
    from mixture_experts_routed_softmax_gb300.w4 import Linear4
    rng = np.random.default_rng(2)
    for T in (4, 20, 200):
        codes, scales = _codes(rng, 1, 520, 72, "int4", 32, wide=True)
        q = _weights4(codes, scales, "int4", 32)
        x = torch.tensor(rng.standard_normal((T, 520))).to(BF16)
        Wd = W.weights(codes, scales.double().numpy(), "int4", 32)[0]
        ref, bound = W.linear_bound(x.double().numpy(), Wd)
        # many rows: code * scale rounded to bf16
        bound = bound + W.U_BF16 * (np.abs(x.double().numpy()) @ np.abs(Wd))
        lin = Linear4(q)
        b = lin.buffers(T)
        clean = lin.apply(x.cuda(), b).clone()
        W.assert_within("y", _np(clean), ref, bound)
        x2 = x.clone()
        x2[1, 7], x2[3, 100] = float("inf"), float("nan")
        y = lin.apply(x2.cuda(), b)
        keep = [r for r in range(T) if r not in (1, 3)]
        assert torch.equal(y[keep], clean[keep])
        assert torch.isnan(y[3]).all() and not torch.isfinite(y[1]).all()
    lin.apply(x.cuda()[:0], lin.buffers(0))
    with pytest.raises(ValueError):
        lin.apply(x.cuda()[:, :512], b)
    with pytest.raises(ValueError):
        lin.apply(x.cuda().float(), b)
    with pytest.raises(ValueError):
        lin.apply(x.cuda(), b, out=torch.empty(T, 72, device="cuda"))
    with pytest.raises(ValueError):
        Linear4(_weights4(*_codes(rng, 2, 64, 16, "int4", 32), "int4", 32))


# ----------------------------------------------------------------- experts --
CASES = {
    # name: (T, d, f, E, k, S, kind, group, act)
    "one": (1, 256, 128, 16, 4, 0, "int4", 64, None),
    "one_k1": (1, 72, 40, 3, 1, 0, "fp4", 32, None),
    "two_shared": (2, 136, 200, 9, 3, 2, "int4", 128, None),
    "eight": (8, 328, 264, 20, 4, 1, "fp4", 64, (7.0, 1.702, 1.0)),
    "few_experts": (30, 136, 72, 2, 2, 0, "int4", 32, None),
    "some": (64, 520, 392, 8, 3, 1, "fp4", 32, (1.0, 1.702, 1.0)),
    "all_experts": (3, 64, 64, 32, 32, 0, "int4", 32, None),
    "widest": (40, 64, 64, 1024, 30, 0, "fp4", 128, None),
    "many": (300, 264, 136, 12, 4, 1, "int4", 32, None),
    "very_many": (1500, 128, 72, 5, 2, 0, "fp4", 64, (7.0, 1.702, 1.0)),
    "skewed": (700, 136, 64, 16, 3, 1, "int4", 64, None),
}


def _experts_case(name, wide=False):
    from mixture_experts_routed_softmax_gb300.w4 import Experts4
    T, d, f, E, k, S, kind, group, act = CASES[name]
    rng = np.random.default_rng(sorted(CASES).index(name) + 50)
    ws, qs = [], []
    for K, N in ((d, f), (d, f), (f, d)):
        codes, scales = _codes(rng, E + S, K, N, kind, group, wide)
        qs.append(_weights4(codes, scales, kind, group))
        ws.append(W.weights(codes, scales.double().numpy(), kind, group))
    lean = 3.0 * rng.standard_normal(E) if name == "skewed" else 0.0
    idx = np.argsort(-(rng.standard_normal((T, E)) + lean), axis=1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    x = torch.tensor(rng.standard_normal((T, d))).to(BF16)
    return Experts4(*qs, k=k, E=E, act=act), ws, x, idx, w, act, E


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("name", sorted(CASES))
def test_experts(name, wide):
    ex, ws, x, idx, w, act, E = _experts_case(name, wide)
    T = x.shape[0]
    b = ex.buffers(T)
    b.ws.fill_(255)                    # NaN wherever something is read that was not written
    b.y.fill_(float("nan"))
    y = ex.forward(x.cuda(), torch.tensor(idx).cuda(), torch.tensor(w).cuda(), b)
    assert ex.status() == 0
    ref, bound = W.experts(x.double().numpy(), idx, w.astype(np.float64), *ws, E, act,
                           rounded=W.U_BF16 if wide else 0.0)
    W.assert_within(name, _np(y), ref, bound)
    first = y.clone()
    y = ex.forward(x.cuda(), torch.tensor(idx).cuda(), torch.tensor(w).cuda(), b)
    assert torch.equal(y, first)


@pytest.mark.parametrize("name", ["one", "one_k1", "two_shared"])
def test_experts_of_few_rows_keep_A(name):
    """T * k <= E: A stands as two bf16 numbers, the second the first's rounding, off by
    2^-8 of that: 2^-16 in all."""
    ex, ws, x, idx, w, act, E = _experts_case(name)
    y = ex.forward(x.cuda(), torch.tensor(idx).cuda(), torch.tensor(w).cuda(),
                   ex.buffers(x.shape[0]))
    ref, bound = W.experts(x.double().numpy(), idx, w.astype(np.float64), *ws, E, act,
                           a_rounded=2.0 ** -16)
    W.assert_within(name, _np(y), ref, bound)


@pytest.mark.parametrize("name", ["eight", "some", "many"])
def test_experts_odd_choices(name):
    """The same expert twice for a token; ids out of range: reported, their pairs left out."""
    ex, ws, x, idx, w, act, E = _experts_case(name)
    T, k = idx.shape
    idx[0, 1] = idx[0, 0]
    b = ex.buffers(T)
    run = lambda i: _np(ex.forward(x.cuda(), torch.tensor(i).cuda(),  # noqa: E731
                                   torch.tensor(w).cuda(), b))
    ref, bound = W.experts(x.double().numpy(), idx, w.astype(np.float64), *ws, E, act)
    W.assert_within("twice", run(idx), ref, bound)
    assert ex.status() == 0
    bad = idx.copy()
    bad[2, 0], bad[5, 2] = E, -1
    ref, bound = W.experts(x.double().numpy(), np.where((bad < 0) | (bad >= E), 10 ** 6, bad),
                           w.astype(np.float64), *ws, E, act)
    got = run(bad)
    assert ex.status() == 5
    W.assert_within("out of range", got, ref, bound)
    # every pair of a small batch out of range
    if T <= 8:
        got = run(np.full_like(bad, -1))
        assert ex.status() == 5
        if not ex.S:
            assert not got.any()


def test_experts_captured_streams_refusals():
    ex, ws, x, idx, w, act, E = _experts_case("some")
    T, k = idx.shape
    b = ex.buffers(T)
    xg, ig, wg = x.cuda(), torch.tensor(idx).cuda(), torch.tensor(w).cuda()
    ex.forward(xg, ig, wg, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ex.forward(xg, ig, wg, b)
    rng = np.random.default_rng(8)
    x2 = torch.tensor(rng.standard_normal(x.shape)).to(BF16)
    idx2 = np.ascontiguousarray(idx[::-1])
    xg.copy_(x2.cuda())
    ig.copy_(torch.tensor(idx2).cuda())
    graph.replay()
    ref, bound = W.experts(x2.double().numpy(), idx2, w.astype(np.float64), *ws, E, act)
    W.assert_within("captured", _np(b.y), ref, bound)
    want = b.y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b2 = ex.buffers(T)
    ex.forward(xg, ig, wg, b2, stream=side)
    side.synchronize()
    assert torch.equal(b2.y, want)
    empty = ex.buffers(0)
    ex.forward(xg[:0], ig[:0], wg[:0], empty)
    for args in ((xg.float(), ig, wg), (xg, ig.long(), wg), (xg, ig, wg.double()),
                 (xg[:-1], ig, wg), (xg[:, :-8], ig, wg)):
        with pytest.raises(ValueError):
            ex.forward(*args, b)


# --------------------------------------------------------------- the layer --
@pytest.mark.parametrize("T", [1, 20, 200])
@pytest.mark.parametrize("scored", [False, True])
def test_layer(T, scored):
    """Quantised from a MoELayer, behind either router: the routing is the layer's own,
    the rest that of the quantised experts on it."""
    import workloads
    from mixture_experts_routed_softmax_gb300.layer import MoELayer
    from mixture_experts_routed_softmax_gb300.router import Router
    E, k, S, act = 16, 3, 1, (7.0, 1.702, 1.0)
    wl = workloads.Workload("w4", T=T, d=136, f=72, E=E + S, k=k, align=16)
    inp = workloads.generate(wl)
    inp["w_router"] = inp["w_router"][:, :E].contiguous()
    inp["bias"] = None
    r = Router(E, k, score="sigmoid", n_groups=4, topk_groups=2, scale=2.5) if scored else None
    layer = MoELayer.from_inputs(inp, k, 16, act=act, router=r)
    q = layer.quantised("fp4", 32)
    x = inp["x"].cuda()
    b, full = q.buffers(T), layer.buffers(T, backward=False)
    y = q.forward(x, b)
    layer.forward(x, full)
    assert q.status() == 0
    assert torch.equal(b.topk_idx, full.topk_idx) and torch.equal(b.topk_w, full.topk_w)
    ws = [_np(m.dequantise()) for m in (q.experts.w_gate, q.experts.w_up, q.experts.w_down)]
    ref, bound = W.experts(inp["x"].double().numpy(), b.topk_idx.cpu().numpy(), _np(b.topk_w), *ws,
                           E, act)
    W.assert_within("y", _np(y), ref, bound)
    forced = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    q.forward(x, b, forced_idx=forced)
    assert torch.equal(b.topk_idx, forced)


@pytest.mark.parametrize("name", ["one", "one_k1", "two_shared", "eight", "some", "many"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_experts_out_of_range_whatever_the_weight(name, value):
    """A pair whose expert is out of range is left out, its weight with it: first and last slots,
    one token and several."""
    ex, ws, x, idx, w, act, E = _experts_case(name)
    T, k = idx.shape
    bad, wb = idx.copy(), w.copy()
    for t, j, e in ((0, 0, -1), (T - 1, k - 1, E), (T // 2, k // 2, 2 ** 31 - 1)):
        bad[t, j], wb[t, j] = e, value
    y = ex.forward(x.cuda(), torch.tensor(bad).cuda(), torch.tensor(wb).cuda(), ex.buffers(T))
    assert ex.status() == 5
    gone = (bad < 0) | (bad >= E)
    ref, bound = W.experts(x.double().numpy(), np.where(gone, 10 ** 6, bad),
                           np.where(gone, 0.0, w.astype(np.float64)), *ws, E, act)
    W.assert_within(name, _np(y), ref, bound)


# ------------------------------------------------------- scales of any size --
@pytest.mark.parametrize("kind,group", [("int4", 32), ("int4", 128), ("fp4", 64)])
@pytest.mark.parametrize("T,K,N", [(1, 520, 72), (5, 1032, 136), (12, 264, 520), (60, 520, 264),
                                   (300, 1032, 264)])
@pytest.mark.parametrize("power", [120, 9, -101, -110])
def test_linear_scales_of_any_size(kind, group, T, K, N, power):
    """Scales by 2^power: what fp32 holds comes out, however large or small the scales are. x goes
    the other way, so that nothing leaves fp32's range."""
    from mixture_experts_routed_softmax_gb300.w4 import Linear4
    rng = np.random.default_rng(T + K + N)
    codes, scales = _codes(rng, 1, K, N, kind, group)
    scales = (scales.double() * 2.0 ** power).to(BF16)
    # every third column's stay as they are: both kinds in one matrix
    scales[..., ::3] = (scales[..., ::3].double() * 2.0 ** -power).to(BF16)
    x = torch.tensor(rng.standard_normal((T, K)) * 2.0 ** (-power // 4)).to(BF16)
    Wd = W.weights(codes, scales.double().numpy(), kind, group)[0]
    q = _weights4(codes, scales, kind, group)
    np.testing.assert_array_equal(_np(q.dequantise())[0], Wd)
    for dtype in (BF16, torch.float32):
        lin = Linear4(q, out_dtype=dtype)
        b = lin.buffers(T)
        b.ws.fill_(255)
        y = _np(lin.apply(x.cuda(), b))
        ref, bound = W.linear_bound(x.double().numpy(), Wd, dtype is BF16)
        unit = np.where(np.arange(N) % 3 == 0, 1.0, 2.0 ** -power) * 2.0 ** (power // 4)
        W.assert_within("y", y * unit, ref * unit, bound * unit)


@pytest.mark.parametrize("name", ["one", "one_k1", "two_shared", "eight", "few_experts", "many",
                                  "very_many", "skewed"])
@pytest.mark.parametrize("which,power", [("gate", 12), ("gate", -104), ("up", 12), ("up", 100),
                                         ("up", -104), ("down", 120), ("down", -104)])
def test_experts_scales_of_any_size(name, which, power):
    """One of the three matrices by 2^power, every other expert of it."""
    from mixture_experts_routed_softmax_gb300.w4 import Experts4
    T, d, f, E, k, S, kind, group, act = CASES[name]
    rng = np.random.default_rng(sorted(CASES).index(name) + 80)
    ws, qs = [], []
    for m, (K, N) in (("gate", (d, f)), ("up", (d, f)), ("down", (f, d))):
        codes, scales = _codes(rng, E + S, K, N, kind, group)
        if m == which:
            scales[::2] = (scales[::2].double() * 2.0 ** power).to(BF16)
        qs.append(_weights4(codes, scales, kind, group))
        ws.append(W.weights(codes, scales.double().numpy(), kind, group))
    # a token's experts alike, so that none hides behind the others
    first = rng.integers(0, 2, (T, 1))
    rank = np.argsort(rng.standard_normal((T, E)) + 100.0 * (np.arange(E) % 2 == first), axis=1)
    idx = rank[:, ::-1][:, :k].astype(np.int32)
    idx = np.where(idx % 2 == first, idx, first % E).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    x = torch.tensor(rng.standard_normal((T, d))).to(BF16)
    ex = Experts4(*qs, k=k, E=E, act=act)
    b = ex.buffers(T)
    b.ws.fill_(255)
    y = _np(ex.forward(x.cuda(), torch.tensor(idx).cuda(), torch.tensor(w).cuda(), b))
    assert ex.status() == 0
    ref, bound = W.experts(x.double().numpy(), idx, w.astype(np.float64), *ws, E, act)
    unit = np.ones((T, 1))
    if which == "down" or (which == "up" and act is None) or (which == "gate" and power < 0):
        unit = np.where(first == 0, 2.0 ** -power, 1.0) if not S else unit
    W.assert_within(name, y * unit, ref * unit, bound * unit)



def test_scales_that_are_not_finite():
    """An infinite scale or NaN shows in its column and nowhere else, few rows or many."""
    from mixture_experts_routed_softmax_gb300.w4 import Linear4
    rng = np.random.default_rng(4)
    for kind in ("int4", "fp4"):
        codes, scales = _codes(rng, 1, 264, 136, kind, 64)
        scales[0, 1, 5], scales[0, 4, 77], scales[0, 0, 130] = float("inf"), float("nan"), -3e38
        clean = scales.clone()
        clean[0, :, [5, 77]] = 1.0
        for T in (1, 6, 200, 600):
            x = torch.tensor(rng.standard_normal((T, 264)) * 2.0 ** -8).to(BF16)
            lin = Linear4(_weights4(codes, scales, kind, 64), out_dtype=torch.float32)
            y = _np(lin.apply(x.cuda(), lin.buffers(T)))
            bad = np.isin(np.arange(136), [5, 77])
            assert not np.isfinite(y[:, bad]).any()
            Wd = W.weights(codes, clean.double().numpy(), kind, 64)[0]
            ref, bound = W.linear_bound(x.double().numpy(), Wd, False)
            # 3e38's code * scale rounded to bf16, where it stays below bf16's top
            bound = bound + W.U_BF16 * (np.abs(x.double().numpy()) @ np.abs(Wd))
            keep = ~bad & (np.abs(Wd).max(0) < W.BF16_MAX)
            W.assert_within("y", y[:, keep], ref[:, keep], bound[:, keep])


@pytest.mark.parametrize("what", ["quantise", "from_codes", "dequantise"])
def test_made_on_another_stream(what):
    """What a call on another stream allocates is memory that work on the current one, not over yet,
    may still write to."""
    from mixture_experts_routed_softmax_gb300.w4 import Weights4
    rng = np.random.default_rng(6)
    E, K, N = 4, 1024, 768
    codes, scales = _codes(rng, E, K, N, "int4", 32)
    cg, sg = torch.tensor(codes).cuda(), scales.cuda()
    w = torch.tensor(rng.standard_normal((E, K, N)), dtype=torch.float32).to(BF16).cuda()
    make = {"quantise": lambda s: Weights4.quantise(w, "int4", 32, stream=s),
            "from_codes": lambda s: Weights4.from_codes(cg, sg, "int4", 32, stream=s),
            "dequantise": None}[what]
    have = Weights4.from_codes(cg, sg, "int4", 32)
    want = (make(None) if make else have).dequantise()
    nc, ns = have.codes.numel(), have.scales.numel()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        junk = [torch.empty(nc, dtype=torch.uint8, device="cuda"),
                torch.empty(ns, dtype=BF16, device="cuda"), torch.empty_like(want)]
        torch.cuda._sleep(20_000_000)
        for j in junk:
            j.fill_(77)
        del junk, j
        got = make(side).dequantise(stream=side) if make else have.dequantise(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del got
