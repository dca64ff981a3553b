"""The scored router on the GPU against its 64-bit reference (router_ref.py):
choice, weights, gradient, the layer with such a router, and the uses that can
go wrong: near ties, masks, odd sizes, unaligned rows, captured calls.

The choice has to be equal. Weights and gradients are held to the error that fp32
arithmetic of these formulas can make (router_ref.half_steps, counted there)."""
import numpy as np
import pytest
import torch

import router_ref as R

pytestmark = pytest.mark.gpu

CASES = {
    # name: (T, E, k, score, kw)
    "one": (1, 256, 8, "sigmoid", dict(n_groups=8, topk_groups=4, scale=2.5, balance=True)),
    "groups_sig": (70, 256, 8, "sigmoid", dict(n_groups=8, topk_groups=4, balance=True)),
    "groups_soft": (70, 160, 6, "softmax", dict(n_groups=8, topk_groups=3, group_rank=1)),
    "groups_two": (33, 160, 6, "softmax", dict(n_groups=16, topk_groups=5)),
    "groups_balance_one": (33, 64, 6, "softmax", dict(n_groups=32, topk_groups=5, group_rank=1,
                                                      balance=True)),
    "groups_of_one": (9, 40, 4, "sigmoid", dict(n_groups=40, topk_groups=7)),
    "every_group": (20, 60, 4, "sigmoid", dict(n_groups=5, topk_groups=5, balance=True)),
    "plain_soft": (100, 32, 4, "softmax", {}),
    "plain_sig": (41, 7, 3, "sigmoid", dict(scale=0.5)),
    "raw_soft": (67, 512, 10, "softmax", dict(renormalise=False, balance=True)),
    "raw_sig": (67, 20, 20, "sigmoid", dict(renormalise=False)),
    "odd_E": (50, 61, 5, "softmax", dict(balance=True)),
    "two_experts": (6, 2, 1, "sigmoid", dict(balance=True)),
    "one_expert": (6, 1, 1, "softmax", dict(renormalise=False)),
    "all_chosen": (5, 32, 32, "sigmoid", {}),
    "widest": (19, 1024, 32, "softmax", dict(n_groups=64, topk_groups=9, balance=True)),
    "widest_sig": (19, 1000, 32, "sigmoid", dict(balance=True)),
}


def _case(name):
    T, E, k, score, kw = CASES[name]
    rng = np.random.default_rng(sorted(CASES).index(name))
    l = (1.5 * rng.standard_normal((T, E)) + rng.standard_normal(E)).astype(np.float32)
    kw = dict(kw, score=score)
    bal = None
    if kw.pop("balance", False):
        bal = (0.1 * rng.standard_normal(E) * (1 if score == "sigmoid" else 4 / E)).astype(
            np.float32)
    return T, E, k, kw, l, bal, rng


def _router(E, k, kw, bal):
    from mixture_experts_routed_softmax_gb300.router import Router
    return Router(E, k, balance=None if bal is None else torch.tensor(bal).cuda(), **kw)


def _choice_args(kw):
    return {n: v for n, v in kw.items() if n in ("score", "n_groups", "topk_groups", "group_rank")}


def _weight_args(kw):
    return {n: v for n, v in kw.items() if n in ("score", "renormalise", "scale")}


def _check_choice(l, k, kw, bal, idx, w, forced=None):
    E = l.shape[1]
    for t in range(l.shape[0]):
        want = R.choose(l[t], k, balance=bal, **_choice_args(kw)) if forced is None else forced[t]
        np.testing.assert_array_equal(idx[t], want, err_msg=f"token {t}")
        ref = R.weights(l[t], want, **_weight_args(kw))
        tol = R.half_steps(E, l[t]) * R.EPS32 * np.abs(ref) + 1e-37
        assert np.all(np.abs(w[t] - ref) <= tol), (t, w[t], ref)


def _check_grad(dw, l, idx, kw, d, base=None):
    E = l.shape[1]
    for t in range(l.shape[0]):
        ref, mag = R.backward(dw[t], l[t], idx[t], **_weight_args(kw))
        # a product of two scores and a sum of k terms beside the scores' own errors
        tol = (2 * R.half_steps(E, l[t]) + len(idx[t])) * R.EPS32 * mag + 1e-37
        if base is not None:                 # added to: the sum's rounding
            ref = ref + base[t]
            tol = tol + 4 * R.EPS32 * (np.abs(base[t]) + 2 * mag)
        assert np.all(np.abs(d[t] - ref) <= tol), (t, np.abs(d[t] - ref).max())


@pytest.mark.parametrize("name", sorted(CASES))
def test_choice_and_gradient(name):
    T, E, k, kw, l, bal, rng = _case(name)
    r = _router(E, k, kw, bal)
    b = r.buffers(T, backward=True)
    lg = torch.tensor(l).cuda()
    r.select(lg, b)
    idx = b.topk_idx.cpu().numpy()
    _check_choice(l, k, kw, bal, idx, b.topk_w.cpu().numpy().astype(np.float64))
    dw = rng.standard_normal((T, k)).astype(np.float32)
    b.d_logits.fill_(float("nan"))
    d = r.select_bwd(torch.tensor(dw).cuda(), lg, b).cpu().numpy().astype(np.float64)
    _check_grad(dw, l, idx, kw, d)
    base = rng.standard_normal((T, E)).astype(np.float32)
    b.d_logits.copy_(torch.tensor(base))
    d = r.select_bwd(torch.tensor(dw).cuda(), lg, b, accumulate=True).cpu().numpy().astype(float)
    _check_grad(dw, l, idx, kw, d, base.astype(np.float64))
    assert r.lib.moe_status(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_near_ties(score, groups):
    """Choice values nearer to one another than fp32 can tell, and equal ones: the
    order is that of 64-bit scores, ties go to the lower index. The balance moves
    half of the experts by what their logits lack, to within a step of fp32."""
    rng = np.random.default_rng(5)
    T, E, k = 64, 64, 8
    l = np.repeat(rng.standard_normal((T, 1)), E, 1).astype(np.float32)
    # logits a few steps of fp32 apart, many of them equal
    step = rng.integers(-2, 3, (T, E))
    for s in range(1, 3):
        l = np.where(np.abs(step) >= s, np.nextafter(l, np.where(step > 0, np.inf, -np.inf)
                                                     .astype(np.float32)), l)
    bal = np.where(rng.random(E) < 0.5, 0.0, 2.0 ** -26).astype(np.float32)
    kw = dict(score=score, n_groups=groups, topk_groups=(groups + 1) // 2)
    r = _router(E, k, kw, bal)
    b = r.buffers(T)
    r.select(torch.tensor(l).cuda(), b)
    _check_choice(l, k, kw, bal, b.topk_idx.cpu().numpy(), b.topk_w.cpu().numpy().astype(float))
    # all equal: the lowest indices
    lz = np.zeros((3, E), dtype=np.float32)
    lz[1] = -0.0
    lz[2, ::2] = -0.0
    for balance in (None, np.zeros(E, dtype=np.float32)):
        r = _router(E, k, kw, balance)
        b = r.buffers(3)
        r.select(torch.tensor(lz).cuda(), b)
        assert b.topk_idx.cpu().tolist() == [list(range(k))] * 3


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("balance", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_masks(score, renormalise, balance, groups):
    """Masked experts (-inf, NaN), the lowest value, rows with nothing left, +inf,
    tiny scores: weights, choice and gradients stay finite and exact."""
    rng = np.random.default_rng(7)
    E, k, inf = 32, 6, np.inf
    rows = [np.full(E, -inf), np.full(E, np.nan), np.full(E, np.finfo(np.float32).min)]
    one = np.full(E, -inf)
    one[17] = 0.5
    rows.append(one)
    some = rng.standard_normal(E)
    some[rng.permutation(E)[:20]] = -inf
    some[3] = np.nan
    rows.append(some)
    low = rng.standard_normal(E)
    low[8:] = np.finfo(np.float32).min
    rows.append(low)
    top = rng.standard_normal(E)
    top[[4, 20]] = inf
    rows.append(top)
    rows.append(rng.standard_normal(E) - 95.0)           # sigmoid scores below fp32's normal range
    rows.append(rng.standard_normal(E) - 300.0)
    rows.append(rng.standard_normal(E) + 30.0)
    l = np.array(rows, dtype=np.float32)
    bal = (0.05 * rng.standard_normal(E)).astype(np.float32) if balance else None
    kw = dict(score=score, renormalise=renormalise, n_groups=groups, topk_groups=2 if groups > 1
              else 1)
    r = _router(E, k, kw, bal)
    T = len(rows)
    b = r.buffers(T, backward=True)
    lg = torch.tensor(l).cuda()
    r.select(lg, b)
    idx, w = b.topk_idx.cpu().numpy(), b.topk_w.cpu().numpy().astype(np.float64)
    _check_choice(l, k, kw, bal, idx, w)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    d = r.select_bwd(torch.tensor(dw).cuda(), lg, b).cpu().numpy().astype(np.float64)
    assert np.isfinite(d).all() and np.isfinite(w).all()
    _check_grad(dw, l, idx, kw, d)
    assert not d[:2].any() and not w[:2].any()


def test_caller_chosen():
    """A caller's choice: any order, the same expert twice, ids out of range."""
    rng = np.random.default_rng(9)
    T, E, k = 12, 24, 5
    l = rng.standard_normal((T, E)).astype(np.float32)
    forced = rng.integers(0, E, (T, k)).astype(np.int32)
    forced[3] = [7, 7, 2, 7, 2]
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for kw in (dict(score="sigmoid"), dict(score="softmax", renormalise=False),
               dict(score="sigmoid", renormalise=False)):
        r = _router(E, k, kw, None)
        b = r.buffers(T, backward=True)
        lg = torch.tensor(l).cuda()
        r.select(lg, b, forced_idx=torch.tensor(forced).cuda())
        _check_choice(l, k, kw, None, b.topk_idx.cpu().numpy(), b.topk_w.cpu().numpy(), forced)
        d = r.select_bwd(torch.tensor(dw).cuda(), lg, b).cpu().numpy()
        _check_grad(dw, l, forced, kw, d)
        stream = torch.cuda.current_stream().cuda_stream
        assert r.lib.moe_status(stream) == 0
        bad = forced.copy()
        bad[5, 1], bad[6, 2] = E, -3
        r.select(lg, b, forced_idx=torch.tensor(bad).cuda())
        assert r.lib.moe_status(stream) == 5
        w = b.topk_w.cpu().numpy()
        assert w[5, 1] == 0 and w[6, 2] == 0
        np.testing.assert_array_equal(w[:5], R32(l, forced, kw, w)[:5])
        r.select_bwd(torch.tensor(dw).cuda(), lg, b)
        assert r.lib.moe_status(stream) == 5


def R32(l, forced, kw, w):
    """The GPU's own weights where they are within the reference's bound."""
    for t in range(5):
        ref = R.weights(l[t], forced[t], **_weight_args(kw))
        assert np.all(np.abs(w[t] - ref) <= R.half_steps(l.shape[1], l[t]) * R.EPS32 * ref)
    return w


def test_unaligned_rows_streams_and_refusals():
    T, E, k, kw, l, bal, rng = _case("groups_sig")
    r = _router(E, k, kw, bal)
    b = r.buffers(T, backward=True)
    store = torch.zeros(T * E + 1, device="cuda")
    lg = store[1:].view(T, E)                # packed, but 4 bytes off a 16-byte boundary
    lg.copy_(torch.tensor(l))
    r.select(lg, b)
    ref, ref_w = b.topk_idx.clone(), b.topk_w.clone()
    _check_choice(l, k, kw, bal, ref.cpu().numpy(), b.topk_w.cpu().numpy())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b2 = r.buffers(T, backward=True)
    r.select(lg.clone(), b2, stream=side)
    side.synchronize()
    assert torch.equal(b2.topk_idx, ref) and torch.equal(b2.topk_w, ref_w)
    # nothing to do
    r.select(lg[:0], r.buffers(0))
    for bad in (lg.double(), lg[:, ::2], lg[:5], lg.t().contiguous().t(), lg.cpu()):
        with pytest.raises(ValueError):
            r.select(bad, b)
    with pytest.raises(ValueError):
        r.select_bwd(b.topk_w, lg, r.buffers(T))
    with pytest.raises(ValueError):
        r.select(lg, b, forced_idx=b.topk_idx.long())


def test_captured():
    """A captured choice and gradient serve later logits and a later balance."""
    T, E, k, kw, l, bal, rng = _case("groups_sig")
    r = _router(E, k, kw, bal)
    b = r.buffers(T, backward=True)
    lg, dw = torch.tensor(l).cuda(), torch.zeros(T, k, device="cuda")
    r.select(lg, b)
    r.select_bwd(dw, lg, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.select(lg, b)
        r.select_bwd(dw, lg, b)
    l2 = (l[::-1] * 0.7).copy()
    bal2 = (bal * -2).astype(np.float32)
    dw2 = rng.standard_normal((T, k)).astype(np.float32)
    lg.copy_(torch.tensor(l2))
    dw.copy_(torch.tensor(dw2))
    r.balance.copy_(torch.tensor(bal2))
    graph.replay()
    idx = b.topk_idx.cpu().numpy()
    _check_choice(l2, k, kw, bal2, idx, b.topk_w.cpu().numpy().astype(np.float64))
    _check_grad(dw2, l2, idx, kw, b.d_logits.cpu().numpy().astype(np.float64))


# ----------------------------------------------------------------- the layer --
LAYERS = {
    # name: (T, d, f, E, k, S, score, kw)
    "one_token": (1, 64, 64, 16, 2, 0, "sigmoid", dict(n_groups=4, topk_groups=2, balance=True)),
    "few": (24, 128, 64, 60, 4, 1, "softmax", dict(renormalise=False)),
    "many_sig": (300, 200, 136, 32, 4, 1, "sigmoid", dict(n_groups=8, topk_groups=3, scale=2.5,
                                                          balance=True)),
    "many_raw": (300, 136, 72, 20, 3, 0, "softmax", dict(renormalise=False, balance=True)),
    "wide": (130, 64, 64, 520, 8, 0, "softmax", dict(renormalise=False, scale=2.0)),
}


def _bf16_close(name, got, ref, mag):
    """got (bf16) against ref: half a step of bf16 and fp32 sums of terms of
    magnitude mag, up to 2^13 additions deep in blocks (2^-17 of mag covers them)."""
    tol = np.abs(ref) * 2.0 ** -8 + mag * 2.0 ** -17 + 1e-30
    worst = float((np.abs(got - ref) / tol).max())
    assert worst <= 1.0, f"{name}: {worst}"


@pytest.mark.parametrize("logits_loss", [False, True])
@pytest.mark.parametrize("name", sorted(LAYERS))
def test_layer(name, logits_loss):
    """Forward and backward of a layer with a scored router: every step of the
    router against 64 bits on what the steps before it left on the GPU."""
    import workloads
    from mixture_experts_routed_softmax_gb300.layer import MoELayer
    T, d, f, E, k, S, score, kw = LAYERS[name]
    kw = dict(kw, score=score)
    wl = workloads.Workload(name, T=T, d=d, f=f, E=E + S, k=k, align=16, zipf_s=None)
    inp = workloads.generate(wl)
    inp["w_router"] = (inp["w_router"][:, :E] * 20).contiguous()
    gen = torch.Generator().manual_seed(4)
    inp["bias"] = 0.3 * torch.randn(E, generator=gen)
    bal = None
    if kw.pop("balance", False):
        bal = (0.02 * torch.randn(E, generator=gen)).numpy()
    r = _router(E, k, kw, bal)
    layer = MoELayer.from_inputs(inp, k, 16, router=r)
    b = layer.buffers(T, logits_loss=logits_loss)
    x, dy = inp["x"].cuda(), inp["dy"].cuda()
    y = layer.forward(x, b)
    assert layer.status() == 0
    X, W = inp["x"].double().numpy(), inp["w_router"].double().numpy()
    l = b.logits.cpu().numpy().astype(np.float64)
    mag = np.abs(X) @ np.abs(W) + 1
    # fp32 sums of exact products: at most d additions one after the other
    assert np.all(np.abs(l - (X @ W + inp["bias"].double().numpy())) <= mag * d * R.EPS32)
    l32 = b.logits.cpu().numpy()
    _check_choice(l32, k, kw, bal, b.topk_idx.cpu().numpy(), b.topk_w.cpu().numpy().astype(float))
    # the combine of what the experts gave
    yp, dst = b.yp.cpu().double().numpy(), b.dst_row.cpu().numpy()
    w = b.topk_w.cpu().double().numpy()
    rows = yp[dst[:T * k]].reshape(T, k, d)
    terms = np.concatenate([rows * w[..., None]] +
                           [yp[dst[T * k + s * T:T * k + (s + 1) * T]][:, None] for s in range(S)],
                           axis=1)
    _bf16_close("y", y.cpu().double().numpy(), terms.sum(1), np.abs(terms).sum(1))
    base = np.zeros((T, E))
    if logits_loss:
        base = torch.randn(T, E, generator=gen).numpy().astype(np.float64) * 0.1
        b.d_logits.copy_(torch.tensor(base))
    layer.expert_bwd(dy, b)
    layer.route_bwd(b, accumulate=logits_loss)
    assert layer.status() == 0
    dw, idx = b.d_topk_w.cpu().numpy(), b.topk_idx.cpu().numpy()
    dl = b.d_logits.cpu().numpy().astype(np.float64)
    _check_grad(dw, l32, idx, kw, dl, base.astype(np.float32) if logits_loss else None)
    # dx: the permute's transpose and the router's term, rounded once
    dxp = b.dxp.cpu().double().numpy()
    terms = np.concatenate([dxp[dst[:T * k]].reshape(T, k, d)] +
                           [dxp[dst[T * k + s * T:T * k + (s + 1) * T]][:, None]
                            for s in range(S)], axis=1)
    _bf16_close("dx", b.dx.cpu().double().numpy(), terms.sum(1) + dl @ W.T,
                np.abs(terms).sum(1) + np.abs(dl) @ np.abs(W.T))
    got = b.dw_router.cpu().double().numpy()
    # T additions, the three bf16 parts of dl beside one another (3 sums)
    assert np.all(np.abs(got - X.T @ dl) <= (T + 8) * R.EPS32 * (np.abs(X.T) @ np.abs(dl)) + 1e-30)
    got = b.dbias.cpu().double().numpy()
    assert np.all(np.abs(got - dl.sum(0)) <= (T + 8) * R.EPS32 * np.abs(dl).sum(0) + 1e-30)
    # dx added to what is there (dxp not given)
    dx0 = torch.randn(T, d, generator=gen).to(torch.bfloat16)
    b.dx.copy_(dx0)
    if logits_loss:
        b.d_logits.copy_(torch.tensor(base))
    layer.route_bwd(b, fused=False, accumulate=logits_loss)
    _bf16_close("dx added", b.dx.cpu().double().numpy(), dx0.double().numpy() + dl @ W.T,
                np.abs(dx0.double().numpy()) + np.abs(dl) @ np.abs(W.T))


def test_softmax_router_equals_the_layers_own():
    """A renormalised softmax router chooses and weights as the layer without one."""
    import workloads
    from mixture_experts_routed_softmax_gb300.layer import MoELayer
    from mixture_experts_routed_softmax_gb300.router import Router
    wl = workloads.Workload("same", T=200, d=128, f=64, E=24, k=4, align=16)
    inp = workloads.generate(wl)
    plain = MoELayer.from_inputs(inp, 4, 16)
    scored = MoELayer.from_inputs(inp, 4, 16, router=Router(24, 4))
    x = inp["x"].cuda()
    for n in (200, 7):
        a, b = plain.buffers(n), scored.buffers(n)
        plain.forward(x[:n], a)
        scored.forward(x[:n], b)
        assert torch.equal(a.logits, b.logits) and torch.equal(a.topk_idx, b.topk_idx)
        assert torch.allclose(a.topk_w, b.topk_w, rtol=2.0 ** -20, atol=0)
    with pytest.raises(ValueError):
        MoELayer.from_inputs(inp, 4, 16, router=Router(32, 4))
    with pytest.raises(ValueError):
        scored.decode_fwd(x[:1], scored.decode_buffers(1))
    with pytest.raises(ValueError):
        plain.route_bwd(plain.buffers(200), accumulate=True)


# Experts of which two a group count, the balances +a and -a on them: a rank is the difference of
# two rounded values, all of whose bits it may lose.
CANCEL = {
    # name: (E, n_groups, topk_groups, k, score, logits around, their spread, sizes of a); k =
    # 2 topk_groups and no two a alike: nothing near another value but the groups' border
    "pairs": (8, 4, 2, 4, "sigmoid", -14.0, 0.03, (0.1,)),
    "whole_lanes": (256, 8, 3, 6, "sigmoid", -13.0, 0.03, (0.1, 0.5, 1.0)),
    "odd_groups": (96, 16, 5, 10, "sigmoid", -12.0, 0.02, (0.75, 1.0, 4.0)),
    "softmax_lanes": (256, 8, 3, 6, "softmax", 0.0, 1e-4, (1.0, 4.0)),
    "softmax_odd": (60, 20, 7, 14, "softmax", 0.0, 2e-5, (1.0, 3.0)),
    "widest": (1024, 64, 9, 18, "sigmoid", -12.0, 0.02, (0.5, 1.0)),
}


def _cancelling(name, masks, T=200):
    """Logits, balance and choice arguments; tokens that 64 bits themselves leave open (a
    border within 1e-14, or 2^-36 of the largest softmax score) are left out."""
    E, n, tg, k, score, mid, spread, sizes = CANCEL[name]
    rng = np.random.default_rng(sorted(CANCEL).index(name) + 90)
    gs = E // n
    l = (mid + 0.5 * rng.standard_normal((T, 1)) + spread * rng.standard_normal((T, E))).astype(
        np.float32)
    bal = np.full((n, gs), -8.0, dtype=np.float32)
    a = rng.choice(sizes, n) * (1 + np.arange(n) / 256)
    bal[:, 0], bal[:, 1] = a, -a
    at = rng.permuted(np.tile(np.arange(gs), (n, 1)), axis=1)
    bal = np.take_along_axis(bal, at, 1).reshape(E)
    if masks:
        rest = np.tile(bal == -8.0, (T, 1))
        l[rest & (rng.random((T, E)) < 0.5)] = -np.inf
        l[rest & (rng.random((T, E)) < 0.1)] = np.nan
        l[np.arange(0, T, 3), :gs] = -np.inf               # a group without anyone
    kw = dict(score=score, n_groups=n, topk_groups=tg)
    keep = []
    for t in range(T):
        s, live = R.scores(l[t], score)
        c = np.where(live, s + bal.astype(np.float64), -np.inf).reshape(n, gs)
        best = np.sort(c, 1)[:, ::-1][:, :2]
        rank = np.sort(np.where(np.isinf(best[:, 1]), best[:, 0], best.sum(1)))[::-1]
        if rank[tg - 1] - rank[tg] > max(1e-14, 2.0 ** -36 * s.max() * (score == "softmax")):
            keep.append(t)
    return l[keep], bal, k, kw


@pytest.mark.parametrize("masks", [False, True])
@pytest.mark.parametrize("name", sorted(CANCEL))
def test_ranks_that_nearly_cancel(name, masks):
    l, bal, k, kw = _cancelling(name, masks)
    T, E = l.shape
    assert T > 100
    r = _router(E, k, kw, bal)
    b = r.buffers(T)
    r.select(torch.tensor(l).cuda(), b)
    got = b.topk_idx.cpu().numpy()
    for t in range(T):
        want = R.choose(l[t], k, balance=bal, **kw)
        np.testing.assert_array_equal(got[t], want, err_msg=f"token {t}")


@pytest.mark.parametrize("l,bal,groups,topk,kept", [
    ([-15.048437, -15.0238905, -14.990487, -14.968859, -14.963728, -14.998065, -14.982132,
      -14.98184], [0.1, -0.1] * 4, 4, 2, [1, 2]),
    ([-12.010436, -11.995859, -11.998528, -12.006201], [1.0, -1.0, 0.75, -0.75], 2, 1, [1])])
def test_ranks_that_nearly_cancel_by_hand(l, bal, groups, topk, kept):
    l, bal = np.array([l], dtype=np.float32), np.array(bal, dtype=np.float32)
    k = 2 * topk
    r = _router(l.shape[1], k, dict(score="sigmoid", n_groups=groups, topk_groups=topk), bal)
    b = r.buffers(1)
    r.select(torch.tensor(l).cuda(), b)
    assert sorted(set(b.topk_idx.cpu()[0].tolist())) == sorted(
        e for g in kept for e in (2 * g, 2 * g + 1))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk,k", [(32, 1, 1, 4), (64, 1, 1, 4), (256, 1, 1, 8), (256, 8, 4, 8),
                                             (60, 20, 7, 5), (1000, 1, 1, 31), (1024, 1, 1, 32)])
def test_balance_of_any_size(score, E, groups, topk, k):
    """A balance of +inf puts experts first, in index order, -inf or NaN last; the largest finite
    ones leave no scores to tell apart."""
    rng = np.random.default_rng(E + groups)
    l = rng.standard_normal((40, E)).astype(np.float32)
    l[5:9, rng.random(E) < 0.3] = -np.inf
    kw = dict(score=score, n_groups=groups, topk_groups=topk)
    big = float(np.finfo(np.float32).max)
    for n, value in ((k // 2, np.inf), (k, np.inf), (k + 1, np.inf), (E // 2, np.inf), (E, np.inf),
                     (E // 2, -np.inf), (E // 2, np.nan), (E, -np.inf), (E, np.nan), (k + 3, big),
                     (E, big), (E, -big)):
        bal = (0.01 * rng.standard_normal(E)).astype(np.float32)
        bal[rng.permutation(E)[:n]] = value
        r = _router(E, k, kw, bal)
        b = r.buffers(len(l))
        r.select(torch.tensor(l).cuda(), b)
        assert r.lib.moe_status(torch.cuda.current_stream().cuda_stream) == 0
        with np.errstate(over="ignore"):
            _check_choice(l, k, kw, bal, b.topk_idx.cpu().numpy(), b.topk_w.cpu().numpy())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_loss_without_room(score):
    """A backward that is refused for its buffers has added nothing to the logits' gradient."""
    import workloads
    from mixture_experts_routed_softmax_gb300.layer import MoELayer
    wl = workloads.Workload("room", T=40, d=64, f=64, E=16, k=3, align=16)
    inp = workloads.generate(wl)
    layer = MoELayer.from_inputs(inp, 3, 16, router=_router(16, 3, dict(score=score), None))
    b = layer.buffers(40)
    layer.forward(inp["x"].cuda(), b)
    layer.expert_bwd(inp["dy"].cuda(), b)
    b.d_logits.fill_(0.25)
    with pytest.raises(ValueError):
        layer.route_bwd(b, accumulate=True)
    assert bool((b.d_logits == 0.25).all())
    layer.route_bwd(b)
    with pytest.raises(ValueError):
        layer.route_bwd(layer.buffers(40, backward=False), x=b.x)
    assert layer.status() == 0


def _gradient_by_pairs(dw, l, idx, score, renormalise, scale):
    """One token's gradient as sums over pairs, p_e sum_f p_f (g_e - g_f), in 64 bits, where no
    difference of nearly equal sums appears; and the magnitudes that fp32 rounds: with * the largest
    chosen score (renormalised weights), or a chosen expert of more than half of the row,
    p_e (|g_e - g_*| + sum_{f not *} p_f |g_f - g_*|), each g_f - g_* of f that is not chosen
    or of raw scores as |g_f| + |g_*|."""
    s, live = R.scores(l, score)
    out, mag = np.zeros(len(s)), np.zeros(len(s))
    if renormalise:
        q = R.chosen_scores(l, idx, score, True)
        g = np.where(live[idx], np.asarray(dw, dtype=np.float64), 0.0)
        top = g[np.argmax(np.where(live[idx], np.asarray(l, dtype=np.float64)[idx], -np.inf))]
        for j, e in enumerate(idx):
            f = 1.0 / (1.0 + np.exp(float(l[e]))) if score == "sigmoid" else 1.0
            if live[e]:
                out[e] += scale * q[j] * f * (q * (g[j] - g)).sum()
                mag[e] += abs(scale) * q[j] * f * (abs(g[j] - top) + (q * np.abs(g - top)).sum())
        return out, mag
    G = np.zeros(len(s))
    np.add.at(G, idx[live[idx]], np.asarray(dw, dtype=np.float64)[live[idx]])
    out = scale * s * (s[None] * (G[:, None] - G[None])).sum(1)
    chosen = np.zeros(len(s), dtype=bool)
    chosen[idx] = True
    mag = s * (np.abs(G) + (s * np.abs(G)).sum())
    star = int(np.argmax(s))
    if chosen[star] and s[star] > 0.5:
        rest = np.delete(s * (np.abs(G) + abs(G[star])), star).sum()
        mag = np.where(chosen, s * (np.abs(G - G[star]) + rest), mag)
    return out, abs(scale) * mag


@pytest.mark.parametrize("score,renormalise", [("softmax", True), ("sigmoid", True),
                                               ("softmax", False)])
@pytest.mark.parametrize("E,k", [(24, 2), (61, 5), (256, 8), (520, 32)])
def test_gradient_of_peaked_rows(score, renormalise, E, k):
    """One expert has nearly the whole row, or the g of several are nearly alike: what is left of
    the differences is the gradient, not rounding."""
    rng = np.random.default_rng(E + k)
    T = 60
    l = rng.standard_normal((T, E)).astype(np.float32)
    l -= np.linspace(0, 3, T, dtype=np.float32)[:, None] * (10 if score == "sigmoid" else 1)
    at = rng.integers(0, E, T)
    l[np.arange(T), at] += np.linspace(0, 40, T).astype(np.float32)
    l[rng.random((T, E)) < 0.05] = -np.inf
    kw = dict(score=score, renormalise=renormalise, scale=2.5)
    r = _router(E, k, kw, None)
    b = r.buffers(T, backward=True)
    lg = torch.tensor(l).cuda()
    r.select(lg, b)
    idx = b.topk_idx.cpu().numpy()
    idx[::7, k - 1] = idx[::7, 0]                  # an expert twice
    idx[5::7] = rng.integers(0, E, idx[5::7].shape)    # a caller's choice, without the largest
    b.topk_idx.copy_(torch.tensor(idx))
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dw[::2] = (1 + 1e-5 * dw[::2]).astype(np.float32)
    d = r.select_bwd(torch.tensor(dw).cuda(), lg, b).cpu().numpy().astype(np.float64)
    base = (1e-6 * rng.standard_normal((T, E))).astype(np.float32)
    b.d_logits.copy_(torch.tensor(base))
    added = r.select_bwd(torch.tensor(dw).cuda(), lg, b, accumulate=True).cpu().numpy()
    for t in range(T):
        ref, mag = _gradient_by_pairs(dw[t], l[t], idx[t], **kw)
        tol = (2 * R.half_steps(E, l[t]) + k) * R.EPS32 * mag + 1e-37
        assert np.all(np.abs(d[t] - ref) <= tol), (t, (np.abs(d[t] - ref) / tol).max())
        # added to: the rounding of the sum, once
        assert np.all(np.abs(added[t] - base[t] - d[t]) <=
                      2 * R.EPS32 * (np.abs(base[t]) + np.abs(d[t])) + 1e-37), t


@pytest.mark.parametrize("E", [32, 100, 512, 1024])
def test_near_ties_below_a_far_maximum(E):
    """One expert far above equal others, where the arguments' roundings weigh most and all go one
    way, and a balance that leaves the order to the last half steps of fp32."""
    rng = np.random.default_rng(E)
    T = 64
    far = 1.0 + np.log(E) - np.log(np.log(E))        # about f + 1 of f e^(f + 1) = E - 1
    open_ = 0
    for half_steps in range(-24, 25, 3):
        l = np.full((T, E), -far / 2, dtype=np.float32)
        l[:, 0] = far / 2 + rng.random() + np.arange(T) * 2.0 ** -22
        s = np.array([R.scores(row, "softmax")[0] for row in l])
        bal = np.full(E, -4.0, dtype=np.float32)
        bal[0], bal[1] = 0.0, (s[:, 0] - s[:, 1]).mean() * (1 + half_steps * R.EPS32)
        r = _router(E, 1, dict(score="softmax"), bal)
        b = r.buffers(T)
        r.select(torch.tensor(l).cuda(), b)
        c = s[:, :2] + bal[:2].astype(np.float64)
        sure = np.abs(c[:, 0] - c[:, 1]) > 2.0 ** -36 * s[:, 0]   # 64 bits can tell them apart
        open_ += (np.abs(c[:, 0] - c[:, 1]) < 2.0 ** -22 * s[:, 0]).sum()
        got = b.topk_idx.cpu().numpy()[:, 0]
        np.testing.assert_array_equal(got[sure], (c[:, 1] > c[:, 0]).astype(int)[sure])
    # the inputs do what they are for: rows lie some 2^-24 of the score apart, so of a call's several are
    # within 2^-22 of the border
    assert open_ > 2 * 17


@pytest.mark.parametrize("E,groups,topk", [(640, 20, 3), (744, 31, 4), (752, 47, 6), (760, 20, 3),
                                           (768, 24, 4), (776, 8, 2), (1024, 128, 9)])
def test_wide_rows_in_groups(E, groups, topk):
    """Rows around what shared memory takes without being asked (E = 768: 48 KB, and the kernel's
    own)."""
    rng = np.random.default_rng(E)
    l = rng.standard_normal((9, E)).astype(np.float32)
    kw = dict(score="sigmoid", n_groups=groups, topk_groups=topk)
    r = _router(E, 6, kw, None)
    b = r.buffers(9)
    r.select(torch.tensor(l).cuda(), b)
    _check_choice(l, 6, kw, None, b.topk_idx.cpu().numpy(), b.topk_w.cpu().numpy())


def test_groups_that_all_stay_are_one():
    """Sigmoids that 64 bits hold as equal: without a balance the logits decide, as for one group."""
    rng = np.random.default_rng(12)
    l = (40 + 5 * rng.standard_normal((30, 64))).astype(np.float32)
    got = []
    for groups in (1, 8):
        r = _router(64, 6, dict(score="sigmoid", n_groups=groups, topk_groups=groups), None)
        b = r.buffers(30)
        r.select(torch.tensor(l).cuda(), b)
        got.append(b.topk_idx.cpu().numpy())
    np.testing.assert_array_equal(got[0], got[1])
    np.testing.assert_array_equal(got[0], np.argsort(-l, axis=1, kind="stable")[:, :6])
