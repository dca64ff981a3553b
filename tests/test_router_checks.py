"""Refusals of the scored router: the C ABI's host checks (they never reach a
device) and those of the Python classes."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from mixture_experts_routed_softmax_gb300 import _lib
    from mixture_experts_routed_softmax_gb300.build import build
    build()
    _lib.load()
    return _lib


P = 0x1000


def _args(L, **kw):
    a = dict(balance=None, E=64, k=4, score=1, n_groups=4, topk_groups=2, group_rank=2,
             renormalise=1, scale=1.0)
    a.update(kw)
    return L.RouterArgs(*(a[n] for n, _ in L.RouterArgs._fields_))


BAD = [dict(E=0), dict(k=0), dict(k=65), dict(score=2), dict(n_groups=0), dict(n_groups=3),
       dict(topk_groups=0), dict(topk_groups=5), dict(group_rank=0), dict(group_rank=3),
       dict(k=33, E=64, topk_groups=2), dict(scale=float("nan")), dict(scale=float("inf")),
       dict(balance=P + 2)]


@pytest.mark.parametrize("kw", BAD, ids=str)
def test_router_arguments(L, kw):
    lib, a = L.load(), _args(L, **kw)
    r = ctypes.addressof(a)
    assert lib.moe_select(r, P, None, 4, P, P, None) == L.MOE_ERR_ARG
    assert lib.moe_select_bwd(r, P, P, P, 4, 0, P, None) == L.MOE_ERR_ARG
    assert lib.moe_route_scored(r, P, P, None, None, 4, 8, P, P, P, P, 1 << 30,
                                None) == L.MOE_ERR_ARG


def test_limits(L):
    lib = L.load()
    big = _args(L, E=2048, n_groups=1, topk_groups=1)
    many = _args(L, E=256, k=40, n_groups=1, topk_groups=1)
    for a in (big, many):
        assert lib.moe_select(ctypes.addressof(a), P, None, 4, P, P, None) == L.MOE_ERR_UNSUPPORTED
    a = _args(L)
    r = ctypes.addressof(a)
    assert lib.moe_select(r, P, None, 1 << 31, P, P, None) == L.MOE_ERR_UNSUPPORTED
    assert lib.moe_select(r, P, None, -1, P, P, None) == L.MOE_ERR_ARG
    assert lib.moe_select(None, P, None, 4, P, P, None) == L.MOE_ERR_ARG
    # nothing to do; missing arrays
    assert lib.moe_select(r, None, None, 0, None, None, None) == L.MOE_OK
    assert lib.moe_select_bwd(r, None, None, None, 0, 0, None, None) == L.MOE_OK
    for arrays in ((None, P, P), (P, None, P), (P, P, None)):
        assert lib.moe_select(r, arrays[0], None, 4, arrays[1], arrays[2], None) == L.MOE_ERR_ARG
    for arrays in ((None, P, P, P * 2), (P, None, P, P * 2), (P, P, None, P * 2), (P, P, P, None)):
        assert lib.moe_select_bwd(r, *arrays[:3], 4, 0, arrays[3], None) == L.MOE_ERR_ARG
    # in place would read what it has written
    assert lib.moe_select_bwd(r, P, P, P, 4, 0, P, None) == L.MOE_ERR_ARG


def test_route_and_logits_bwd(L):
    lib = L.load()
    a = _args(L)
    r = ctypes.addressof(a)
    ws = lib.moe_workspace_size(3, 4, 8, 64, 4, 16)
    call = lambda d=8, x=P, w=P, n=ws: lib.moe_route_scored(  # noqa: E731
        r, x, P, None, None, 4, d, P, P, P, w, n, None)
    assert call(d=12) == L.MOE_ERR_UNSUPPORTED
    assert call(d=0) == L.MOE_ERR_ARG
    assert call(x=P + 8) == L.MOE_ERR_ARG
    assert call(n=ws - 1) == L.MOE_ERR_ARG
    assert call(w=P + 16) == L.MOE_ERR_ARG
    for dense in (0, 1):
        n = lib.moe_logits_bwd_workspace_size(4, 8, 64, dense)
        assert n > 0
        bwd = lambda T=4, d=8, E=64, k=4, S=0, dl=P, dx=P, dxp=None, row=None, nb=n, w=P, \
            dw=P: lib.moe_logits_bwd(dl, P, P, T, d, E, dense, k, S, dx, dxp, row, dw, None, w,  # noqa: E731,B023
                                     nb, None)
        assert bwd(T=-1) == L.MOE_ERR_ARG
        assert bwd(E=1025) == L.MOE_ERR_UNSUPPORTED
        assert bwd(d=12) == L.MOE_ERR_UNSUPPORTED
        assert bwd(k=30, S=3) == L.MOE_ERR_UNSUPPORTED
        assert bwd(dl=None) == L.MOE_ERR_ARG
        assert bwd(dx=P + 2) == L.MOE_ERR_ARG
        assert bwd(dxp=P) == L.MOE_ERR_ARG           # without its rows' places
        assert bwd(dxp=P + 4, row=P) == L.MOE_ERR_ARG
        assert bwd(nb=n - 1) == L.MOE_ERR_ARG
        assert bwd(w=P + 128) == L.MOE_ERR_ARG
        assert bwd(dw=None) == L.MOE_ERR_ARG
    assert lib.moe_logits_bwd_workspace_size(-1, 8, 64, 0) == 0
    assert lib.moe_logits_bwd_workspace_size(4, 12, 64, 0) == 0
    assert lib.moe_logits_bwd_workspace_size(4, 8, 2000, 0) == 0


def test_python_refusals(L):
    from mixture_experts_routed_softmax_gb300.router import Router
    for kw in (dict(E=0, k=1), dict(E=8, k=9), dict(E=2048, k=2), dict(E=64, k=33),
               dict(E=8, k=2, score="tanh"), dict(E=8, k=2, n_groups=3),
               dict(E=8, k=2, n_groups=4, topk_groups=5), dict(E=8, k=3, n_groups=4),
               dict(E=8, k=2, group_rank=3), dict(E=8, k=2, scale=float("inf")),
               dict(E=8, k=2, balance=torch.zeros(8))):
        with pytest.raises(ValueError):
            Router(**kw)
    r = Router(8, 2)
    with pytest.raises(ValueError):
        r.select(torch.zeros(3, 8), r.buffers(3, device="cpu"))


def test_balance_cannot_be_replaced(L):
    from mixture_experts_routed_softmax_gb300.router import Router
    with pytest.raises(AttributeError):
        Router(8, 2).balance = torch.zeros(8)
