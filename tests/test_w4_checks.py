"""4-bit weights without a GPU: the reference's own quantiser against brute force,
the arrays' sizes, and the refusals of the C ABI's host checks (they never reach a
device) and of the Python classes."""
import ctypes

import numpy as np
import pytest
import torch

import w4_ref as W

P = 0x1000


@pytest.fixture(scope="module")
def L():
    from mixture_experts_routed_softmax_gb300 import _lib
    from mixture_experts_routed_softmax_gb300.build import build
    build()
    _lib.load()
    return _lib


@pytest.mark.parametrize("kind", ["int4", "fp4"])
def test_reference_quantiser(kind):
    """Scales have few bits and cover the group; codes are nearest; code * scale is bf16."""
    rng = np.random.default_rng(1)
    w = torch.tensor(rng.standard_normal((64, 40)) * np.exp(3 * rng.standard_normal(40)))
    w = w.to(torch.bfloat16).double().numpy()
    codes, scales = W.quantise(w, kind, 32)
    got = W.weights(codes, scales, kind, 32)
    assert np.array_equal(got, torch.tensor(got).to(torch.bfloat16).double().numpy())
    top = {"int4": 7, "fp4": 6}[kind]
    a = np.abs(w).reshape(2, 32, 40).max(1)
    assert np.all(a <= top * scales) and np.all(top * scales <= a * (1 + 1 / 8 if kind == "int4"
                                                                     else 2))
    grid = np.unique(np.concatenate([W.values(np.arange(16), kind), [-top, top]]))
    grid = grid[np.abs(grid) <= top]
    s = np.repeat(scales, 32, 0)
    best = np.abs(w[..., None] - grid * s[..., None]).min(-1)
    assert np.allclose(np.abs(w - got), best, rtol=0, atol=0)


def _w4(L, **kw):
    a = dict(codes=P, scales=P, E=1, K=64, N=32, group=32, kind=0)
    a.update(kw)
    return L.W4(*(a[n] for n, _ in L.W4._fields_))


def test_sizes(L):
    lib = L.load()
    # 2880 rows: 45 blocks of 64; 640 columns: 40 blocks of 16; 23 steps of 128 rows
    assert lib.moe_w4_codes_bytes(3, 2880, 640) == 3 * 40 * 45 * 512
    assert lib.moe_w4_scales_bytes(3, 2880, 640, 32) == 3 * 40 * 23 * 16 * 4 * 2 + 16
    assert lib.moe_w4_scales_bytes(3, 2880, 640, 128) == 3 * 40 * 23 * 16 * 2 + 16
    assert lib.moe_w4_codes_bytes(1, 8, 8) == 512
    for bad in ((0, 64, 64), (1, 60, 64), (1, 64, 4), (1025, 64, 64), (1, 65544, 64)):
        assert lib.moe_w4_codes_bytes(*bad) == 0
    assert lib.moe_w4_scales_bytes(1, 64, 64, 16) == 0


BAD = [(dict(codes=None), 1), (dict(scales=None), 1), (dict(codes=P + 8), 1),
       (dict(scales=P + 2), 1), (dict(kind=2), 1), (dict(group=16), 1), (dict(group=0), 1),
       (dict(E=0), 1), (dict(K=0), 1), (dict(N=-8), 1), (dict(K=60), 2), (dict(N=12), 2),
       (dict(E=2000), 2), (dict(K=65600), 2)]


@pytest.mark.parametrize("kw,code", BAD, ids=str)
def test_weights_arguments(L, kw, code):
    lib, a = L.load(), _w4(L, **kw)
    r = ctypes.addressof(a)
    assert lib.moe_w4_quantise(r, P, None) == code
    assert lib.moe_w4_pack(r, P, P, None) == code
    assert lib.moe_w4_dequantise(r, P, None) == code
    assert lib.moe_w4_linear(r, P, 64, 1, P, 32, 0, P, 1 << 30, None) == code


def test_other_arguments(L):
    lib, a = L.load(), _w4(L)
    r = ctypes.addressof(a)
    for fn in (lib.moe_w4_quantise, lib.moe_w4_dequantise):
        assert fn(None, P, None) == L.MOE_ERR_ARG
        assert fn(r, None, None) == L.MOE_ERR_ARG
        assert fn(r, P + 8, None) == L.MOE_ERR_ARG
    assert lib.moe_w4_pack(r, P + 4, P, None) == L.MOE_ERR_ARG
    assert lib.moe_w4_pack(r, P, None, None) == L.MOE_ERR_ARG
    lin = lambda x=P, xs=64, T=2, y=P, ys=32, f=0, w=r: lib.moe_w4_linear(  # noqa: E731
        w, x, xs, T, y, ys, f, P, 1 << 40, None)
    assert lin(T=0, x=None, y=None) == L.MOE_OK
    assert lin(T=-1) == L.MOE_ERR_ARG
    assert lin(T=1 << 26) == L.MOE_ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(y=None), dict(x=P + 8), dict(xs=63), dict(xs=68), dict(ys=31),
               dict(y=P + 1), dict(y=P + 2, f=1)):
        assert lin(**kw) == L.MOE_ERR_ARG, kw
    two = _w4(L, E=2)
    assert lin(w=ctypes.addressof(two)) == L.MOE_ERR_ARG


def test_experts_arguments(L):
    lib = L.load()
    mk = lambda **kw: _w4(L, **{**dict(E=6, K=64, N=32), **kw})  # noqa: E731
    n = lib.moe_expert_fwd_w4_workspace_size(4, 2, 4, 2, 64, 32)
    assert n > 0

    def call(gate=None, up=None, down=None, act=None, x=P, idx=P, w=P, T=4, k=2, E=4, S=2, y=P,
             ws=P, nb=n):
        ms = [gate or mk(), up or mk(), down or mk(K=32, N=64)]
        return lib.moe_expert_fwd_w4(*(ctypes.addressof(m) for m in ms),
                                     None if act is None else ctypes.addressof(act), x, idx, w, T,
                                     k, E, S, y, ws, nb, None)

    assert call(T=0, x=None, idx=None, w=None, y=None, ws=None, nb=0) == L.MOE_OK
    for kw in (dict(x=None), dict(idx=None), dict(w=None), dict(y=None), dict(ws=None),
               dict(nb=n - 1), dict(ws=P + 128), dict(x=P + 8), dict(y=P + 8), dict(T=-1),
               dict(k=0), dict(k=5), dict(S=-1), dict(E=3), dict(S=1), dict(gate=mk(N=40)),
               dict(up=mk(K=72)), dict(down=mk()), dict(up=mk(kind=1)), dict(gate=mk(group=64)),
               dict(down=mk(K=32, N=64, E=5)), dict(act=L.Swiglu(0.0, 1.0, 0.0)),
               dict(act=L.Swiglu(1.0, float("nan"), 0.0))):
        assert call(**kw) == L.MOE_ERR_ARG, kw
    assert call(gate=mk(E=40), up=mk(E=40), down=mk(E=40, K=32, N=64), k=31, E=38,
                S=2) == L.MOE_ERR_UNSUPPORTED
    for bad in ((0, 2, 4, 0, 64, 32), (4, 0, 4, 0, 64, 32), (4, 5, 4, 0, 64, 32),
                (4, 2, 4, 0, 60, 32), (4, 2, 4, -1, 64, 32)):
        assert lib.moe_expert_fwd_w4_workspace_size(*bad) == 0


def test_python_refusals(L):
    from mixture_experts_routed_softmax_gb300.w4 import Weights4
    c, s = torch.zeros(512, dtype=torch.uint8), torch.zeros(64, dtype=torch.bfloat16)
    for kw in (dict(kind="int8", group=32), dict(kind="int4", group=16), dict(kind="int4", group=32)):
        with pytest.raises(ValueError):
            Weights4(c, s, 1, 64, 16, **kw)          # the last: not on a device
    with pytest.raises(ValueError):
        Weights4(c, s, 1, 60, 16, "int4", 32)
