"""The attention operators without a GPU: argument checks of the C ABI (the
calls return before any CUDA work) and the frequencies' binary fractions."""
import ctypes
import math
from fractions import Fraction

import pytest


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_routed_softmax_gb300.build import build
    from mixture_experts_routed_softmax_gb300 import _lib
    build()
    return _lib.load()


P = 0x1000    # a non-null, 256-byte aligned stand-in: never touched


def _structs(cache=None, batch=None, rot=None):
    from mixture_experts_routed_softmax_gb300 import _lib as L
    c = dict(k=P, v=P, n_pages=9, page_stride=2 * 16 * 64, head_stride=16 * 64, token_stride=64,
             page_size=16, Hkv=2, D=64)
    b = dict(cu_q=P, kv_len=P, page_table=P, table_stride=4, T=3, B=2, max_pages=4, max_q=1)
    r = dict(turns=P, axis=None, rd=64, n_axes=1, interleaved=0, scale=1.0)
    c.update(cache or {})
    b.update(batch or {})
    r.update(rot or {})
    return L.KVCache(**c), L.KVBatchArgs(**b), L.Rotary(**r)


def _attn(lib, cache=None, batch=None, q=P, q_stride=512, Hq=8, scale=0.125, window=0, out=P,
          out_stride=512, ws=P, ws_bytes=1 << 40):
    c, b, _ = _structs(cache, batch)
    return lib.moe_attn_paged(ctypes.addressof(c), ctypes.addressof(b), q, q_stride, Hq, scale, 1,
                              window, None, out, out_stride, None, ws, ws_bytes, None)


def _append(lib, cache=None, batch=None, rot=None, k=P, k_stride=128, v=P, v_stride=128, q=P,
            q_stride=512, Hq=8, q_out=P, qo_stride=512):
    c, b, r = _structs(cache, batch, rot)
    return lib.moe_kv_append(ctypes.addressof(c), ctypes.addressof(b), ctypes.addressof(r), None,
                             k, k_stride, v, v_stride, q, q_stride, Hq, q_out, qo_stride, None)


def _rope(lib, rot=None, pos=P, T=3, D=64, q=P, q_stride=512, Hq=8, q_out=P, k=None, Hk=0,
          k_out=None):
    _, _, r = _structs(rot=rot)
    return lib.moe_rope(ctypes.addressof(r), pos, T, D, 0, q, q_stride, Hq, q_out, 512, k, 128, Hk,
                        k_out, 128, None)


CACHE = [({"k": None}, 1), ({"v": P + 8}, 1), ({"n_pages": 0}, 1), ({"page_size": 0}, 1),
         ({"Hkv": 0}, 1), ({"D": 0}, 1), ({"D": 60}, 2), ({"D": 136, "head_stride": 16 * 136,
          "token_stride": 136}, 2), ({"token_stride": 56}, 1), ({"head_stride": 1028}, 1),
         ({"page_stride": -2048}, 1), ({"n_pages": 1 << 31}, 2)]
BATCH = [({"cu_q": None}, 1), ({"kv_len": None}, 1), ({"page_table": None}, 1), ({"T": -1}, 1),
         ({"B": -1}, 1), ({"table_stride": 3}, 1), ({"max_pages": 1 << 27, "table_stride": 1 << 27},
                                                    2), ({"T": 1 << 30}, 2), ({"max_q": -1}, 1)]


@pytest.mark.parametrize("change,code", CACHE)
def test_bad_caches(lib, change, code):
    assert _attn(lib, cache=change) == code
    assert _append(lib, cache=change) == code


@pytest.mark.parametrize("change,code", BATCH)
def test_bad_batches(lib, change, code):
    assert _attn(lib, batch=change) == code
    assert _append(lib, batch=change) == code


def test_bad_attention_arguments(lib):
    assert lib.moe_attn_paged(None, None, P, 512, 8, 0.1, 1, 0, None, P, 512, None, P, 1, None) == 1
    for kw in ({"q": None}, {"q": P + 2}, {"out": None}, {"q_stride": 504}, {"q_stride": 516},
               {"out_stride": 8}, {"Hq": 7}, {"Hq": 0}, {"window": -1}, {"scale": 0.0},
               {"scale": -1.0}, {"scale": math.inf}, {"scale": math.nan}, {"ws": None},
               {"ws": P + 16}, {"ws_bytes": 16}):
        assert _attn(lib, **kw) == 1, kw
    # nothing to do: no tokens, no sequences
    assert _attn(lib, batch={"T": 0}, q=None, out=None) == 0
    assert _attn(lib, batch={"B": 0, "cu_q": None, "kv_len": None, "page_table": None}) == 0


def test_bad_append_and_rope_arguments(lib):
    for kw in ({"k": None}, {"v": None}, {"k_stride": 120}, {"v_stride": 132}, {"q_out": None},
               {"Hq": 0}, {"qo_stride": 0}, {"rot": {"turns": None}}, {"rot": {"rd": 66}},
               {"rot": {"rd": 0}}, {"rot": {"rd": 7}}, {"rot": {"n_axes": 0}},
               {"rot": {"n_axes": 9}}, {"rot": {"scale": math.nan}}):
        assert _append(lib, **kw) == 1, kw
    assert _append(lib, batch={"T": 0}, k=None, v=None, q=None, Hq=0) == 0
    for kw in ({"q": None}, {"q_out": None}, {"pos": None}, {"T": -1}, {"Hq": 0}, {"D": 0},
               {"k": P, "Hk": 2}, {"k": P, "k_out": P, "Hk": 0}, {"q_stride": 500},
               {"rot": {"rd": 128}}):
        assert _rope(lib, **kw) == 1, kw
    assert _rope(lib, D=132) == 2
    assert lib.moe_rope(None, P, 3, 64, 0, P, 512, 8, P, 512, None, 0, 0, None, 0, None) == 1
    assert _rope(lib, T=0, q=None, q_out=None, pos=None) == 0


def test_workspace_size_of_rejected_shapes(lib):
    for bad in ((0, 2, 64), (8, 0, 64), (8, 3, 64), (8, 2, 0), (8, 2, 60), (8, 2, 136)):
        assert lib.moe_attn_paged_workspace_size(*bad) == 0
    assert lib.moe_attn_paged_workspace_size(8, 2, 64) > 0


def test_turns_are_exact_fractions():
    """position * turns mod 2^64 is the angle's fraction of a turn to position *
    2^-65: far positions keep the angle."""
    from mixture_experts_routed_softmax_gb300.attention import turns_of
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    ws = [1.0, 150000.0 ** -0.5, 1e-7, 7.25, -0.3]
    for w, f in zip(ws, turns_of(ws)):
        assert 0 <= f < 1 << 64
        exact = Fraction(w) / (2 * pi)
        for p in (1, 12345, 2 ** 31 - 1, -7):
            got = Fraction((p * f) % (1 << 64), 1 << 64)
            diff = (got - p * exact) % 1
            diff = min(diff, 1 - diff)
            assert diff <= abs(p) * Fraction(1, 1 << 65) + Fraction(1, 10 ** 30)


def test_the_python_layer_refuses_what_does_not_fit(lib):
    """Raised before any call: nothing here touches a device."""
    import torch
    from mixture_experts_routed_softmax_gb300 import attention as A
    i32 = dict(dtype=torch.int32)
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        A.PagedAttention(kc, kc, 8)
    with pytest.raises(ValueError, match="cu_q"):
        A.KVBatch(torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, 4, **i32), 2)
    with pytest.raises(ValueError, match="pair"):
        A.Rope([], device="cpu")
    for axis, n in (([0, 1], 1), ([0], 2), ([-1, 0], 1)):
        with pytest.raises(ValueError, match="axis"):
            A.Rope([1.0, 0.5], axis=axis, n_axes=n, device="cpu")
    rope = A.Rope([1.0, 0.5], n_axes=2, device="cpu")
    assert rope.rd == 4 and rope.args.n_axes == 2
    q = torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="pos"):
        rope.apply(q, torch.zeros(2, 3, **i32), q)
