"""What the Python layer of the attention operators refuses before any call, with
stand-ins for CUDA tensors and for the library: nothing here touches a device."""
import types

import pytest
import torch

from mixture_experts_routed_softmax_gb300 import attention as A

BF16 = torch.bfloat16


class Tensor:
    """A CUDA tensor as far as the checks look at one."""

    def __init__(self, shape, dtype=BF16, strides=None, index=0):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.is_cuda = index >= 0
        self.device = torch.device("cuda", index) if self.is_cuda else torch.device("cpu")
        if strides is None:
            strides, n = [], 1
            for d in reversed(shape):
                strides.insert(0, n)
                n *= d
        self.strides = tuple(strides)

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return self.strides == Tensor(self.shape).strides

    def contiguous(self):
        return self

    def data_ptr(self):
        return 0x1000


@pytest.fixture
def calls(monkeypatch):
    """The calls that reached the library."""
    seen = []

    def entry(name, result=0):
        return lambda *a: seen.append((name, a)) or result

    lib = types.SimpleNamespace(
        moe_rope=entry("rope"), moe_kv_append=entry("append"), moe_attn_paged=entry("attend"),
        moe_attn_paged_workspace_size=lambda *a: 512, moe_status=entry("status"))
    monkeypatch.setattr(A._lib, "load", lambda: lib)
    monkeypatch.setattr(A, "_current_stream", lambda index: 0)
    monkeypatch.setattr(A, "_current_device", lambda: 0)
    return seen


I32 = torch.int32


def _layer(index=0, **kw):
    c = Tensor((9, 2, 16, 64), index=index)
    return A.PagedAttention(c, Tensor((9, 2, 16, 64), index=index), 8, **kw)


def _batch(T=3, B=2, index=0):
    return A.KVBatch(Tensor((B + 1,), I32, index=index), Tensor((B,), I32, index=index),
                     Tensor((B, 4), I32, index=index), T)


def _buffers(T=3, index=0, **kw):
    b = dict(T=T, q=Tensor((T, 8, 64), index=index), out=Tensor((T, 8, 64), index=index),
             lse=Tensor((T, 8), torch.float32, index=index),
             ws=Tensor((512,), torch.uint8, index=index))
    b.update(kw)
    return A.AttnBuffers(**b)


def test_the_stand_ins_pass(calls):
    layer, q, k = _layer(), Tensor((3, 8, 64)), Tensor((3, 2, 64))
    layer.append(k, k, _batch(), q=q, q_out=q)
    layer.attend(q, _batch(), _buffers())
    layer.attend(q, _batch(), _buffers(lse=None))
    assert [c[0] for c in calls] == ["append", "attend", "attend"]
    assert calls[1][1][13] == 512


@pytest.mark.parametrize("lse", [
    Tensor((3, 8), BF16), Tensor((3, 8), torch.float64), Tensor((3, 8), torch.float32, index=-1),
    Tensor((3, 8), torch.float32, (16, 1)), Tensor((2, 8), torch.float32)],
    ids=["bf16", "fp64", "cpu", "strided", "short"])
def test_log_sum_exps_of_another_type_are_refused(calls, lse):
    """The kernel writes four bytes an element, packed."""
    with pytest.raises(ValueError, match="lse"):
        _layer().attend(Tensor((3, 8, 64)), _batch(), _buffers(lse=lse))
    assert not calls


@pytest.mark.parametrize("ws", [
    Tensor((512,), torch.float32), Tensor((512,), torch.uint8, index=-1),
    Tensor((512,), torch.uint8, (2,))], ids=["fp32", "cpu", "strided"])
def test_workspaces_of_another_type_are_refused(calls, ws):
    """Its size in bytes is taken from its elements."""
    with pytest.raises(ValueError, match="ws"):
        _layer().attend(Tensor((3, 8, 64)), _batch(), _buffers(ws=ws))
    assert not calls


def test_another_current_device_is_refused(calls, monkeypatch):
    """The library launches on the current device."""
    layer, batch, q, k = _layer(), _batch(), Tensor((3, 8, 64)), Tensor((3, 2, 64))
    rope = _rope()
    monkeypatch.setattr(A, "_current_device", lambda: 1)
    for call in (lambda: layer.attend(q, batch, _buffers()),
                 lambda: layer.append(k, k, batch), lambda: layer.buffers(3),
                 lambda: layer.status(), lambda: rope.apply(q, Tensor((1, 3), I32), q)):
        with pytest.raises(ValueError, match="current device is cuda:1"):
            call()
    assert not calls


def _rope(index=0):
    rope = A.Rope([1.0, 0.5], device="cpu")
    rope.turns, rope._dev = Tensor((2,), torch.int64, index=index), index
    return rope


@pytest.mark.parametrize("what", ["q", "out", "lse", "ws", "batch", "stream"])
def test_attention_over_two_devices_is_refused(calls, what):
    q, b = Tensor((3, 8, 64), index=int(what == "q")), _buffers()
    if what in ("out", "lse", "ws"):
        t = getattr(b, what)
        setattr(b, what, Tensor(t.shape, t.dtype, index=1))
    stream = None
    if what == "stream":
        stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=64)
    with pytest.raises(ValueError, match=what):
        _layer().attend(q, _batch(index=int(what == "batch")), b, stream=stream)
    assert not calls


@pytest.mark.parametrize("what", ["k", "v", "q", "q_out", "pos", "batch"])
def test_an_append_over_two_devices_is_refused(calls, what):
    t = {n: Tensor(s, index=int(what == n)) for n, s in
         (("k", (3, 2, 64)), ("v", (3, 2, 64)), ("q", (3, 8, 64)), ("q_out", (3, 8, 64)))}
    pos = Tensor((1, 3), I32, index=int(what == "pos"))
    with pytest.raises(ValueError, match=what):
        _layer(rope=_rope()).append(t["k"], t["v"], _batch(index=int(what == "batch")), q=t["q"],
                                    q_out=t["q_out"], pos=pos)
    assert not calls


@pytest.mark.parametrize("what", ["q", "q_out", "k", "k_out", "pos"])
def test_a_rotation_over_two_devices_is_refused(calls, what):
    t = {n: Tensor((3, 2, 64), index=int(what == n)) for n in ("q", "q_out", "k", "k_out")}
    with pytest.raises(ValueError, match=what):
        _rope().apply(t["q"], Tensor((1, 3), I32, index=int(what == "pos")), t["q_out"], k=t["k"],
                      k_out=t["k_out"])
    assert not calls


def test_layers_and_batches_over_two_devices_are_refused(calls):
    c, far = Tensor((9, 2, 16, 64)), Tensor((9, 2, 16, 64), index=1)
    for args, kw in (((c, far, 8), {}), ((c, c, 8), {"rope": _rope(1)}),
                     ((c, c, 8), {"sinks": Tensor((8,), torch.float32, index=1)})):
        with pytest.raises(ValueError, match="cuda:1"):
            A.PagedAttention(*args, **kw)
    for i in range(3):
        at = [int(i == j) for j in range(3)]
        with pytest.raises(ValueError, match="different devices"):
            A.KVBatch(Tensor((3,), I32, index=at[0]), Tensor((2,), I32, index=at[1]),
                      Tensor((2, 4), I32, index=at[2]), 3)


def test_another_device_works_where_it_is_the_current_one(calls, monkeypatch):
    monkeypatch.setattr(A, "_current_device", lambda: 1)
    layer, batch = _layer(1, rope=_rope(1)), _batch(index=1)
    q, k = Tensor((3, 8, 64), index=1), Tensor((3, 2, 64), index=1)
    layer.append(k, k, batch, q=q, q_out=q, pos=Tensor((1, 3), I32, index=1))
    layer.attend(q, batch, _buffers(index=1))
    assert [c[0] for c in calls] == ["append", "attend"]


@pytest.mark.parametrize("v", [2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1])
def test_windows_and_hints_past_a_c_int(calls, v):
    """Not their low 32 bits: a window of 2^32 + 5 keys is not one of 5."""
    _layer(window=v).attend(Tensor((3, 8, 64)), _batch(), _buffers())
    name, args = calls.pop()
    assert name == "attend" and args[7] == 2 ** 31 - 1
    batch = A.KVBatch(Tensor((3,), I32), Tensor((2,), I32), Tensor((2, 4), I32), 3, max_q=v)
    assert batch.args.max_q == 2 ** 31 - 1


def test_negative_windows_and_hints_are_refused(calls):
    with pytest.raises(ValueError, match="window"):
        _layer(window=-1)
    with pytest.raises(ValueError, match="max_q"):
        A.KVBatch(Tensor((3,), I32), Tensor((2,), I32), Tensor((2, 4), I32), 3, max_q=-1)
