"""Attention in front of the expert layer, driven through the C ABI: rotary
positions (moe_rope), the append of new keys and values to a paged cache
(moe_kv_append) and the attention of new tokens over it (moe_attn_paged).

PyTorch supplies device memory and the stream; every step runs in the
library's kernels, on the current device, which has to be the tensors'. A
serving step is ``PagedAttention.forward`` (append, then attend); ``Rope.apply``
rotates without a cache, and with ``transpose=True`` takes gradients back
through the rotation in training.
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from fractions import Fraction
from typing import Optional, Sequence

import torch

from . import _lib

BF16 = torch.bfloat16
_ref = _lib.ctypes.addressof
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _c_int(name: str, v) -> int:
    """A size that means the same from 2^31 - 1 on, for a C int (ctypes would take
    its low 32 bits)."""
    if int(v) < 0:
        raise ValueError(f"{name}: {v} is negative")
    return min(int(v), 2 ** 31 - 1)


def _stream(dev: int, stream) -> int:
    """The raw stream of a call on tensors of device ``dev``. The library launches
    on the current device, so that has to be theirs."""
    if _current_device() != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is "
                         f"cuda:{_current_device()}")
    if stream is None:
        return _current_stream(dev)
    if stream.device.index != dev:
        raise ValueError(f"stream: one of cuda:{dev} is needed, not {stream.device}")
    return stream.cuda_stream


def _view(name: str, t: torch.Tensor, T: int, H: int, D: int, dev: int) -> int:
    """Check a [T, H, D] bf16 view with packed heads on device ``dev``; its token
    stride. (These checks are a good part of a one-token call's host time: the
    usual case, tokens of packed heads, is looked at first.)"""
    if t.dtype is not BF16 or t.get_device() != dev:
        raise ValueError(f"{name}: a bf16 tensor on cuda:{dev} is needed")
    if t.shape != (T, H, D):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(T, H, D)}")
    st, sh, sd = t.stride()
    if sd == 1 and sh == D:
        return st if T > 1 else H * D
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}: heads must be packed (strides {t.stride()})")
    return st if T > 1 else H * D


def _check(fn: str, code: int) -> None:
    if code:
        raise _lib.MoEError(fn, code)


def _int32(name: str, t: torch.Tensor, shape) -> torch.Tensor:
    """Check an index array. Nothing is copied: a copy would be made on the
    current stream, while the call may run on another."""
    if t.dtype != torch.int32 or t.device.type != "cuda" or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: an int32 CUDA tensor of shape {tuple(shape)} is needed")
    if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: its last axis must be packed")
    return t


def turns_of(inv_freq: Sequence[float]) -> list[int]:
    """Frequencies in radians a position -> turns a position as 64-bit binary
    fractions (moe_rotary.turns), from the exact value of each given double."""
    # pi to 60 digits: the fraction's 64 bits need 20
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    return [round(Fraction(float(w)) / two_pi * (1 << 64)) % (1 << 64) for w in inv_freq]


class Rope:
    """Rotary positions: frequencies, the axis each pair follows, the pairing.

    inv_freq: rd/2 frequencies in radians a position (doubles); axis: the
    position axis of each pair (None: all the first of n_axes); interleaved:
    pairs (2i, 2i+1) instead of (i, i + rd/2); scale multiplies the result.
    """

    def __init__(self, inv_freq: Sequence[float], axis: Optional[Sequence[int]] = None,
                 n_axes: int = 1, interleaved: bool = False, scale: float = 1.0, device="cuda"):
        self.lib = _lib.load()
        turns = turns_of(inv_freq)
        if not turns:
            raise ValueError("Rope needs at least one pair")
        if axis is not None and (len(axis) != len(turns) or min(axis) < 0 or max(axis) >= n_axes):
            raise ValueError(f"axis needs {len(turns)} entries in [0, {n_axes})")
        self.rd, self.n_axes = 2 * len(turns), n_axes
        signed = [v - (1 << 64) if v >= (1 << 63) else v for v in turns]
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)
        self.axis = (None if axis is None
                     else torch.tensor(list(axis), dtype=torch.int32, device=device))
        self.args = _lib.Rotary(_p(self.turns), _p(self.axis), self.rd, n_axes, int(interleaved),
                                float(scale))
        self._ref = _ref(self.args)
        self._call = self.lib.moe_rope
        self._dev = self.turns.device.index

    @classmethod
    def from_base(cls, rd: int, base: float, **kw) -> "Rope":
        """Frequencies base^(-2i / rd), i = 0 .. rd/2 - 1."""
        return cls([base ** (-2.0 * i / rd) for i in range(rd // 2)], **kw)

    def _pos(self, pos: torch.Tensor, T: int) -> torch.Tensor:
        if pos.dim() == 1:
            pos = pos[None]
        if (pos.dtype is not torch.int32 or pos.get_device() != self._dev
                or pos.shape != (self.n_axes, T)):
            raise ValueError(f"pos: an int32 tensor of shape {(self.n_axes, T)} on "
                             f"cuda:{self._dev} is needed")
        if not pos.is_contiguous():
            raise ValueError("pos: its rows must be packed")
        return pos

    def apply(self, q, pos, q_out, k=None, k_out=None, transpose: bool = False, stream=None):
        """q_out = R q (and k_out = R k), [T, H, D] views; pos [n_axes, T] (or [T])
        int32. transpose: R^T, the gradient's way back. In place is fine."""
        T, H, D = q.shape
        pos, dev = self._pos(pos, T), self._dev
        Hk = 0 if k is None else int(k.shape[1])
        if (k is None) != (k_out is None):
            raise ValueError("k and k_out go together")
        ks = kos = 0
        kp = kop = None
        if k is not None:
            ks, kos = _view("k", k, T, Hk, D, dev), _view("k_out", k_out, T, Hk, D, dev)
            kp, kop = k.data_ptr(), k_out.data_ptr()
        _check("moe_rope", self._call(
            self._ref, pos.data_ptr(), T, D, int(transpose), q.data_ptr(),
            _view("q", q, T, H, D, dev), H, q_out.data_ptr(),
            _view("q_out", q_out, T, H, D, dev), kp, ks, Hk, kop, kos, _stream(dev, stream)))
        return q_out


class KVBatch:
    """A ragged batch: cu_q [B+1], kv_len [B] (new tokens included), page_table
    [B, max_pages], all int32 on the device; T rows; max_q: the largest number
    of new tokens of one sequence (a hint: T always works). The kernel is chosen
    by max_q and by the keys that the table's width allows a sequence, so a narrow
    table serves short sequences faster (include/moe.h, moe_kv_batch)."""

    def __init__(self, cu_q, kv_len, page_table, T: int, max_q: Optional[int] = None):
        B = int(kv_len.shape[0])
        self.cu_q = _int32("cu_q", cu_q, (B + 1,))
        self.kv_len = _int32("kv_len", kv_len, (B,))
        self.page_table = _int32("page_table", page_table, (B, page_table.shape[1]))
        self._dev = cu_q.get_device()
        if kv_len.get_device() != self._dev or page_table.get_device() != self._dev:
            raise ValueError("cu_q, kv_len and page_table are on different devices")
        self.T, self.B = int(T), B
        pages = int(self.page_table.shape[1])
        stride = self.page_table.stride(0) if B > 1 else pages
        self.args = _lib.KVBatchArgs(_p(self.cu_q), _p(self.kv_len), _p(self.page_table), stride,
                                     self.T, B, pages,
                                     _c_int("max_q", self.T if max_q is None else max_q))
        self._ref = _ref(self.args)


@dataclass
class AttnBuffers:
    """Device buffers of one call of T tokens."""
    T: int
    q: torch.Tensor            # rotated queries
    out: torch.Tensor
    lse: Optional[torch.Tensor]
    ws: torch.Tensor


class PagedAttention:
    """One attention layer over its paged cache.

    k_cache, v_cache: bf16 [n_pages, Hkv, page_size, D] (or, with
    heads_first=False, [n_pages, page_size, Hkv, D]), any strides with D packed;
    Hq query heads, Hq / Hkv of them to a key head. rope: the rotation keys and
    queries take in ``append`` (None: none). scale: D^-1/2 unless given.
    window: how many keys a token sees, itself included (0: all). sinks [Hq]
    fp32: a logit per head that joins the denominator.
    """

    def __init__(self, k_cache, v_cache, Hq: int, rope: Optional[Rope] = None,
                 scale: Optional[float] = None, causal: bool = True, window: int = 0,
                 sinks: Optional[torch.Tensor] = None, heads_first: bool = True):
        self.lib = _lib.load()
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t.dtype != BF16 or t.device.type != "cuda" or t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{name}: a bf16 CUDA tensor of 4 axes with D packed is needed")
        if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
            raise ValueError("k_cache and v_cache differ in shape or strides")
        for name, t in (("v_cache", v_cache), ("sinks", sinks),
                        ("rope", None if rope is None else rope.turns)):
            if t is not None and t.device != k_cache.device:
                raise ValueError(f"{name} is on {t.device}, k_cache on {k_cache.device}")
        self.k_cache, self.v_cache = k_cache, v_cache
        ha, sa = (1, 2) if heads_first else (2, 1)
        self.n_pages, self.Hkv = int(k_cache.shape[0]), int(k_cache.shape[ha])
        self.page_size, self.D = int(k_cache.shape[sa]), int(k_cache.shape[3])
        self.Hq = int(Hq)
        if self.Hq <= 0 or self.Hq % self.Hkv:
            raise ValueError(f"{Hq} query heads over {self.Hkv} key heads")
        if sinks is not None and (sinks.dtype != torch.float32 or tuple(sinks.shape) != (self.Hq,)
                                  or sinks.device.type != "cuda"):
            raise ValueError(f"sinks: fp32 [{self.Hq}] on the device is needed")
        self.sinks = None if sinks is None else sinks.contiguous()
        self.rope, self.causal, self.window = rope, bool(causal), _c_int("window", window)
        self.scale = 1.0 / math.sqrt(self.D) if scale is None else float(scale)
        self.device = k_cache.device
        st = k_cache.stride()
        self.cache = _lib.KVCache(_p(k_cache), _p(v_cache), self.n_pages, st[0], st[ha], st[sa],
                                  self.page_size, self.Hkv, self.D)
        self._ref = _ref(self.cache)
        self._rope = None if rope is None else _ref(rope.args)
        self._sinks = _p(self.sinks)
        self._call_append, self._call_attend = self.lib.moe_kv_append, self.lib.moe_attn_paged
        self._dev = self.device.index

    def buffers(self, T: int, lse: bool = False) -> AttnBuffers:
        _stream(self._dev, None)       # the workspace's size is the current device's
        kw = dict(device=self.device)
        ws = int(self.lib.moe_attn_paged_workspace_size(self.Hq, self.Hkv, self.D))
        return AttnBuffers(
            T=T, q=torch.empty(T, self.Hq, self.D, dtype=BF16, **kw),
            out=torch.empty(T, self.Hq, self.D, dtype=BF16, **kw),
            lse=torch.empty(T, self.Hq, dtype=torch.float32, **kw) if lse else None,
            ws=torch.empty(max(ws, 256), dtype=torch.uint8, **kw))

    def append(self, k, v, batch: KVBatch, q=None, q_out=None, pos=None, stream=None):
        """The new tokens' keys (rotated) and values into the cache; q rotated
        into q_out when given. pos [n_axes, T] int32, or None: each token's
        position in its sequence."""
        T, Hkv, Hq, D, dev = batch.T, self.Hkv, self.Hq, self.D, self._dev
        if batch._dev != dev:
            raise ValueError(f"the batch is on cuda:{batch._dev}, the cache on cuda:{dev}")
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out go together")
        if pos is not None:
            if self.rope is None:
                raise ValueError("positions without a rotation")
            pos = self.rope._pos(pos, T)
        qs = qos = 0
        qp = qop = pp = None
        if q is not None:
            qs, qos = _view("q", q, T, Hq, D, dev), _view("q_out", q_out, T, Hq, D, dev)
            qp, qop = q.data_ptr(), q_out.data_ptr()
        if pos is not None:
            pp = pos.data_ptr()
        _check("moe_kv_append", self._call_append(
            self._ref, batch._ref, self._rope, pp, k.data_ptr(), _view("k", k, T, Hkv, D, dev),
            v.data_ptr(), _view("v", v, T, Hkv, D, dev), qp, qs, Hq, qop, qos,
            _stream(dev, stream)))
        return q_out

    def attend(self, q, batch: KVBatch, b: AttnBuffers, out=None, stream=None):
        """Attention of q [T, Hq, D] over the cache into ``out`` (default b.out);
        b.lse, when there, takes the log-sum-exp of every row."""
        out = b.out if out is None else out
        T, Hq, D, dev = batch.T, self.Hq, self.D, self._dev
        if batch._dev != dev:
            raise ValueError(f"the batch is on cuda:{batch._dev}, the cache on cuda:{dev}")
        lse, ws = b.lse, b.ws
        if lse is not None and (lse.dtype is not torch.float32 or lse.get_device() != dev
                                or lse.shape != (T, Hq) or not lse.is_contiguous()):
            raise ValueError(f"lse: a packed fp32 tensor of shape {(T, Hq)} on cuda:{dev} is "
                             "needed")
        if ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
            raise ValueError(f"ws: a packed uint8 tensor on cuda:{dev} is needed (buffers() "
                             "makes one)")
        _check("moe_attn_paged", self._call_attend(
            self._ref, batch._ref, q.data_ptr(), _view("q", q, T, Hq, D, dev), Hq, self.scale,
            self.causal, self.window, self._sinks, out.data_ptr(),
            _view("out", out, T, Hq, D, dev), None if lse is None else lse.data_ptr(),
            ws.data_ptr(), ws.numel(), _stream(dev, stream)))
        return out

    def forward(self, q, k, v, batch: KVBatch, b: AttnBuffers, pos=None, stream=None):
        """One step: append k and v, rotate q into b.q, attend into b.out."""
        self.append(k, v, batch, q=q, q_out=b.q, pos=pos, stream=stream)
        return self.attend(b.q, batch, b, stream=stream)

    def status(self, stream=None) -> int:
        """Synchronise and read (and clear) the device status word."""
        return int(self.lib.moe_status(_stream(self._dev, stream)))
