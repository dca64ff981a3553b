"""Weights in 4 bits with group scales, driven through the C ABI: their making
(moe_w4_quantise, moe_w4_pack, moe_w4_dequantise), a linear layer (moe_w4_linear) and
the experts' forward with them (moe_expert_fwd_w4). For inference.

``MoELayer.quantised`` makes a ``MoELayer4`` of a layer: the same router in front of
experts in 4 bits.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from .attention import _check, _p, _ref, _stream
from .router import _packed

BF16 = torch.bfloat16
KINDS = {"int4": _lib.MOE_W4_INT4, "fp4": _lib.MOE_W4_FP4}


def _fresh(stream, dev: int, *tensors) -> None:
    """Tensors just allocated, to be written by a call on ``stream``: their memory may be what work
    still to come on the current stream uses, so ``stream`` waits for that, and is not given
    out again before the call has ended."""
    _stream(dev, stream)
    current = torch.cuda.current_stream(dev)
    if stream is not None and stream != current:
        stream.wait_stream(current)
        for t in tensors:
            t.record_stream(stream)


class Weights4:
    """Matrices [E, K, N] in 4 bits: value(code) * scale, one scale for ``group``
    (32, 64 or 128) neighbouring rows of a column.

    kind: "int4" (-8 .. 7) or "fp4" (+-{0, 1/2, 1, 3/2, 2, 3, 4, 6}). Codes and scales lie in
    the library's own layout (``codes``, ``scales``: flat arrays to be kept or copied whole).
    """

    # the kernels read them at these addresses: they can be written to, not replaced
    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)

    def __init__(self, codes, scales, E: int, K: int, N: int, kind: str, group: int):
        self.lib = _lib.load()
        if kind not in KINDS:
            raise ValueError(f"kind: one of {sorted(KINDS)} is needed, not {kind!r}")
        if group not in (32, 64, 128):
            raise ValueError(f"group: 32, 64 or 128 rows, not {group}")
        nc = int(self.lib.moe_w4_codes_bytes(E, K, N))
        ns = int(self.lib.moe_w4_scales_bytes(E, K, N, group)) // 2
        if not nc:
            raise ValueError(f"[{E}, {K}, {N}]: up to 1024 matrices of multiples of 8, at most "
                             "65536, are supported")
        if codes.get_device() < 0 or codes.get_device() != scales.get_device():
            raise ValueError("codes and scales: CUDA tensors on one device are needed")
        self._dev = codes.get_device()
        _packed("codes", codes, torch.uint8, (nc,), self._dev)
        _packed("scales", scales, BF16, (ns,), self._dev)
        self._codes, self._scales = codes, scales
        self.E, self.K, self.N, self.kind, self.group = int(E), int(K), int(N), kind, int(group)
        self.args = _lib.W4(_p(codes), _p(scales), self.E, self.K, self.N, self.group,
                            KINDS[kind])
        self._ref = _ref(self.args)

    @classmethod
    def empty(cls, E: int, K: int, N: int, kind: str = "int4", group: int = 32,
              device="cuda") -> "Weights4":
        """Room for matrices that quantise_from or pack_from will fill."""
        lib = _lib.load()
        return cls(torch.empty(int(lib.moe_w4_codes_bytes(E, K, N)), dtype=torch.uint8,
                               device=device),
                   torch.empty(int(lib.moe_w4_scales_bytes(E, K, N, group)) // 2, dtype=BF16,
                               device=device), E, K, N, kind, group)

    @classmethod
    def quantise(cls, w, kind: str = "int4", group: int = 32, stream=None) -> "Weights4":
        """4-bit weights of w [E, K, N] bf16."""
        E, K, N = w.shape
        q = cls.empty(E, K, N, kind, group, w.device)
        _fresh(stream, q._dev, q.codes, q.scales)
        return q.quantise_from(w, stream)

    @classmethod
    def from_codes(cls, codes, scales, kind: str = "int4", group: int = 32,
                   stream=None) -> "Weights4":
        """Weights given as codes [E, K, N] uint8 and scales [E, ceil(K/group), N] bf16."""
        E, K, N = codes.shape
        q = cls.empty(E, K, N, kind, group, codes.device)
        _fresh(stream, q._dev, q.codes, q.scales)
        return q.pack_from(codes, scales, stream)

    def quantise_from(self, w, stream=None) -> "Weights4":
        _check("moe_w4_quantise", self.lib.moe_w4_quantise(
            self._ref, _packed("w", w, BF16, (self.E, self.K, self.N), self._dev),
            _stream(self._dev, stream)))
        return self

    def pack_from(self, codes, scales, stream=None) -> "Weights4":
        shape = (self.E, -(-self.K // self.group), self.N)
        _check("moe_w4_pack", self.lib.moe_w4_pack(
            self._ref, _packed("codes", codes, torch.uint8, (self.E, self.K, self.N), self._dev),
            _packed("scales", scales, BF16, shape, self._dev), _stream(self._dev, stream)))
        return self

    def dequantise(self, out=None, stream=None) -> torch.Tensor:
        """The weights as bf16 [E, K, N] (code * scale, rounded)."""
        shape = (self.E, self.K, self.N)
        if out is None:
            out = torch.empty(shape, dtype=BF16, device=self.codes.device)
            _fresh(stream, self._dev, out)
        _check("moe_w4_dequantise", self.lib.moe_w4_dequantise(
            self._ref, _packed("out", out, BF16, shape, self._dev), _stream(self._dev, stream)))
        return out


@dataclass
class Buffers4:
    """Output and workspace of one call of T tokens."""
    T: int
    y: torch.Tensor
    ws: torch.Tensor


def _ws(b: Buffers4, dev: int) -> int:
    ws = b.ws
    if ws.dtype is not torch.uint8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: a packed uint8 tensor on cuda:{dev} is needed (buffers() makes one)")
    return ws.data_ptr()


class Linear4:
    """y = x W with one 4-bit matrix [1, K, N]; out_dtype: bf16 or fp32."""

    def __init__(self, weights: Weights4, out_dtype=BF16):
        if weights.E != 1:
            raise ValueError(f"one matrix is needed, not {weights.E}")
        if out_dtype not in (BF16, torch.float32):
            raise ValueError(f"out_dtype: bf16 or fp32, not {out_dtype}")
        self.lib, self.weights, self.out_dtype = weights.lib, weights, out_dtype
        self.K, self.N, self._dev = weights.K, weights.N, weights._dev
        self._w, self._fp32 = weights._ref, int(out_dtype is torch.float32)
        self._call = self.lib.moe_w4_linear

    def buffers(self, T: int) -> Buffers4:
        _stream(self._dev, None)
        ws = int(self.lib.moe_w4_linear_workspace_size(self._w, T))
        kw = dict(device=self.weights.codes.device)
        return Buffers4(T, torch.empty(T, self.N, dtype=self.out_dtype, **kw),
                        torch.empty(max(ws, 256), dtype=torch.uint8, **kw))

    def apply(self, x, b: Buffers4, out=None, stream=None) -> torch.Tensor:
        """x [T, K] bf16 (rows packed, any stride of a multiple of 8 between them) times W
        into ``out`` (default b.y) [T, N]."""
        T, dev = b.T, self._dev
        out = b.y if out is None else out
        if x.dtype is not BF16 or x.get_device() != dev or x.shape != (T, self.K):
            raise ValueError(f"x: a bf16 tensor of shape {(T, self.K)} on cuda:{dev} is needed")
        if out.dtype is not self.out_dtype or out.get_device() != dev or out.shape != (T, self.N):
            raise ValueError(f"out: a {self.out_dtype} tensor of shape {(T, self.N)} on cuda:{dev} "
                             "is needed")
        if x.stride(1) != 1 or out.stride(1) != 1:
            raise ValueError("x and out: rows must be packed")
        _check("moe_w4_linear", self._call(
            self._w, x.data_ptr(), x.stride(0) if T > 1 else self.K, T, out.data_ptr(),
            out.stride(0) if T > 1 else self.N, self._fp32, _ws(b, dev), b.ws.numel(),
            _stream(dev, stream)))
        return out


class Experts4:
    """The experts of a layer in 4 bits: w_gate, w_up [E+S, d, f] of one kind and group, w_down
    [E+S, f, d]; E routed experts (default: all), then S shared ones; top-k; act as in MoELayer."""

    def __init__(self, w_gate: Weights4, w_up: Weights4, w_down: Weights4, k: int,
                 E: Optional[int] = None, act=None):
        self.lib = _lib.load()
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        self.E = w_gate.E if E is None else int(E)
        self.S, self.k = w_gate.E - self.E, int(k)
        self.d, self.f, self._dev = w_gate.K, w_gate.N, w_gate._dev
        if self.S < 0 or not 0 < self.k <= self.E:
            raise ValueError(f"{k} of {self.E} experts, {w_gate.E} given")
        shapes = [(w.E, w.K, w.N) for w in (w_gate, w_up, w_down)]
        if shapes[1] != shapes[0] or shapes[2] != (w_gate.E, self.f, self.d):
            raise ValueError(f"gate, up and down of shapes {shapes}")
        if (w_up.kind, w_up.group) != (w_gate.kind, w_gate.group):
            raise ValueError("gate and up of different kinds or groups")
        if w_up._dev != self._dev or w_down._dev != self._dev:
            raise ValueError("gate, up and down are on different devices")
        self.act = None if act is None else _lib.Swiglu(*[float(v) for v in act])
        self._act = None if self.act is None else _ref(self.act)
        self._call = self.lib.moe_expert_fwd_w4

    def buffers(self, T: int) -> Buffers4:
        _stream(self._dev, None)
        ws = int(self.lib.moe_expert_fwd_w4_workspace_size(T, self.k, self.E, self.S, self.d,
                                                           self.f))
        kw = dict(device=self.w_gate.codes.device)
        return Buffers4(T, torch.empty(T, self.d, dtype=BF16, **kw),
                        torch.empty(max(ws, 256), dtype=torch.uint8, **kw))

    def forward(self, x, topk_idx, topk_w, b: Buffers4, stream=None) -> torch.Tensor:
        """y [T, d] (b.y) of x [T, d] bf16 and its routing topk_idx, topk_w [T, k]."""
        T, k, dev = b.T, self.k, self._dev
        _check("moe_expert_fwd_w4", self._call(
            self.w_gate._ref, self.w_up._ref, self.w_down._ref, self._act,
            _packed("x", x, BF16, (T, self.d), dev),
            _packed("topk_idx", topk_idx, torch.int32, (T, k), dev),
            _packed("topk_w", topk_w, torch.float32, (T, k), dev), T, k, self.E, self.S,
            _packed("y", b.y, BF16, (T, self.d), dev), _ws(b, dev), b.ws.numel(),
            _stream(dev, stream)))
        return b.y

    def status(self, stream=None) -> int:
        """Synchronise and read (and clear) the device status word."""
        return int(self.lib.moe_status(_stream(self._dev, stream)))


@dataclass
class LayerBuffers4:
    """Routing, output and workspaces of one call of T tokens of a MoELayer4."""
    T: int
    logits: torch.Tensor
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    ws_route: torch.Tensor
    experts: Buffers4

    @property
    def y(self) -> torch.Tensor:
        return self.experts.y


class MoELayer4:
    """A layer for inference with experts in 4 bits: logits, top-k and weights as
    MoELayer's (the renormalised softmax, or ``router``), then moe_expert_fwd_w4."""

    def __init__(self, w_router, bias, experts: Experts4, router=None):
        self.lib = _lib.load()
        self.experts, self.router, self._dev = experts, router, experts._dev
        E, k = experts.E, experts.k
        self.w_router = w_router.contiguous()
        _packed("w_router", self.w_router, torch.float32, (experts.d, E), self._dev)
        self.bias = None if bias is None else bias.contiguous()
        if bias is not None:
            _packed("bias", self.bias, torch.float32, (E,), self._dev)
        if router is not None and (router.E, router.k) != (E, k):
            raise ValueError(f"the router chooses {router.k} of {router.E} experts, the layer "
                             f"{k} of {E}")
        if router is not None and router._dev not in (None, self._dev):
            raise ValueError("the router's balance is on another device than the experts")

    def buffers(self, T: int) -> LayerBuffers4:
        e = self.experts
        b = e.buffers(T)
        kw = dict(device=b.y.device)
        ws = int(self.lib.moe_workspace_size(_lib.MOE_WS_ROUTE, T, e.d, e.E, e.k, 16))
        return LayerBuffers4(
            T, torch.empty(T, e.E, dtype=torch.float32, **kw),
            torch.empty(T, e.k, dtype=torch.int32, **kw),
            torch.empty(T, e.k, dtype=torch.float32, **kw),
            torch.empty(max(ws, 256), dtype=torch.uint8, **kw), b)

    def route(self, x, b: LayerBuffers4, forced_idx=None, stream=None):
        e, dev = self.experts, self._dev
        T, s = b.T, _stream(dev, stream)
        xp = _packed("x", x, BF16, (T, e.d), dev)
        fp = None
        if forced_idx is not None:
            fp = _packed("forced_idx", forced_idx, torch.int32, (T, e.k), dev)
        out = (b.logits.data_ptr(), b.topk_idx.data_ptr(), b.topk_w.data_ptr(),
               b.ws_route.data_ptr(), b.ws_route.numel(), s)
        if self.router is not None:
            _check("moe_route_scored", self.lib.moe_route_scored(
                self.router._ref, xp, self.w_router.data_ptr(), _p(self.bias), fp, T, e.d, *out))
        else:
            _check("moe_route", self.lib.moe_route(
                xp, self.w_router.data_ptr(), _p(self.bias), fp, T, e.d, e.E, e.k, *out))

    def forward(self, x, b: LayerBuffers4, forced_idx=None, stream=None) -> torch.Tensor:
        """y = layer(x) into b.y; forced_idx [T, k]: the caller's choice of experts."""
        self.route(x, b, forced_idx, stream)
        return self.experts.forward(x, b.topk_idx, b.topk_w, b.experts, stream)

    def status(self, stream=None) -> int:
        """Synchronise and read (and clear) the device status word."""
        return self.experts.status(stream)
