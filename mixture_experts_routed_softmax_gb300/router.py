"""The scored router, driven through the C ABI: the choice of experts by softmax or
sigmoid scores with a bias for balance, groups and renormalised weights
(moe_select), and its gradient (moe_select_bwd).

A ``Router`` works on given logits; ``MoELayer(router=...)`` puts it behind the
layer's own (moe_route_scored) and into its backward pass (moe_logits_bwd).
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from .attention import _check, _ref, _stream

SCORES = {"softmax": _lib.MOE_SCORE_SOFTMAX, "sigmoid": _lib.MOE_SCORE_SIGMOID}


def _packed(name: str, t: torch.Tensor, dtype, shape, dev: int) -> int:
    """Check a packed array on device ``dev``; its address."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a packed {dtype} tensor of shape {tuple(shape)} on cuda:{dev} "
                         "is needed")
    return t.data_ptr()


@dataclass
class Choice:
    """The chosen experts of T tokens, their weights and, for training, the
    logits' gradient."""
    T: int
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    d_logits: Optional[torch.Tensor] = None


class Router:
    """How k of E experts are chosen and weighted.

    score: "softmax" or "sigmoid" of the logits. balance [E] fp32: added to the
    scores for the choice alone, held by reference, so a training loop moves it in place.
    n_groups, topk_groups, group_rank: runs of E / n_groups experts of which the
    best topk_groups stay, ranked by the sum of their group_rank (1 or 2) largest values.
    renormalise: weights sum to ``scale``; otherwise they are scale * score.
    """

    # the kernels read it at this address: it can be written to, not replaced
    balance = property(lambda self: self._balance)

    def __init__(self, E: int, k: int, score: str = "softmax", n_groups: int = 1,
                 topk_groups: int = 1, group_rank: int = 2, renormalise: bool = True,
                 scale: float = 1.0, balance: Optional[torch.Tensor] = None):
        self.lib = _lib.load()
        if score not in SCORES:
            raise ValueError(f"score: one of {sorted(SCORES)} is needed, not {score!r}")
        if E <= 0 or E > 1024 or not 0 < k <= min(E, 32):
            raise ValueError(f"{k} of {E} experts: 1 <= k <= min(E, 32) and E <= 1024 are needed")
        if n_groups < 1 or E % n_groups or not 1 <= topk_groups <= n_groups:
            raise ValueError(f"{topk_groups} of {n_groups} groups of {E} experts")
        if k > topk_groups * (E // n_groups):
            raise ValueError(f"{k} experts from {topk_groups} groups of {E // n_groups}")
        if group_rank not in (1, 2):
            raise ValueError(f"group_rank: 1 or 2, not {group_rank}")
        if not math.isfinite(scale):
            raise ValueError(f"scale: {scale}")
        if balance is not None and (balance.dtype != torch.float32
                                    or tuple(balance.shape) != (E,) or not balance.is_cuda
                                    or not balance.is_contiguous()):
            raise ValueError(f"balance: a packed fp32 tensor of {E} values on the device is needed")
        self.E, self.k, self.score, self.scale = int(E), int(k), score, float(scale)
        self.renormalise, self._balance = bool(renormalise), balance
        # every expert has a gradient where softmax scores stay as they are
        self.dense = score == "softmax" and not self.renormalise
        self.args = _lib.RouterArgs(None if balance is None else balance.data_ptr(), self.E,
                                    self.k, SCORES[score], int(n_groups), int(topk_groups),
                                    int(group_rank), int(self.renormalise), self.scale)
        self._ref = _ref(self.args)
        self._dev = None if balance is None else balance.device.index
        self._call, self._call_bwd = self.lib.moe_select, self.lib.moe_select_bwd

    def buffers(self, T: int, backward: bool = False, device="cuda") -> Choice:
        return Choice(
            T=T, topk_idx=torch.empty(T, self.k, dtype=torch.int32, device=device),
            topk_w=torch.empty(T, self.k, dtype=torch.float32, device=device),
            d_logits=(torch.empty(T, self.E, dtype=torch.float32, device=device) if backward
                      else None))

    def _device(self, logits: torch.Tensor) -> int:
        dev = logits.get_device()
        if dev < 0 or (self._dev is not None and dev != self._dev):
            raise ValueError(f"logits: on {logits.device}, "
                             + ("a CUDA tensor is needed" if self._dev is None else
                                f"the balance is on cuda:{self._dev}"))
        return dev

    def select(self, logits, b: Choice, forced_idx=None, stream=None) -> Choice:
        """The choice from logits [T, E] fp32 into b.topk_idx and b.topk_w
        [T, k]; forced_idx [T, k] int32: the weights of that choice instead."""
        T, E, k, dev = b.T, self.E, self.k, self._device(logits)
        fp = None
        if forced_idx is not None:
            fp = _packed("forced_idx", forced_idx, torch.int32, (T, k), dev)
        _check("moe_select", self._call(
            self._ref, _packed("logits", logits, torch.float32, (T, E), dev), fp, T,
            _packed("topk_idx", b.topk_idx, torch.int32, (T, k), dev),
            _packed("topk_w", b.topk_w, torch.float32, (T, k), dev), _stream(dev, stream)))
        return b

    def select_bwd(self, d_topk_w, logits, b: Choice, accumulate: bool = False, stream=None):
        """The logits' gradient from that of b's weights into b.d_logits [T, E],
        written whole or (accumulate) added to."""
        T, E, k, dev = b.T, self.E, self.k, self._device(logits)
        if b.d_logits is None:
            raise ValueError("buffers without d_logits: make them with backward=True")
        _check("moe_select_bwd", self._call_bwd(
            self._ref, _packed("d_topk_w", d_topk_w, torch.float32, (T, k), dev),
            _packed("logits", logits, torch.float32, (T, E), dev),
            _packed("topk_idx", b.topk_idx, torch.int32, (T, k), dev), T, int(accumulate),
            _packed("d_logits", b.d_logits, torch.float32, (T, E), dev), _stream(dev, stream)))
        return b.d_logits
