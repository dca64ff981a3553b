"""Attention over very long caches on the GPU. Every entry of the page table names
the same page, so a cache of up to 2^30 keys takes little memory and its results
follow from one page's: the mean over the page, and a log-sum-exp that is longer
by the logarithm of the repetitions."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _mod():
    from mixture_experts_routed_softmax_gb300.build import build
    build()
    from mixture_experts_routed_softmax_gb300 import attention
    return attention


def _repeated(Hq, Hkv, D, ps, pages, ql, n, k, v, **kw):
    """Queries of zeros (every weight is the same), len(ql) sequences of n keys in
    the same page over and over: the layer, its buffers."""
    A = _mod()
    layer = A.PagedAttention(k, v, Hq, causal=False, **kw)
    B, T = len(ql), sum(ql)
    cu = torch.tensor([sum(ql[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    batch = A.KVBatch(cu, torch.full((B,), n, dtype=torch.int32, device="cuda"),
                      torch.zeros(B, pages, dtype=torch.int32, device="cuda"), T, max(ql))
    b = layer.buffers(T, lse=True)
    layer.attend(torch.zeros(T, Hq, D, dtype=BF16, device="cuda"), batch, b)
    return layer, b


def test_units_that_take_seconds():
    """The longest caches: one block works for seconds on one unit, of which some of
    its warps have little to do but wait. Waits give up when nothing moves, not
    when a unit is long.

    The log-sum-exp shows that no key is left out: the sums are multiples of 64
    below 2^30 but for the last keys, joined over at most 16 parts in fp32 (16
    2^-24 of the sum), and the logarithm near 21 is off by two steps of 2^-19 at
    most; together below 2^-17."""
    H, D, ps, pages = 17, 8, (1 << 20) - 1, 1024
    n = pages * ps - 5
    k = torch.zeros(1, H, ps, D, dtype=BF16, device="cuda")
    v = torch.ones(1, H, ps, D, dtype=BF16, device="cuda")
    layer, b = _repeated(H, H, D, ps, pages, [40], n, k, v)
    assert layer.status() == 0
    assert float((b.lse.double() - math.log(n)).abs().max()) <= 2.0 ** -17
