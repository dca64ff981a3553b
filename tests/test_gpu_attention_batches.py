"""Batches of no sequences and of more sequences than a block has threads, on the
GPU against the plain 64-bit forms."""
import pytest
import torch

import attention_ref as R
from test_gpu_attention import _i32, _mod, _rot, _same

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("positions", [True, False])
def test_rows_of_a_batch_without_sequences(positions):
    """A captured step's rows while no sequence is being served: queries are rotated,
    the cache stays, and attention writes nothing."""
    A = _mod()
    rope, w, axis = _rot(64, False, 1)
    cache = torch.randn(4, 2, 16, 64, device="cuda").to(BF16)
    before = cache.clone()
    layer = A.PagedAttention(cache, cache, 8, rope=rope)
    T = 5
    batch = A.KVBatch(_i32([0]), _i32([]), torch.empty(0, 3, dtype=torch.int32, device="cuda"), T)
    q = torch.randn(T, 8, 64, device="cuda").to(BF16)
    k = torch.randn(T, 2, 64, device="cuda").to(BF16)
    pos = _i32([[3, 1, 4, 1, 5]]) if positions else None
    b = layer.buffers(T, lse=True)
    b.out.fill_(7.0)
    b.lse.fill_(7.0)
    layer.forward(q, k, k, batch, b, pos=pos)
    assert layer.status() == 0
    ref, tol = R.rotate(q, pos if positions else _i32([[0] * T]), w, axis)
    _same(b.q, ref, tol, "q")
    assert torch.equal(cache, before)
    assert bool((b.out == 7).all()) and bool((b.lse == 7).all())
