"""Batches of no sequences and of more sequences than a block has threads, on the
GPU against the plain 64-bit forms."""
import pytest
import torch

import attention_ref as R
from test_gpu_attention import Case, _i32, _mod, _rot, _same

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


@pytest.mark.parametrize("window", [0, 800])
@pytest.mark.parametrize("ps", [16, 13])
@pytest.mark.parametrize("alone", [True, False])
def test_chunks_among_more_sequences_than_threads(alone, ps, window):
    """600 sequences, most of them empty or single tokens, chunks of several row tiles
    in front of and behind the 384th (a block looks at so many at a time). `alone`: the
    hint makes one kernel take all of them, else each takes its own."""
    B, Hq, Hkv = 600, 8, 1
    ql = [1 if i % 6 == 5 else 0 for i in range(B)]
    for i, n in {3: 650, 200: 431, 383: 380, 384: 333, 385: 64, 520: 512, 598: 389}.items():
        ql[i] = n
    ql[100] += 5 * B - sum(ql)             # on average five: 40 rows of a key head
    assert 0 < ql[100] < 200
    kv = [max(n, 1) + (i * 37) % 90 if n < 9 else n + (i * 53) % 400 for i, n in enumerate(ql)]
    c = Case(Hq, Hkv, 64, ps, ql, kv, seed=40)
    c.check(max_q=5 if alone else 700, window=window)


@pytest.mark.parametrize("G,nq,window", [(2, 1, 0), (8, 2, 0), (4, 3, 20)])
def test_many_units_of_a_few_keys(G, nq, window):
    """Enough of them for a warp each, empty ones in between."""
    kv = [(i * 53) % 176 for i in range(90)]
    ql = [min(nq, n) if i % 7 else 0 for i, n in enumerate(kv)]
    c = Case(8 * G, 8, 64, 16, ql, kv, seed=41)
    assert len(c.table[0]) * 16 <= 192
    c.check(window=window, sinks=torch.linspace(-4, 4, 8 * G, device="cuda"))
