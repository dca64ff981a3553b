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


def _one_page(q, k, v, scale):
    """Attention of q [nq, G, D] over the one page in 64 bits: out, sum of weights
    times |values|, log-sum-exp, the largest sum of |terms| of a score."""
    x, K, V = q.double().flatten(0, 1), k[0, 0].double(), v[0, 0].double()
    s = x @ K.T * scale
    lse = torch.logsumexp(s, 1, keepdim=True)
    p = torch.exp(s - lse)
    mag = (x.abs() @ K.abs().T * scale).amax(1, keepdim=True)
    return [t.view(*q.shape[:2], -1) for t in (p @ V, p @ V.abs(), lse, mag)]


# new tokens, heads of the one key head, sequences, D, page size, keys: enough
# sequences that units are not cut into many parts. Up to 32 rows a unit, then more.
LONG = ([(nq, G, 304, D, 65536, 1 << 24) for nq, G in ((1, 8), (1, 1), (4, 8)) for D in (64, 128)]
        + [(nq, 8, 304, D, 65535, 1 << 24) for nq, D in ((1, 64), (3, 40), (3, 128))]
        + [(nq, G, 304, D, 65536, 1 << 22) for nq, G in ((16, 16), (8, 16), (45, 5))
           for D in (64, 128)]
        + [(16, 16, 152, D, 65535, 1 << 21) for D in (40, 128)])


@pytest.mark.parametrize("grow", [0.0, 30.0])
@pytest.mark.parametrize("nq,G,B,D,ps,n", LONG)
def test_long_sums(nq, G, B, D, ps, n, grow):
    """Values of one sign, and weights that are all alike or grow along the page by
    e^30, so that references move between and inside its 512 tiles.

    The matrix unit cuts the 16 products it adds, and the sum they join, at the
    sum's last place: 17 times 2^-23 of it in each 16-key step at most. An
    accumulator takes 65536 keys, 4096 steps, and over these is half of its end in
    the mean: 17 2^-23 2^11. Sums in fp32, half an ulp for each term: up to 1024
    groups of 32 terms, joined up to 64 times, 2^-13; up to 32 rows a unit, one term
    at a time, 16384 of them and half of the sum in the mean, 2^-11. Weights are
    rounded to bf16 up to twice, and a score is off by e at most
    (tests/attention_ref.py)."""
    u = torch.finfo(BF16).eps / 2
    g = torch.Generator(device="cuda").manual_seed(nq * G + D)
    k = torch.zeros(1, 1, ps, D, dtype=BF16, device="cuda")
    v = (1.0 + torch.rand(1, 1, ps, D, generator=g, device="cuda")).to(BF16)
    q = torch.randn(nq, G, D, generator=g, device="cuda").to(BF16)
    scale = D ** -0.5
    if grow:
        q[..., 0] = 2.0
        k[0, 0] = (0.3 * torch.randn(ps, D, generator=g, device="cuda")).to(BF16)
        k[0, 0, :, 0] = torch.linspace(-grow / 2 / scale, 0.0, ps, device="cuda").to(BF16)
    pages = n // ps
    A = _mod()
    layer = A.PagedAttention(k, v, G, causal=False)
    T = B * nq
    batch = A.KVBatch((torch.arange(B + 1, device="cuda") * nq).int(),
                      torch.full((B,), pages * ps, dtype=torch.int32, device="cuda"),
                      torch.zeros(B, pages, dtype=torch.int32, device="cuda"), T, nq)
    b = layer.buffers(T, lse=True)
    layer.attend(q.repeat(B, 1, 1), batch, b)
    assert layer.status() == 0
    out, a, lse, mag = _one_page(q, k, v, scale)
    e = (D + 16) * 2.0 ** -23 * mag + 2.0 ** -20
    sums = 2.0 ** -11 if nq * G <= 32 else 2.0 ** -13
    tol = u * out.abs() + (2 * u + 2 * e + 17 * 2.0 ** -12 + sums) * (1 + u) * a
    if not grow:                     # weights of one: nothing is rounded
        tol = u * out.abs() + (17 * 2.0 ** -12 + sums) * (1 + u) * a
    err = (b.out.view(B, nq, G, D).double() - out).abs()
    assert float((err / tol).max()) <= 1.0, float((err / out).max())
    lse = lse[..., 0] + math.log(pages)
    err = (b.lse.view(B, nq, G).double() - lse).abs()
    ltol = e[..., 0] + sums + 2.0 ** -20 * (1 + lse.abs())
    assert float((err / ltol).max()) <= 1.0, float(err.max())


def test_long_units_where_the_hint_says_short_ones():
    """A batch taken for many sequences of few keys, of which one has 140000 new
    tokens that see all that follow: units of one warp, in several pieces. Weights
    of one: a row's output is the mean of the values from its first key on."""
    A = _mod()
    B, D, n, window = 640, 64, 140000, 100
    g = torch.Generator(device="cuda").manual_seed(5)
    pages = (n + 15) // 16
    k = torch.zeros(pages, 1, 16, D, dtype=BF16, device="cuda")
    v = (1.0 + torch.rand(pages, 1, 16, D, generator=g, device="cuda")).to(BF16)
    cu = torch.full((B + 1,), n, dtype=torch.int32, device="cuda")
    cu[:18] = 0
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[17] = n
    table = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
    table[17] = torch.arange(pages, device="cuda")
    batch = A.KVBatch(cu, lens, table, n, max_q=0)
    layer = A.PagedAttention(k, v, 1, causal=False, window=window)
    b = layer.buffers(n, lse=True)
    layer.attend(torch.zeros(n, 1, D, dtype=BF16, device="cuda"), batch, b)
    assert layer.status() == 0
    first = (torch.arange(n, device="cuda") - window + 1).clamp(min=0)
    seen = (n - first).double()
    V = v.view(-1, D)[:n].double()
    ahead = torch.cat([torch.zeros(1, D, dtype=torch.float64, device="cuda"), V.cumsum(0)])
    out = (ahead[n] - ahead[first]) / seen[:, None]
    tol = torch.finfo(BF16).eps / 2 * out + (17 * 2.0 ** -12 + 2.0 ** -11) * 1.01 * out
    assert float(((b.out[:, 0].double() - out).abs() / tol).max()) <= 1.0
    assert float((b.lse[:, 0].double() - seen.log()).abs().max()) <= 2.0 ** -11 + 2.0 ** -16
