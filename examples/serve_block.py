"""One transformer block as a server runs it: attention over a paged cache in
front of the routed expert layer.

    python examples/serve_block.py

A batch of prompts of different lengths goes through in one ragged step
(prefill); after that every sequence takes one token a step (decode), with the
step captured once into a CUDA graph: lengths and page table are read on the
device, so the same graph serves every step. Random weights; a token's output
row stands in for the next token's embedding. Projections and norms are
PyTorch's; rotary positions, the append to the cache, attention and the expert
layer are the library's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_routed_softmax_gb300.attention import (  # noqa: E402
    KVBatch, PagedAttention, Rope)
from mixture_experts_routed_softmax_gb300.layer import MoELayer  # noqa: E402

BF16 = torch.bfloat16


def rms(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-5)).to(BF16)


class Block:
    """Weights, cache and the calls of one block; ``lens`` on the host."""

    def __init__(self, d=2880, Hq=64, Hkv=8, D=64, f=2880, E=32, k=4, page_size=64,
                 max_pages=16, B=4, window=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*s, scale=1.0):
            return torch.randn(*s, generator=g, device="cuda") * scale

        self.d, self.Hq, self.Hkv, self.D, self.B = d, Hq, Hkv, D, B
        self.wqkv = rnd(d, (Hq + 2 * Hkv) * D, scale=d ** -0.5).to(BF16)
        self.wo = rnd(Hq * D, d, scale=(Hq * D) ** -0.5).to(BF16)
        self.moe = MoELayer(rnd(d, E, scale=d ** -0.5), None,
                            rnd(E, d, f, scale=d ** -0.5).to(BF16),
                            rnd(E, d, f, scale=d ** -0.5).to(BF16),
                            rnd(E, f, d, scale=f ** -0.5).to(BF16), k)
        shape = (B * max_pages, Hkv, page_size, D)
        self.attn = PagedAttention(torch.zeros(shape, dtype=BF16, device="cuda"),
                                   torch.zeros(shape, dtype=BF16, device="cuda"), Hq,
                                   rope=Rope.from_base(D, 150000.0), window=window,
                                   sinks=rnd(Hq))
        # every sequence has its pages from the start; a server hands them out
        order = torch.randperm(B * max_pages, generator=torch.Generator().manual_seed(seed))
        self.table = order.view(B, max_pages).to(torch.int32).cuda()
        self.kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")

    def batch(self, ql):
        """The ragged batch of ql[b] new tokens for sequence b; kv_len counts them
        once they are added (``step`` does not)."""
        cu = torch.tensor([0] + ql, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        return KVBatch(cu, self.kv_len, self.table, sum(ql), max(ql))

    def buffers(self, T):
        return self.attn.buffers(T), self.moe.fused_buffers(T)

    def step(self, x, batch, buf):
        """x [T, d] bf16, the batch's tokens -> [T, d]."""
        ab, mb = buf
        T, Hq, Hkv, D = batch.T, self.Hq, self.Hkv, self.D
        q, k, v = (rms(x) @ self.wqkv).split([Hq * D, Hkv * D, Hkv * D], dim=1)
        o = self.attn.forward(q.view(T, Hq, D), k.view(T, Hkv, D), v.view(T, Hkv, D), batch, ab)
        x = x + o.view(T, Hq * D) @ self.wo
        return x + self.moe.forward_fused(rms(x), mb)

    def prefill(self, x, ql):
        """Prompts of ql[b] tokens, x [sum(ql), d]; each sequence's last row."""
        self.kv_len += torch.tensor(ql, dtype=torch.int32, device="cuda")
        batch = self.batch(ql)
        y = self.step(x, batch, self.buffers(batch.T))
        return y[(batch.cu_q[1:] - 1).long()]


class Decoder:
    """A captured step of one token a sequence, the rows ``x`` [B, d] in and out.
    The graph holds addresses only: what it reads and writes stays with it."""

    def __init__(self, block, x):
        self.block, self.x = block, x.clone()
        self.batch, self.buf = block.batch([1] * block.B), block.buffers(block.B)
        s = torch.cuda.Stream()            # warm-up: a step that is taken back
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self._one()
            block.kv_len.sub_(1)
            self.x.copy_(x)
        torch.cuda.current_stream().wait_stream(s)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self._one()

    def _one(self):
        self.block.kv_len.add_(1)
        self.x.copy_(self.block.step(self.x, self.batch, self.buf))

    def step(self):
        self.graph.replay()
        return self.x


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 64, 333, 512])
    ap.add_argument("--tokens", type=int, default=64)
    args = ap.parse_args(argv)
    pages = (max(args.prompts) + args.tokens + 63) // 64
    block = Block(B=len(args.prompts), max_pages=pages)
    x = torch.randn(sum(args.prompts), block.d, device="cuda").to(BF16)
    last = block.prefill(x, args.prompts)
    dec = Decoder(block, last)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(args.tokens):
        dec.step()
    b.record()
    torch.cuda.synchronize()
    if block.attn.status():
        raise SystemExit("a kernel reported an error")
    print(f"{sum(args.prompts)} prompt tokens, then {args.tokens} steps of {block.B} sequences: "
          f"{a.elapsed_time(b) / args.tokens * 1e3:.1f} us a step; lengths "
          f"{block.kv_len.tolist()}")


if __name__ == "__main__":
    main()
