"""Calls of several threads at once, each with its own stream and buffers: what a call sets for
a kernel holds for every other call of that kernel."""
import threading

import numpy as np
import pytest
import torch

import router_ref as R

pytestmark = pytest.mark.gpu


def _together(jobs):
    """Runs the jobs in a thread each, started together; raises what one of them raised."""
    gate, errors = threading.Barrier(len(jobs)), []

    def work(job):
        try:
            gate.wait()
            job()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


def test_choices_of_different_E():
    from mixture_experts_routed_softmax_gb300.router import Router
    rng = np.random.default_rng(0)
    jobs, checks = [], []
    for E, groups in ((1024, 64), (800, 50), (1000, 40), (784, 49)):
        r = Router(E, 4, n_groups=groups, topk_groups=5)
        l = rng.standard_normal((8, E)).astype(np.float32)
        lg, b, s = torch.tensor(l).cuda(), r.buffers(8), torch.cuda.Stream()

        def job(r=r, lg=lg, b=b, s=s):
            for _ in range(2000):
                r.select(lg, b, stream=s)

        jobs.append(job)
        checks.append((l, groups, b))
    torch.cuda.synchronize()
    _together(jobs)
    for l, groups, b in checks:
        want = [R.choose(row, 4, n_groups=groups, topk_groups=5) for row in l]
        np.testing.assert_array_equal(b.topk_idx.cpu().numpy(), want)


def test_permutes_of_different_E():
    import workloads
    from mixture_experts_routed_softmax_gb300.layer import MoELayer
    jobs, checks = [], []
    for E in (8, 1024, 64, 512):
        wl = workloads.Workload("threads", T=5000, d=64, f=64, E=E, k=4, align=16)
        inp = workloads.generate(wl)
        layer = MoELayer.from_inputs(inp, 4, 16)
        x, b, s = inp["x"].cuda(), layer.buffers(5000, backward=False), torch.cuda.Stream()
        layer.route(x, b)
        layer.permute(x, b)
        torch.cuda.synchronize()
        want = b.dst_row.clone()
        b.dst_row.fill_(-7)

        def job(layer=layer, x=x, b=b, s=s):
            for _ in range(1000):
                layer.permute(x, b, None, s)

        jobs.append(job)
        checks.append((want, b))
    torch.cuda.synchronize()
    _together(jobs)
    for want, b in checks:
        assert torch.equal(b.dst_row, want)


def test_4_bit_calls_at_once():
    """Rows and tile kernels of several streams on the GPU at a time: the bits of calls alone."""
    from mixture_experts_routed_softmax_gb300.w4 import Experts4, Linear4, Weights4
    gen = torch.Generator("cuda").manual_seed(3)

    def weights(E, K, N, kind):
        w = torch.randn(E, K, N, generator=gen, device="cuda") / K ** 0.5
        return Weights4.quantise(w.to(torch.bfloat16), kind, 64)

    jobs, checks = [], []
    for T, kind in ((1, "int4"), (30, "fp4"), (400, "int4"), (900, "fp4")):
        ex = Experts4(weights(12, 520, 264, kind), weights(12, 520, 264, kind),
                      weights(12, 264, 520, kind), k=3)
        lin = Linear4(weights(1, 520, 1032, kind))
        x = torch.randn(T, 520, generator=gen, device="cuda").to(torch.bfloat16)
        idx = torch.argsort(torch.rand(T, 12, generator=gen, device="cuda"), 1)[:, :3]
        idx, w = idx.to(torch.int32).contiguous(), torch.rand(T, 3, generator=gen, device="cuda")
        be, bl, s = ex.buffers(T), lin.buffers(T), torch.cuda.Stream()
        want = (ex.forward(x, idx, w, be).clone(), lin.apply(x, bl).clone())
        be.y.zero_()
        bl.y.zero_()

        def job(ex=ex, lin=lin, x=x, idx=idx, w=w, be=be, bl=bl, s=s):
            for _ in range(200):
                ex.forward(x, idx, w, be, stream=s)
                lin.apply(x, bl, stream=s)

        jobs.append(job)
        checks.append((want, be, bl))
    torch.cuda.synchronize()
    _together(jobs)
    for want, be, bl in checks:
        assert torch.equal(be.y, want[0]) and torch.equal(bl.y, want[1])
