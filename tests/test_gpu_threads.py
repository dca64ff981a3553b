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
