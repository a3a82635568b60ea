"""Host threads that call the learner operators at the same time, with sizes
that need different amounts of shared memory in the same kernels: no call is
refused, and each gives the bits that it gives alone."""
import threading

import pytest

import nvfp4_w4a4_moe_top_gb300 as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def together(jobs, calls):
    """Each job called `calls` times by a thread of its own on a stream of its
    own; the errors of all."""
    import torch
    errors, gate = [], threading.Barrier(len(jobs))

    def work(job):
        s = torch.cuda.Stream()
        gate.wait()
        try:
            for i in range(calls):
                job(s)
                if i % 100 == 99:
                    s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))
        s.synchronize()
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


def test_norm_gradients():
    import torch
    jobs, outs = [], []
    for d in [2560, 4096, 2304, 3584]:
        x = torch.randn((8, d), device="cuda").to(torch.bfloat16)
        r, w, dx = torch.ones(8, device="cuda"), torch.ones(d, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
        job = lambda s, x=x, r=r, w=w, dx=dx: M.moe_add_rmsnorm_backward(x, None, x, r, w, dx, None, None, None, s)  # noqa: E731
        job(None)
        jobs.append(job)
        outs.append((dx, dx.clone()))
    torch.cuda.synchronize()
    for dx, _ in outs:
        dx.zero_()
    torch.cuda.synchronize()
    assert together(jobs, 4000) == []
    for dx, alone in outs:
        assert torch.equal(dx, alone)


def test_distillation():
    import torch
    jobs, outs = [], []
    for V in [70000, 1000000, 150000, 600000]:
        z = torch.randn((1, V), device="cuda").to(torch.bfloat16)
        ids, a = torch.arange(8, dtype=torch.int32, device="cuda")[None], torch.randn((1, 8), device="cuda")
        g, loss, dl = torch.ones(1, device="cuda"), torch.empty(1, device="cuda"), torch.empty_like(z)

        def job(s, z=z, ids=ids, a=a, g=g, loss=loss, dl=dl):
            M.moe_distill_topk(z, ids, a, None, 1.0, loss, None, None, s)
            M.moe_distill_topk_train(z, ids, a, None, 1.0, g, loss, dl, None, s)
        job(None)
        jobs.append(job)
        outs.append((loss, dl, loss.clone(), dl.clone()))
    torch.cuda.synchronize()
    for loss, dl, _, _ in outs:
        loss.zero_()
        dl.zero_()
    torch.cuda.synchronize()
    assert together(jobs, 2000) == []
    for loss, dl, alone, grad in outs:
        assert torch.equal(loss, alone) and torch.equal(dl, grad)
