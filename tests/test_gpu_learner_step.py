"""The learner-step example: the operators together with the expert layer.  Its
loss and logit gradient against float64 autograd on its own logits, the first
and the final norm's gradients against float64 autograd from the gradients that
enter them, and the status word.

Tolerances: the loss is a mean of FP32 rows, 1e-5; the logit gradient is the
sum of two BF16 roundings and rounded again, each 2^-8 of the largest of its
parts (row maxima differ by far more between entries, so elementwise against
the sum of magnitudes); norms as in test_gpu_norm.py, with BF16's 2^-8."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("args", [[], ["--layer", "small", "--vocab", "8192"]])
def test_learner_step(args):
    import learner_step as S
    import torch
    r = S.main(args)
    x, res, _, tokens, adv, (ids, values, lse) = r["inputs"]
    T, V = r["logits"].shape
    z = r["logits"].double().requires_grad_()
    logp = torch.log_softmax(z, 1)
    act = (tokens >= 0).double()
    n = act.sum()
    lp = logp.gather(1, tokens.long().clamp(min=0)[:, None]).squeeze(1) * act
    ent = -(logp.exp() * logp).sum(1)
    q = torch.exp(values.double() - lse.double()[:, None])
    rest = 1 - q.sum(1)
    on = torch.zeros_like(z, dtype=torch.bool).scatter_(1, ids.long(), True)
    ls = torch.logsumexp(z.masked_fill(on, -float("inf")), 1) - torch.logsumexp(z, 1)
    kl = (q * (q.log() - logp.gather(1, ids.long()))).sum(1) + rest * (rest.log() - ls)
    policy = -(adv.double() * lp).sum() / n - 0.01 * (ent * act).sum() / n
    loss = policy + 0.5 * kl.mean()
    assert abs(loss.item() - r["loss"].item()) <= 1e-5 * (1 + abs(loss.item()))
    g1, = torch.autograd.grad(policy, z, retain_graph=True)
    g2, = torch.autograd.grad(0.5 * kl.mean(), z)
    off = (r["dlogits"].double() - (g1 + g2)).abs()
    assert (off <= 2.0 ** -7.9 * (g1.abs() + g2.abs()) * 2 + 1e-9).all()
    assert torch.equal(r["seen"]["top_ids"][:, 0].long(), r["logits"].float().max(1).values[:, None]
                       .eq(r["logits"].float()).int().argmax(1))
    b = r["block"]
    # both norms, from what the example kept
    h1 = (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(b.h1, h1)
    h2 = b.h2.double().requires_grad_()
    w = b.w_out.double().requires_grad_()
    y2 = h2 / (h2.square().mean(1, keepdim=True) + S.EPS).sqrt() * w
    up = (r["dlogits"] @ b.head).double()
    gh, gw = torch.autograd.grad((y2 * up).sum(), (h2, w))
    assert (r["grads"]["dw_out"].double() - gw).norm() <= 1e-5 * gw.norm()
    assert (b.y2.double() - y2).abs().max() <= 2.0 ** -7.9 * y2.abs().max()
    h = b.h1.double().requires_grad_()
    wi = b.w_in.double().requires_grad_()
    y1 = h / (h.square().mean(1, keepdim=True) + S.EPS).sqrt() * wi
    codes = b.y8.view(torch.float8_e4m3fn).double()
    d = h.shape[1]
    rr, cc = np.arange(T)[:, None], np.arange(d // 32)[None, :]
    at = ((rr // 128) * (d // 128) + cc // 4) * 512 + (rr % 32) * 16 + (rr % 128) // 32 * 4 + cc % 4
    sc = torch.from_numpy(np.ldexp(1.0, b.y8_sf.cpu().numpy()[at].astype(int) - 127)).cuda().repeat_interleave(32, 1)
    # E4M3: half a step of 2^-3 of the value, or of the smallest steps of its block
    assert ((codes * sc - y1).abs() <= 2.0 ** -4 * 1.001 * y1.abs() + 2.0 ** -9 * sc).all()
    assert torch.isfinite(r["grads"]["dx"].float()).all() and torch.isfinite(r["grads"]["dw_in"]).all()
    assert all(torch.isfinite(r["grads"][k]).all() and r["grads"][k].abs().sum() > 0 for k in ["dW1", "dW2"])
