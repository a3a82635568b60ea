"""The rollout example: embedding, block, draw and the way back to the table run
together.  The drawn tokens against their definition on the example's own logits,
the learner's log-probabilities against the sampler's, the logit gradient against
float64 autograd, and the table's gradient against the sum of the rows that reach
it.

Tolerances: log-probabilities as in test_gpu_sample.py, on both sides; the logit
gradient is rounded to BF16 once, 2^-9 of the value and half the smallest step, and
carries FP32 errors of 2^-18 of its parts; the table's gradient as in
test_gpu_embed.py."""
import os
import sys

import numpy as np
import pytest

import tokens_ref as R

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("args", [[], ["--layer", "small", "--vocab", "8192", "--steps", "2"]])
def test_rollout_step(args):
    import rollout_step as S
    import torch
    r = S.main(args)
    p, seen, step = r["policy"], r["seen"], r["step"]
    T, E, k, d, F = p.shape
    z = seen["logits"].float().cpu().numpy()
    inv_t = np.float32(1.0 / 0.8)
    drawn = seen["drawn"].cpu().numpy()
    for t in range(0, T, max(1, T // 40)):
        want = R.sample(z[t], inv_t, 50, np.float32(0.95), 0.0, seen["u"][t].item())
        assert want[3] > 2.0 ** -33 and drawn[t] == want[0]
        for got, w in [(seen["logprob"][t].item(), want[1]), (seen["kept_logprob"][t].item(), want[2])]:
            assert abs(got - w) <= 2.0 ** -22 * (abs(w) + 2 * np.log(p.vocab)) + 2.0 ** -18
    # the learner runs the same block on the same tokens: the same logits, and the
    # sampler's log-probability
    assert ((step["logprob"] - seen["logprob"]).abs() <= 2.0 ** -17 + 2.0 ** -21 * seen["logprob"].abs()).all()
    fed = seen["fed"]
    assert (fed[T - T // 16:] == -1).all() and (p.x[fed < 0] == 0).all()
    assert torch.equal(p.x[fed >= 0], (p.table[fed[fed >= 0].long()].float() * S.SCALE).to(torch.bfloat16))
    # the logit gradient
    x = seen["logits"].double().requires_grad_()
    lp = torch.log_softmax(x * float(inv_t), 1).gather(1, seen["drawn"].long()[:, None]).squeeze(1)
    g = torch.zeros(T, dtype=torch.float64, device="cuda")
    has = fed >= 0
    gen = torch.Generator(device="cuda").manual_seed(7)
    torch.randint(0, p.vocab, (T,), generator=gen, device="cuda", dtype=torch.int64)
    adv = torch.randn(T, generator=gen, device="cuda").double()  # as main drew them
    g[has] = -adv[has] / has.sum()
    dx, = torch.autograd.grad((g * lp).sum(), x)
    parts = float(inv_t) * g.abs()[:, None]
    assert ((step["dlogits"].double() - dx).abs() <= 2.0 ** -8 * dx.abs() + 2.0 ** -17 * parts).all()
    # the table's gradient
    dtable = step["grads"]["dtable"].cpu().numpy()
    want, mag, n = R.embed_grad(step["grads"]["dx"].float().cpu().numpy(), fed.cpu().numpy(), p.vocab, S.SCALE)
    assert (np.abs(dtable - want) <= 2.0 ** -24 * (n[:, None] + 2) * mag).all()
    assert (np.abs(dtable).sum(1)[n == 0] == 0).all() and np.abs(dtable).sum() > 0
