"""Lists that hold all of the teacher's mass, with the teacher's lse given: r =
1 - sum q is then what FP32 leaves of a difference of equals.

Tolerances.  The definition over the list (softmax of its entries, r = 0) and
the one with lse differ by the relative error of q that test_gpu_distill.py
states and bounds in tolerances(): as much again as the kernel may be off, so
twice that."""
import numpy as np
import pytest

import learner_ref as R
from test_gpu_distill import step, tolerances
from test_gpu_logprobs import near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def lse_of(a, inv_t, how):
    import torch
    x = torch.from_numpy(a)
    if how == "64 bits":
        return torch.logsumexp(x.double() * inv_t, 1).float().numpy()
    if how == "32 bits":
        return torch.logsumexp(x * inv_t, 1).numpy()
    return torch.logsumexp(x / np.float32(1 / inv_t), 1).numpy()


@pytest.mark.parametrize("how", ["64 bits", "32 bits", "by the temperature"])
@pytest.mark.parametrize("V,K,mean,inv_t", [(4099, 5, 0.0, 1.0), (2000, 32, 20.0, 1 / 0.7), (700, 256, -90.0, 0.5),
                                            (131072, 64, 30.0, 1.0), (33, 33, 5.0, 1.0)])
def test_nothing_off_the_list(V, K, mean, inv_t, how):
    """The same mask for teacher and student: K ids, the rest -inf (or no other
    ids at all).  Finite losses and gradients, and the list's own."""
    rng = np.random.default_rng(V + K)
    T = 200 if V < 10000 else 40
    z = np.full((T, V), -np.inf, np.float32)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    x = (2 * rng.standard_normal((T, K))).astype(np.float32)
    np.put_along_axis(z, ids, x, 1)
    a = (x + 0.5 * rng.standard_normal((T, K)) + mean).astype(np.float32)
    lse = lse_of(a, inv_t, how)
    g = rng.uniform(0.5, 2, T).astype(np.float32)
    o, loss2, grad2 = step(R.device_rows(z, "f32"), ids, a, lse, inv_t, g)
    assert o["status"] == 0
    loss, grad, _ = R.distill(z, ids, a, None, inv_t)
    tl, tg = tolerances(z, ids, a, lse, inv_t, g)
    for l in [o["loss"], loss2]:
        near(l.cpu().numpy(), loss, 2 * tl)
    for d in [o["grad"], grad2]:
        near(d.cpu().numpy(), grad * g.astype(float)[:, None], 2 * tg)


def test_small_masses_off_the_list_still_count():
    """A teacher's rest of 2^-14 and 1e-4 is no rounding: with nothing of the
    student off the list the loss is infinite, and with something there it is
    the definition's."""
    rng = np.random.default_rng(1)
    V, K = 900, 8
    for rest in [2.0 ** -14, 1e-4]:
        z = np.full((3, V), -np.inf, np.float32)
        z[:, :K] = rng.standard_normal((3, K))
        z[1:, K:] = -4.0
        ids = np.tile(np.arange(K, dtype=np.int32), (3, 1))
        a = rng.standard_normal((3, K)).astype(np.float32)
        lse = (np.log(np.exp(a.astype(float)).sum(1)) - np.log1p(-rest)).astype(np.float32)
        o, loss2, _ = step(R.device_rows(z, "f32"), ids, a, lse, 1.0, np.ones(3, np.float32))
        loss = R.distill(z, ids, a, lse, 1.0)[0]
        tl = tolerances(z, ids, a, lse, 1.0, np.ones(3, np.float32))[0]
        for l in [o["loss"].cpu().numpy(), loss2.cpu().numpy()]:
            assert np.isposinf(l[0])
            near(l[1:], loss[1:], tl[1:])
