"""The gradient through the entropy with weights that are large numbers: a
masked id's probability of 0 stays 0."""
import numpy as np
import pytest

import learner_ref as R
from test_gpu_logprobs import backward, forward, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inv_t,weight", [(1e6, 1e5), (1e6, 1e20), (1.0, 1e12), (1e-6, 1e25)])
def test_masked_ids_get_zero(inv_t, weight, dtype):
    """Tolerances as in test_gpu_logprobs.py."""
    import torch
    rng = np.random.default_rng(3)
    T, V = 4, 3001
    z = R.round_to(rng.standard_normal((T, V)) / inv_t, dtype)
    z[0, rng.random(V) < 0.3] = -np.inf
    z[1, rng.random(V) < 0.3] = R.LOWEST[dtype]
    z[2, 7:] = -np.inf
    masked = ~(z > -1e30)
    y = np.array([np.flatnonzero(~masked[t])[0] for t in range(T)], np.int32)
    g, ge = rng.standard_normal(T).astype(np.float32), (weight * rng.standard_normal(T)).astype(np.float32)
    for lead in [0, 1]:
        zd, yd = R.device_rows(z, dtype, 3, lead), torch.from_numpy(y).cuda()
        f = forward(zd, yd, inv_t, 0)
        dl = torch.full((T, V), 55.0, dtype=zd.dtype, device="cuda")
        assert backward(zd, yd, inv_t, f, torch.from_numpy(g).cuda(), torch.from_numpy(ge).cuda(), dl) == 0
        ref = R.logprobs_grad(z, y, inv_t, g.astype(float), ge.astype(float))
        r = R.logprobs(z, y, inv_t, 0)
        p, H = np.exp(r["lp"]), r["entropy"][:, None]
        with np.errstate(invalid="ignore"):
            lpH = np.where(p > 0, np.abs(r["lp"]) + H, 0)
            rel = 6e-6 + 4e-7 * np.where(p > 0, -r["lp"], 0)
        A, B = np.abs(g)[:, None], np.abs(ge)[:, None]
        tol = inv_t * (rel * p * (A + B * lpH) + B * p * 2e-5 * (1 + H) + 2e-7 * A) + 1e-37
        if dtype == "bf16":
            tol = tol + 2.0 ** -7.99 * np.abs(ref)
        got = dl.float().cpu().numpy()
        assert (got[masked] == 0).all()
        near(got, ref, tol)
