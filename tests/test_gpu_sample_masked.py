"""Masked ids (-inf, the type's lowest value) at the start and the end of a row:
u = 0 and a u far below any weight draw the lowest of the ids that each filter
keeps, u next to 1 the highest, both from the definition in 64 bits."""
import numpy as np
import pytest

import learner_ref as LR
import tokens_ref as R
from test_gpu_sample import draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("T", [6, 60])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_first_and_last_kept_id(T, dtype):
    rng = np.random.default_rng(T)
    V = 5000
    f = lambda v, t=np.float32: np.full(T, v, t)  # noqa: E731
    for mask in [-np.inf, LR.LOWEST[dtype]]:
        z = LR.round_to(rng.standard_normal((T, V)), dtype)
        z[:, :1000] = mask
        z[:, 4000:] = mask
        for k, p, m in [(0, 1.0, 0.0), (40, 1.0, 0.0), (2500, 1.0, 0.0), (4500, 1.0, 0.0), (0, 0.5, 0.0), (0, 0.97, 0.0),
                        (0, 1 - 2.0 ** -24, 0.0), (0, 1.0, 1e-30), (0, 1.0, 0.1), (300, 0.8, 0.05)]:
            for u, least in [(0.0, True), (1e-30, True), (1 - 2.0 ** -24, False)]:
                tokens, lp, kept = draw(z, dtype, None, f(k, np.int32), f(p), f(m), f(u))
                for t in range(T):
                    # its first id with any weight; for the last, the definition itself: an
                    # id of 3000 such has more than 2^-24 of the weight
                    want = R.sample(z[t], 1.0, k, np.float32(p), np.float32(m), np.float32(0.0 if least else u))
                    assert least or want[3] > 2.0 ** -33
                    assert tokens[t] == want[0] and 1000 <= tokens[t] < 4000, (mask, k, p, m, u, t)
                assert np.isfinite(lp).all() and (kept >= lp - 2.0 ** -17).all()
