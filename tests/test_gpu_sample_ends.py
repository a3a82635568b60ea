"""The draw at the two ends of [0, 1): ids of little weight before and behind one
that has nearly all of it, whose weights FP32 sums of the row round away; against
the definition in 64 bits.  Tolerances as in test_gpu_sample.py."""
import numpy as np
import pytest

import learner_ref as LR
import tokens_ref as R
from test_gpu_sample import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def heavy_rows(rng, T, V, light, where):
    """One id of weight 1 at about `where` of the row, `light` others of about half
    2^-24 each on both sides of it."""
    z = np.full((T, V), -np.inf)
    for t in range(T):
        z[t, rng.choice(V, min(light, V), replace=False)] = np.log(2.0 ** -25) + 0.5 * rng.standard_normal(min(light, V))
        z[t, int(where * (V - 1))] = 0.0
    return z


NEAR_1 = [1 - 2.0 ** -24, 1 - 2.0 ** -23, 1 - 2.0 ** -22, 1 - 3 * 2.0 ** -24]
NEAR_0 = [2.0 ** -24, 2.0 ** -23, 2.0 ** -26, 3 * 2.0 ** -24]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,light", [(4, 40, 24), (7, 9001, 40), (24, 500, 100), (60, 40, 30), (60, 9001, 60),
                                       (310, 1000, 50), (320, 33000, 100)])
def test_light_ids_at_the_ends(T, V, light, dtype):
    rng = np.random.default_rng(T + V + (dtype == "f32"))
    filters = [(0, 1.0, 0.0), (V // 2, 1.0, 0.0), (0, 1.0, 1e-9), (0, 1 - 2.0 ** -23, 0.0)]
    full = lambda f: (np.ones(T, np.float32), np.full(T, f[0], np.int32), np.full(T, f[1], np.float32),  # noqa: E731
                      np.full(T, f[2], np.float32))
    for where, us in [(0.1, NEAR_1), (0.6, NEAR_1), (0.9, NEAR_0), (0.5, NEAR_0)]:
        z = LR.round_to(heavy_rows(rng, 2 * T, V, light, where), dtype)
        u = rng.choice(us, 2 * T).astype(np.float32)
        # the weight of such an id is 2^-25: T of the rows in which no border is near
        far = [t for t in range(2 * T)
               if all(R.sample(z[t], 1.0, f[0], np.float32(f[1]), np.float32(f[2]), u[t])[3] > 2.0 ** -33 for f in filters)]
        z, u = z[far[:T]], u[far[:T]]
        for f in filters:
            check(z, dtype, *full(f), u, pad=3, lead=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(12, 700), (30, 2000), (100, 300), (100, 9001), (400, 4000), (320, 33000)])
def test_two_to_four_light_ids_behind(T, V, dtype):
    """One by one less than half an FP32 step of the row's sum, together more than
    1 - u: the row does not end with the heavy id."""
    rng = np.random.default_rng(3 * T + V + (dtype == "f32"))
    z = np.full((2 * T, V), -np.inf)
    for t in range(2 * T):
        at = int(rng.integers(0, V // 2))
        z[t, at] = 0.0
        n = int(rng.integers(2, 5))
        z[t, rng.choice(np.arange(at + 1, V), n, replace=False)] = np.log(2.0 ** -24 * rng.uniform(0.55, 0.97, n))
    z = LR.round_to(z, dtype)
    u = np.full(2 * T, 1 - 2.0 ** -24, np.float32)
    far = [t for t in range(2 * T) if R.sample(z[t], 1.0, 0, 1.0, 0.0, u[t])[3] > 2.0 ** -33][:T]
    check(z[far], dtype, np.ones(T, np.float32), np.zeros(T, np.int32), np.ones(T, np.float32), np.zeros(T, np.float32),
          u[far], pad=3, lead=1)
