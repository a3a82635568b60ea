"""The draw from rows whose weight reaches far below zero: hot temperatures over
wide logits, so that a filter's edge lies among values of any size; against the
definition in 64 bits.

Tolerance of kept_logprob = (x - m) inv_t - log1p(S - 1): the difference, the
product and S - 1 are rounded once each, 2^-24 of them; weights are whole numbers
to 2^-34; log1pf is documented to one unit in the last place, 2^-23; the last
subtraction is rounded once more.  With |z| and ln S: 2^-23 |z| + 2^-24 + 2^-23 ln S
+ 2^-24 (|z| + ln S) + 2^-34, less than 2^-22 (|z| + ln S) + 2^-23.  What filters
keep is weighed so in every launch; the tokens have no tolerance."""
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


def check(z, dtype, inv_t, k, p, m, u):
    tokens, _, kept = draw(z, dtype, inv_t, k, p, m, u)
    want = R.sample_rows(z, inv_t, k, p, m, u)
    assert (want[3] > 2.0 ** -33).all(), "a decision of these inputs lies on its border"
    assert np.array_equal(tokens, want[0]), np.nonzero(tokens != want[0])
    zt = (z.astype(np.float64).max(1) - z[np.arange(len(z)), want[0]]) * inv_t.astype(np.float64)
    ln_sum = -want[2] - zt
    off = np.abs(kept - want[2])
    assert (off <= 2.0 ** -22 * (zt + ln_sum) + 2.0 ** -23).all(), off.max()


def wide_rows(rng, T, V, dtype):
    """Logits from -100 up to a row's maximum of 1 to 40, or of -1."""
    top = rng.choice([1.0, 10.0, 40.0, -1.0], (T, 1))
    return LR.round_to(top - rng.random((T, V)) * (100 + top), dtype)


# T: a cluster per row with one and with two blocks per SM; few open rows behind the
# first launch; many, a block each.  5003 ids: small blocks.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(5, 9001), (24, 9001), (48, 9001), (310, 8200), (40, 5003)])
def test_min_p_far_below_zero(T, V, dtype):
    """min_p alone; with a top_k that all of a row's ids reach, and with top_p."""
    rng = np.random.default_rng(T + (dtype == "f32"))
    f32 = np.float32
    for k, p in [(0, 1.0), (V - 1, 1.0), (0, 0.999)]:
        z = wide_rows(rng, T, V, dtype)
        if k:
            z[:, ::97] = -np.inf  # fewer ids than top_k
        inv_t = rng.choice([0.05, 0.1, 0.2], T).astype(f32)
        m = rng.choice([1e-3, 1e-4, 5.5e-4, 1e-5], T).astype(f32)
        check(z, dtype, inv_t, np.full(T, k, np.int32), np.full(T, p, f32), m, rng.random(T).astype(f32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(5, 9001), (48, 9001), (200, 8200)])
def test_edges_about_zero_and_at_the_end(T, V, dtype):
    """min_p's edge on, just above and just below a value that thousands of ids
    have, among them the last value with a bin of its own and those about zero."""
    rng = np.random.default_rng(7 * T + (dtype == "f32"))
    f32 = np.float32
    for value in [-63.75, -64.0, -64.5, -80.0, 0.0, -2.0 ** -11, 2.0 ** -14]:
        top = 10.0
        z = LR.round_to(rng.choice([value, value + 6.0, value - 6.0, -90.0, 9.0], (T, V)), dtype)
        z[:, 17] = top
        inv_t = np.full(T, 0.09375, f32)
        edge = np.exp((value - top) * 0.09375)
        m = (edge * rng.choice([1 - 2.0 ** -20, 1 + 2.0 ** -20], T)).astype(f32)
        check(z, dtype, inv_t, np.zeros(T, np.int32), np.ones(T, f32), m, rng.random(T).astype(f32))
