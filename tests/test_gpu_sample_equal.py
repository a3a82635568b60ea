"""Rows of equal logits whose number of ids is a power of two: their weights add up
to the largest sum that a row can have.  Sums are exact and every border is met
exactly; tolerances of the log-probabilities as in test_gpu_sample.py."""
import numpy as np
import pytest

import learner_ref as LR
from test_gpu_sample import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(6, 2048), (40, 2048), (320, 2048), (6, 131072), (40, 131072), (3, 1 << 20), (37, 1 << 20)])
def test_largest_sums(T, V, dtype):
    u = np.resize(np.array([0, 0.5, 1 - 2.0 ** -24, 2.0 ** -24, 0.25, 0.75], np.float32), T)
    for value in [0.0, -7.5] if V < 1 << 20 else [7.5]:
        z = LR.round_to(np.full((T, V), value), dtype)
        for k, p, m in [(None, None, None), (3, None, None), (V // 2, None, None), (None, 0.5, None), (None, None, 1.0)]:
            f = lambda v: None if v is None else np.full(T, v)  # noqa: E731
            check(z, dtype, None, f(k), f(p), f(m), u)
