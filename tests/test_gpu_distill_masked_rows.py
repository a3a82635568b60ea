"""Rows of the distillation that a batch masks: weight 0, whatever their
numbers hold."""
import numpy as np
import pytest

import learner_ref as R
import nvfp4_w4a4_moe_top_gb300 as M
from test_gpu_distill import dev, step, teacher, teacher_lse

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 3001, 131072])
def test_weight_zero_gives_zeros_whatever_the_row_holds(V, dtype):
    """Rows with NaN or +inf among the logits (on the list and off it, in and
    outside the 16-byte vectors) or in the teacher's numbers and g = 0 get
    zeros; the rows between them the bits that they get beside clean rows."""
    import torch
    rng = np.random.default_rng(V)
    T, K = 16, 6
    z = R.round_to(rng.standard_normal((T, V)) * 2, dtype)
    ids, a = teacher(rng, z, K, True)
    ids[:, 0], a[:, 0] = V // 2, 0.5  # an entry in every row
    ids[:, 1:][ids[:, 1:] == V // 2] = -1
    lse = teacher_lse(rng, a, ids, 1.0)
    g = np.where(np.arange(T) % 2 == 0, 0.0, 1.5).astype(np.float32)
    bad = z.copy(), a.copy(), lse.copy()
    off = next(v for v in range(1, V) if v not in ids[0])
    bad[0][0, off] = np.nan
    bad[0][2, V // 2] = np.nan
    bad[0][4, 0] = np.inf
    bad[0][6, V - 1] = np.nan
    bad[1][8, 0] = np.nan
    bad[1][10, 0] = np.inf
    bad[2][12] = np.nan
    bad[0][14] = -np.inf
    for with_lse in [True, False]:
        for lead in [0, 1]:
            clean = step(R.device_rows(z, dtype, 3, lead), ids, a, lse if with_lse else None, 1.0, g)
            got = step(R.device_rows(bad[0], dtype, 3, lead), ids, bad[1], bad[2] if with_lse else None, 1.0, g)
            for x, y in [(got[0]["grad"], clean[0]["grad"]), (got[2], clean[2])]:
                assert torch.count_nonzero(x[::2]).item() == 0  # counts NaN
                assert torch.equal(x[1::2], y[1::2]) and torch.count_nonzero(x[1::2]).item() > 0
            assert torch.equal(got[1][1::2], clean[1][1::2])  # the losses, which g does not weigh
            inplace = R.device_rows(bad[0], dtype, 3, lead)
            M.moe_distill_topk_train(inplace, dev(ids), dev(bad[1]), dev(bad[2]) if with_lse else None, 1.0, dev(g),
                                     torch.empty(T, device="cuda"), inplace)
            assert torch.equal(inplace, got[2])
