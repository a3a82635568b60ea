"""The draw for more rows than a cluster of blocks each, and rows that its first
launch leaves open: few of them, many, and all; against the definition in 64 bits
and against the same rows in other company.  Tolerances as in test_gpu_sample.py."""
import numpy as np
import pytest

import learner_ref as LR
import nvfp4_w4a4_moe_top_gb300 as M
import tokens_ref as R
from test_gpu_sample import FILTERS, check, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def mixed_rows(rng, T, V, dtype, flat):
    """Peaked rows, a part of them flat: their weight lies in thousands of ids."""
    z = LR.logit_rows(rng, T, V, dtype)
    wide = np.nonzero(rng.random(T) < flat)[0]
    wide = wide[wide > 5]
    z[wide] = LR.round_to(rng.standard_normal((len(wide), V)) * rng.choice([0.3, 1.0, 2.0], (len(wide), 1)), dtype)
    return z


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,flat", [(20, 3000, 0.5), (45, 9001, 0.1), (60, 12000, 1.0), (310, 8192, 0.05),
                                      (330, 6000, 0.9)])
def test_many_rows(T, V, flat, dtype):
    rng = np.random.default_rng(T + V + (dtype == "f32"))
    for i, kind in enumerate(FILTERS):
        if T > 100 and i % 3 != (dtype == "f32"):
            continue
        check(mixed_rows(rng, T, V, dtype, flat), dtype, *R.filters(rng, T, kind), pad=[0, 3][i % 2], lead=[0, 1, 5][i % 3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_rows_than_blocks(dtype):
    """Blocks take rows in turn, the short rows of a small vocabulary."""
    rng = np.random.default_rng(4)
    T, V = 10007, 211
    z = LR.logit_rows(rng, T, V, dtype)
    for kind in ["", "kpm"]:
        check(z, dtype, *R.filters(rng, T, kind), pad=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["", "p", "kpm"])
def test_company(kind, dtype):
    """The same rows alone, in tens and in hundreds: the same tokens, and the same
    bits from call to call."""
    rng = np.random.default_rng(5)
    T, V = 340, 20011
    z = mixed_rows(rng, T, V, dtype, 0.6)
    args = R.filters(rng, T, kind)
    tokens, lp, kept = draw(z, dtype, *args)
    again = draw(z, dtype, *args)
    assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip((tokens, lp, kept), again))
    for n in [1, 19, 20, 64, 300]:
        part = draw(z[:n], dtype, *(a[:n] for a in args))
        assert np.array_equal(part[0], tokens[:n])


def test_extremes_in_many_rows():
    """Temperatures that leave FP32's range of exponents, rows below zero, rows of
    zeros of both signs, tiny numbers, rows at the lowest value."""
    rng = np.random.default_rng(6)
    T, V = 48, 5003
    for dtype in ["bf16", "f32"]:
        z = rng.standard_normal((T, V)) * 2
        z[0:8] = -np.abs(z[0:8]) - 1e-3
        z[8:12] = np.where(rng.random((4, V)) < 0.5, 0.0, -0.0)
        z[12:16] *= 1e-30
        z[16:20] = -np.abs(z[16:20]) * 1e-6
        z[20:24] *= 1e4
        z[24:26] = -1e30
        z = LR.round_to(z, dtype)
        z[26:28] = LR.LOWEST[dtype]
        z[26, rng.random(V) < 0.5] = -np.inf
        z[28:30, 10:] = LR.LOWEST[dtype]
        for inv_t, k, p, m in [(1.0, 0, 1.0, 0.0), (1.0, 700, 1.0, 0.0), (1.0, 0, 0.6, 0.0), (1e6, 0, 1.0, 0.0),
                               (1e-6, 0, 0.3, 0.0), (1e6, 900, 0.5, 0.5), (0.01, 0, 1.0, 0.97), (3.0, 3000, 0.9, 1e-3)]:
            u = rng.random(T).astype(np.float32)
            check(z, dtype, np.full(T, inv_t, np.float32), np.full(T, k), np.full(T, p, np.float32),
                  np.full(T, m, np.float32), u)


def test_outputs_left_out():
    """Without log-probabilities the tokens are the same."""
    import torch
    rng = np.random.default_rng(7)
    for T in [5, 50]:
        V = 9000
        z = LR.device_rows(mixed_rows(rng, T, V, "bf16", 0.5), "bf16")
        u = torch.rand(T, device="cuda")
        p = torch.full((T,), 0.9, device="cuda")
        a, b = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
        M.moe_sample_tokens(z, u, a, top_p=p)
        M.moe_sample_tokens(z, u, b, top_p=p, logprob=torch.empty(T, device="cuda"),
                            kept_logprob=torch.empty(T, device="cuda"))
        assert torch.equal(a, b)


def test_bad_rows_among_many():
    """NaN, infinities and bad numbers leave the other rows as they are."""
    import torch
    rng = np.random.default_rng(8)
    T, V = 40, 4000
    z = mixed_rows(rng, T, V, "f32", 0.5)
    args = R.filters(rng, T, "pm")
    good = draw(z, "f32", *args)
    z[7, 5], z[20, 0], z[33] = np.nan, np.inf, -np.inf
    u = args[4].copy()
    u[11] = np.nan
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = draw(z, "f32", *args[:4], u, status=status)
    bad = [7, 20, 33, 11]
    assert (got[0][bad] == -1).all() and int(status.item()) == M.STATUS_NONFINITE_LOGITS | M.STATUS_BAD_SAMPLING
    assert np.isnan(got[1][[7, 20, 11]]).all() and np.isneginf(got[1][33])
    rest = np.setdiff1d(np.arange(T), bad)
    for a, b in zip(good, got):
        assert np.array_equal(a[rest], b[rest])
