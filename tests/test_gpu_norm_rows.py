"""The norm and its gradient by the plans of many rows: a warp per row up to d =
2048, and groups of threads that take many rows in turn, each with its part of
dw.  Tolerances of the outputs as in test_gpu_norm.py.

dw: a thread adds its rows one by one, then come the block's groups (8 at most),
the blocks' parts in 32 slices, and the slices in pairs; a term has three
roundings.  Its error is at most the number of additions in a row plus 3, times
2^-24, of the sum of the terms' magnitudes."""
import numpy as np
import pytest

import learner_ref as R
import nvfp4_w4a4_moe_top_gb300 as M
from test_gpu_logprobs import near
from test_gpu_norm import backward, bf, check8, rows, run, unswizzle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("T,d", [(1024, 2048), (1031, 1040), (1100, 1024), (1025, 1920), (1024, 528)])
def test_forward_a_warp_per_row(T, d):
    rng = np.random.default_rng(T + d)
    x, res = rows(rng, T, d), rows(rng, T, d)
    w = R.round_to(1 + 0.3 * rng.standard_normal(d), "bf16")
    for eps, with_res in [(1e-6, True), (1e-5, False)]:
        o = run(bf(x), bf(res) if with_res else None, bf(w), eps, d % 128 == 0)
        h = R.round_to(x + res if with_res else x, "bf16")
        assert np.array_equal(o["h"].float().cpu().numpy(), h)
        assert int(o["status"].item()) == 0
        hd = h.astype(float)
        rstd = 1 / np.sqrt((hd * hd).mean(1) + eps)
        y = hd * rstd[:, None] * w.astype(float)
        near(o["rstd"].cpu().numpy(), rstd, 1e-6 * rstd)
        near(o["y"].float().cpu().numpy(), y, (2.0 ** -7.99 + 4e-6) * np.abs(y) + 1e-40)
        if d % 128 == 0:
            check8(y, o["y8"].cpu().numpy(), unswizzle(o["sf"].cpu().numpy(), T, d))


# rows in one step of the launch: blocks x groups x rows of a group (152 SMs)
STEPS = {128: 152 * 6 * 8 * 2, 1024: 152 * 4 * 2 * 2, 1040: 152 * 2 * 2, 2048: 152 * 2 * 2, 4096: 152 * 2 * 2,
         8192: 152 * 2, 16384: 152}


@pytest.mark.parametrize("T,d", [(40000, 128), (10001, 1024), (3001, 1040), (3000, 2048), (2501, 4096), (1300, 8192),
                                 (700, 16384)])
def test_backward_rows_in_turn(T, d):
    import torch
    rng = np.random.default_rng(T + d)
    h, dy, dh = rows(rng, T, d), R.round_to(rng.standard_normal((T, d)), "bf16"), R.round_to(rng.standard_normal((T, d)), "bf16")
    w = R.round_to(1 + 0.3 * rng.standard_normal(d), "bf16")
    rstd = (1 / np.sqrt((h.astype(float) ** 2).mean(1) + 1e-6)).astype(np.float32)
    args = (bf(dy), bf(dh), bf(h), torch.from_numpy(rstd).cuda(), bf(w))
    dx, dw = backward(*args)
    n = h.astype(float) * rstd.astype(float)[:, None]
    gy, r = dy.astype(float) * w, rstd.astype(float)[:, None]
    ref = r * (gy - n * (gy * n).mean(1, keepdims=True)) + dh
    tol = 4e-6 * (r * (np.abs(gy) + np.abs(n) * np.abs(gy * n).mean(1, keepdims=True)) + np.abs(dh))
    near(dx.float().cpu().numpy(), ref, tol + 2.0 ** -7.99 * np.abs(ref) + 1e-40)
    adds = 2 * -(-T // STEPS[d]) + 8 + 152 * 6 // 32 + 1 + 5
    near(dw.cpu().numpy(), (dy * n).sum(0), (adds + 3) * 2.0 ** -24 * np.abs(dy * n).sum(0) + 1e-40)
    again = args[0].clone()
    dx2, dw2 = backward(again, *args[1:], out=again)  # in place, the same bits
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_dw_of_a_million_rows():
    """2^20 + 300 rows, T d > 2^31: dw against sums in 64 bits by parts."""
    import torch
    T, d = (1 << 20) + 300, 2048
    gen = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn((T, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn((T, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    r = 0.5 + torch.rand(T, generator=gen, device="cuda")
    w, dw = torch.ones(d, dtype=torch.bfloat16, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(M.add_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    ref, size = torch.zeros(d, dtype=torch.float64, device="cuda"), torch.zeros(d, dtype=torch.float64, device="cuda")
    for t in range(0, T, 1 << 15):
        terms = dy[t:t + (1 << 15)].double() * (h[t:t + (1 << 15)].double() * r[t:t + (1 << 15)].double()[:, None])
        ref += terms.sum(0)
        size += terms.abs().sum(0)
    M.moe_add_rmsnorm_backward(dy, None, h, r, w, dy, dw, ws)
    adds = 2 * -(-T // STEPS[d]) + 8 + 152 * 6 // 32 + 1 + 5
    assert ((dw.double() - ref).abs() <= (adds + 3) * 2.0 ** -24 * size).all()
