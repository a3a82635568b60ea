"""moe_add_rmsnorm and its gradient against the definitions in 64 bits.

Tolerances.  h is one rounding of an exact sum: equal bit for bit.  The mean of
squares sums at most 64 non-negative terms a thread and then halves: 1e-6 is
the bound asked of rstd.  y adds two products, 2e-6 relative, and BF16's 2^-8.  An E4M3 code may differ from
the 64-bit quotient's only by one step, where that quotient lies within 3e-6
of the midpoint; a scale byte only where the block's largest value lies within
3e-6 of a power of two times 448.  dx: products and a mean of d terms, 4e-6 of
the magnitudes entering, and BF16's 2^-8; dw: a sum of T terms, (T + 16) 2^-24
of the sum of magnitudes."""
import numpy as np
import pytest

import learner_ref as R
import nvfp4_w4a4_moe_top_gb300 as M
from test_gpu_logprobs import near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def rows(rng, T, d):
    x = rng.standard_normal((T, d))
    x[:, rng.integers(d, size=max(1, d // 200))] *= 30
    if T > 3:
        x[1] *= 1e-4
        x[2] = 0
        x[3, : d // 2] = 0
        if T > 5:
            x[4] *= 1e15
            x[5] *= 1e-18  # far below eps
    return R.round_to(x, "bf16")


def bf(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()


def unswizzle(sf, T, d):
    r, c = np.arange(T)[:, None], np.arange(d // 32)[None, :]
    return sf[((r // 128) * (d // 128) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4]


def run(x, res, w, eps, with8):
    import torch
    T, d = x.shape
    o = dict(h=torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda"),
             y=torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda"),
             rstd=torch.full((T,), 7.0, device="cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if with8:
        o["y8"] = torch.full((T, d), 0x77, dtype=torch.uint8, device="cuda")
        o["sf"] = torch.full((M.mx8_sf_bytes(T, d),), 0xA5, dtype=torch.uint8, device="cuda")
    M.moe_add_rmsnorm(x, res, w, eps, o["h"], o["y"], o.get("y8"), o.get("sf"), o["rstd"], o["status"])
    return o


def check8(y, codes, sb):
    """The 8-bit output of the 64-bit y: scale bytes and codes, but for values
    within 3e-6 of a boundary."""
    import torch
    T, d = y.shape
    amax = np.abs(y).reshape(T, d // 32, 32).max(2)

    def scale_of(a):
        f, e = np.frexp(a)
        return np.where(a == 0, 0, np.maximum(np.where(f > 0.875, e - 8, e - 9) + 127, 0))
    lo, hi = scale_of(amax * (1 - 3e-6)), scale_of(amax * (1 + 3e-6))
    assert ((sb == lo) | (sb == hi)).all()
    S = np.ldexp(1.0, sb.astype(int) - 127).repeat(32, 1)
    v = y / S
    got = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).float().numpy().astype(float)
    # half a step of E4M3 at the value's size: 3 mantissa bits, subnormals below 2^-6
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -20))), -6) - 3)
    assert (np.abs(got - v) <= step / 2 + 3e-6 * np.abs(v)).all()
    assert np.abs(got).max() <= 448


@pytest.mark.parametrize("T,d", [(1, 16), (7, 48), (6, 128), (4, 2048), (130, 1024), (129, 2176), (33, 4096), (9, 6144 - 128),
                                 (6, 16384), (1, 8192), (2000, 256), (5, 8208)])
def test_forward(T, d):
    import torch
    rng = np.random.default_rng(T * 17 + d)
    x, res = rows(rng, T, d), rows(rng, T, d)
    w = R.round_to(1 + 0.3 * rng.standard_normal(d), "bf16")
    for eps, with_res in [(1e-6, True), (1e-5, False)]:
        with8 = d % 128 == 0
        o = run(bf(x), bf(res) if with_res else None, bf(w), eps, with8)
        h = R.round_to(x + res if with_res else x, "bf16")
        assert np.array_equal(o["h"].float().cpu().numpy(), h)
        assert int(o["status"].item()) == 0
        hd = h.astype(float)
        rstd = 1 / np.sqrt((hd * hd).mean(1) + eps)
        y = hd * rstd[:, None] * w.astype(float)
        near(o["rstd"].cpu().numpy(), rstd, 1e-6 * rstd)
        near(o["y"].float().cpu().numpy(), y, (2.0 ** -7.99 + 4e-6) * np.abs(y) + 1e-40)
        if with8:
            check8(y, o["y8"].cpu().numpy(), unswizzle(o["sf"].cpu().numpy(), T, d))


def test_strides_in_place_and_left_out_outputs():
    import torch
    rng = np.random.default_rng(5)
    T, d = 37, 1024
    x, res = rows(rng, T, d), rows(rng, T, d)
    w = bf(R.round_to(1 + 0.3 * rng.standard_normal(d), "bf16"))
    a = run(bf(x), bf(res), w, 1e-6, True)
    wide = lambda v, n: torch.full((T, n), float("nan"), dtype=torch.bfloat16, device="cuda")[:, 8:8 + d].copy_(bf(v))  # noqa: E731
    b = run(wide(x, d + 24), wide(res, d + 8), w, 1e-6, True)
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
    r2, x2 = bf(res), bf(x)
    y = torch.empty_like(r2)
    M.moe_add_rmsnorm(x2, r2, w, 1e-6, r2, y)                     # h over res
    assert torch.equal(r2, a["h"]) and torch.equal(y, a["y"])
    M.moe_add_rmsnorm(x2, bf(res), w, 1e-6, x2, None)             # h over x, no other output
    assert torch.equal(x2, a["h"])
    y8, sf = torch.empty((T, d), dtype=torch.uint8, device="cuda"), torch.full_like(a["sf"], 0xA5)
    M.moe_add_rmsnorm(a["h"], None, w, 1e-6, None, None, y8, sf)  # no residual, 8 bits alone
    assert torch.equal(y8, a["y8"]) and torch.equal(sf, a["sf"])
    used = unswizzle(np.arange(sf.numel()), T, d).reshape(-1)     # bytes of rows past T stay
    rest = np.setdiff1d(np.arange(sf.numel()), used)
    assert (sf.cpu().numpy()[rest] == 0xA5).all()
    M.moe_add_rmsnorm(x2[:0], None, w, 1e-6, None, y[:0])
    with pytest.raises(ValueError):
        M.moe_add_rmsnorm(x2, None, w[:8], 1e-6, None, y)
    with pytest.raises(ValueError):
        M.moe_add_rmsnorm(x2, None, w, 1e-6, None, y, y8, sf[:16])
    with pytest.raises(ValueError):
        M.moe_add_rmsnorm(x2.float(), None, w, 1e-6, None, y)
    with pytest.raises(M.MoeError) as e:
        M.moe_add_rmsnorm(x2, bf(res), w, 1e-6, None, y)
    assert e.value.code == M.MOE_ERR_POINTER


def test_extreme_values_keep_their_scales():
    """Blocks from subnormal to near the largest BF16, and exact powers of two
    and 448 times them, with w = 1 and a norm of one."""
    import torch
    d = 2048
    x = np.zeros((2, d), np.float32)
    x[0, ::32] = np.ldexp(1.0, -np.arange(d // 32) * 2)
    x[0, 1::32] = 0.875 * np.ldexp(1.0, -np.arange(d // 32) * 2)
    x[1, :] = R.round_to(3e38 * np.ones(d) / 64, "bf16")
    x[1, 5] = 1.0
    x = R.round_to(x, "bf16")
    w = np.ones(d, np.float32)
    o = run(bf(x), None, bf(w), 1e-6, True)
    y = o["y"].float().cpu().numpy()
    hd = x.astype(float)
    rstd = 1 / np.sqrt((hd * hd).mean(1) + 1e-6)
    check8(hd[:1] * rstd[:1, None], o["y8"].cpu().numpy()[:1], unswizzle(o["sf"].cpu().numpy(), 2, d)[:1])
    assert np.isfinite(y[0]).all()
    o = run(bf(np.full((1, d), np.inf, np.float32)), None, bf(w), 1e-6, True)
    assert int(o["status"].item()) == M.STATUS_NONFINITE_X


def backward(dy, dh, h, rstd, w, with_dw=True, out=None):
    import torch
    T, d = dy.shape
    dx = torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    dw = torch.full((d,), 7.0, device="cuda") if with_dw else None
    ws = torch.full((M.add_rmsnorm_backward_workspace_bytes(T, d),), 0xFF, dtype=torch.uint8, device="cuda")
    M.moe_add_rmsnorm_backward(dy, dh, h, rstd, w, dx, dw, ws if with_dw else None)
    return dx, dw


@pytest.mark.parametrize("T,d", [(1, 16), (7, 48), (5, 2048), (1003, 1024), (700, 4096), (130, 2176), (17, 16384), (3000, 128),
                                 (40, 8208), (9, 8192)])
def test_backward(T, d):
    import torch
    rng = np.random.default_rng(T + d)
    h, dy, dh = rows(rng, T, d), R.round_to(rng.standard_normal((T, d)), "bf16"), R.round_to(rng.standard_normal((T, d)), "bf16")
    w = R.round_to(1 + 0.3 * rng.standard_normal(d), "bf16")
    rstd = (1 / np.sqrt((h.astype(float) ** 2).mean(1) + 1e-6)).astype(np.float32)
    for with_dh in [True, False]:
        args = (bf(dy), bf(dh) if with_dh else None, bf(h), torch.from_numpy(rstd).cuda(), bf(w))
        dx, dw = backward(*args)
        n = h.astype(float) * rstd.astype(float)[:, None]
        gy = dy.astype(float) * w
        c = (gy * n).mean(1, keepdims=True)
        r = rstd.astype(float)[:, None]
        ref = r * (gy - n * c) + (dh if with_dh else 0)
        tol = 4e-6 * (r * (np.abs(gy) + np.abs(n) * np.abs(gy * n).mean(1, keepdims=True)) + np.abs(dh) * with_dh)
        near(dx.float().cpu().numpy(), ref, tol + 2.0 ** -7.99 * np.abs(ref) + 1e-40)
        near(dw.cpu().numpy(), (dy * n).sum(0), (T + 16) * 2.0 ** -24 * np.abs(dy * n).sum(0) + 1e-40)
        dx2, dw2 = backward(*args)  # the same bits again, and without dw
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
        assert torch.equal(backward(*args, with_dw=False)[0], dx)
        again = args[0].clone()
        assert torch.equal(backward(again, *args[1:], out=again)[0], dx)  # dx over dy
        if with_dh:
            again = args[1].clone()
            assert torch.equal(backward(args[0], again, *args[2:], out=again)[0], dx)


def test_backward_of_no_rows_and_small_workspace():
    import torch
    z = torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda")
    w, dw = torch.ones(128, dtype=torch.bfloat16, device="cuda"), torch.full((128,), 3.0, device="cuda")
    M.moe_add_rmsnorm_backward(z, None, z, torch.zeros(0, device="cuda"), w, z, dw,
                               torch.zeros(1024, dtype=torch.uint8, device="cuda"))
    assert (dw == 0).all()
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(M.MoeError) as e:
        M.moe_add_rmsnorm_backward(x, None, x, torch.zeros(4, device="cuda"), w, x, dw,
                                   torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == M.MOE_ERR_WORKSPACE


def test_backward_matches_differences():
    """Central differences of sum(dy y + dh h) in 64 bits, y without its
    rounding; BF16 output 2^-8 relative, differences below 1e-7."""
    import torch
    rng = np.random.default_rng(8)
    T, d, e = 2, 32, 1e-5
    h = R.round_to(rng.standard_normal((T, d)), "bf16").astype(float)
    dy, dh = R.round_to(rng.standard_normal((T, d)), "bf16"), R.round_to(rng.standard_normal((T, d)), "bf16")
    w = R.round_to(1 + 0.3 * rng.standard_normal(d), "bf16").astype(float)

    def f(hh, ww):
        return ((hh / np.sqrt((hh * hh).mean(1, keepdims=True) + 1e-6) * ww) * dy + hh * dh).sum(1)
    ndx, ndw = np.zeros((T, d)), np.zeros(d)
    for i in range(d):
        u = np.zeros(d)
        u[i] = e
        ndx[:, i] = (f(h + u, w) - f(h - u, w)) / (2 * e)
        ndw[i] = (f(h, w + u) - f(h, w - u)).sum() / (2 * e)
    rstd = (1 / np.sqrt((h * h).mean(1) + 1e-6)).astype(np.float32)
    dx, dw = backward(bf(dy), bf(dh), bf(h.astype(np.float32)), torch.from_numpy(rstd).cuda(), bf(w.astype(np.float32)))
    near(dx.float().cpu().numpy(), ndx, 2.0 ** -7.99 * np.abs(ndx) + 1e-5)
    near(dw.cpu().numpy(), ndw, 1e-5)
