"""moe_token_logprobs and its gradient against the definitions in 64 bits.

Tolerances.  FP32 with the maximum taken out: exponents d = (x - m) inv_t of
weights that count (d > -20) are formed with two roundings, so a weight is off
by at most 20 * 2^-23 + 2^-22 (the exponential) < 3e-6 relative, mostly
cancelling; a sum of non-negative terms in blocks adds below 1e-6.  Hence
ln-sum within 4e-6, a log-probability within that plus its own rounding, 4e-6
+ 3e-7 |lp|, the entropy (l plus a weighted mean of d) within 8e-6 (1 + H).  A
gradient is a probability (relative error: the log-probability's) times
factors that hold the entropy's error.  BF16 output adds half a unit of its
8-bit significand, 2^-8."""
import numpy as np
import pytest

import learner_ref as R
import nvfp4_w4a4_moe_top_gb300 as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def forward(zd, targets, inv_t, n_top):
    import torch
    T = zd.shape[0]
    f = lambda *s: torch.full(s, 777.0, device="cuda")  # noqa: E731
    o = dict(logprob=f(T), entropy=f(T), stats=f(T, 2), top_ids=torch.full((T, n_top), 777, dtype=torch.int32,
                                                                        device="cuda"), top_logprob=f(T, n_top),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    M.moe_token_logprobs(zd, targets, inv_t, n_top, o["logprob"], o["entropy"], o["stats"],
                         o["top_ids"] if n_top else None, o["top_logprob"] if n_top else None, o["status"])
    return o


def host(o):
    return {k: v.cpu().numpy() for k, v in o.items()}


def near(got, ref, tol):
    """Equal within tol; what FP32 cannot hold is infinite in both."""
    with np.errstate(over="ignore"):
        got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float32).astype(np.float64)
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin], equal_nan=True)
    assert np.isfinite(got[fin]).all()
    off = np.abs(got[fin] - ref[fin]) - np.broadcast_to(tol, ref.shape)[fin]
    assert off.size == 0 or off.max() <= 0, (off.max(), np.argmax(off))


SHAPES = [(1, 1), (6, 1), (7, 2), (6, 5), (9, 8), (6, 31), (40, 257), (7, 1000), (6, 4096), (11, 12345), (6, 50001),
          (1, 131072), (3, 131071), (300, 2048), (1, 262147), (4000, 65), (600, 17000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", SHAPES)
def test_forward(T, V, dtype):
    import torch
    rng = np.random.default_rng(T * 1000003 + V)
    for inv_t, n_top, pad, lead, ties in [(1.0, 0, 0, 0, False), (1.0, 20, 0, 0, False), (1 / 0.7, 5, 3, 1, True),
                                          (0.5, 32, 8, 0, True), (1.0, 1, 5, 3, False)]:
        z = R.logit_rows(rng, T, V, dtype, ties)
        y = rng.integers(-1, V, T).astype(np.int32)
        zd = R.device_rows(z, dtype, pad, lead)
        got = host(forward(zd, torch.from_numpy(y).cuda(), inv_t, n_top))
        ref = R.logprobs(z, y, inv_t, n_top)
        assert got["status"][0] == 0
        near(got["logprob"], ref["logprob"], 4e-6 + 3e-7 * np.abs(ref["logprob"]))
        near(got["entropy"], ref["entropy"], 8e-6 * (1 + ref["entropy"]))
        near(got["stats"][:, 0], ref["stats"][:, 0], 0.0)
        near(got["stats"][:, 1], ref["stats"][:, 1], 4e-6)
        assert np.array_equal(got["top_ids"], ref["top_ids"])
        near(got["top_logprob"], ref["top_logprob"], 4e-6 + 3e-7 * np.abs(ref["top_logprob"]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ties_take_the_lower_ids(dtype):
    import torch
    V = 40000
    z = np.zeros((4, V), np.float32)
    z[1, 1::2] = -0.0                                    # equal to +0
    z[2, -7:] = 1.0                                      # the best ids at the end of the row
    z[3, :] = np.repeat(np.arange(V // 8), 8)[::-1] % 5  # runs of ties everywhere
    got = host(forward(R.device_rows(z, dtype), torch.zeros(4, dtype=torch.int32, device="cuda"), 1.0, 32))
    assert np.array_equal(got["top_ids"], R.logprobs(z, np.zeros(4, int), 1.0, 32)["top_ids"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alternatives_all_in_one_place(dtype):
    """The alternatives adjacent, and a period apart that puts them on one
    thread or one block for many block shapes."""
    import torch
    V = 70000
    for step in [1, 8, 512, 4096, 2048]:
        z = np.random.default_rng(step).standard_normal((2, V)).astype(np.float32)
        z = R.round_to(z, dtype)
        z[0, 17:17 + 16 * step:step] = R.round_to(np.linspace(20, 30, 16), dtype)
        z[1, V - 1 - 15 * step::step] = R.round_to(np.linspace(30, 20, 16), dtype)
        y = np.zeros(2, np.int32)
        got = host(forward(R.device_rows(z, dtype), torch.from_numpy(y).cuda(), 1.0, 32))
        assert np.array_equal(got["top_ids"], R.logprobs(z, y, 1.0, 32)["top_ids"]), step


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,n_top", [(1, 131072, 20), (3, 70001, 32), (320, 40000, 20), (320, 9000, 8), (40, 6007, 32),
                                       (33, 700, 20)])
def test_masks_leave_fewer_ids_than_alternatives(T, V, n_top, dtype):
    """Rows that a mask leaves 0, 1, 2, .. ids, the others -inf or the type's
    lowest value."""
    import torch
    rng = np.random.default_rng(V + n_top)
    for mask in [-np.inf, R.LOWEST[dtype]]:
        full = R.round_to(rng.standard_normal((T, V)).astype(np.float32), dtype)
        z = np.full((T, V), mask, np.float32)
        y = np.full(T, -1, np.int32)
        for t in range(T):
            left = rng.choice(V, t % (n_top + 2), replace=False)
            z[t, left] = full[t, left]
            if len(left):
                y[t] = left[0]
        got = host(forward(R.device_rows(z, dtype, 1, 1), torch.from_numpy(y).cuda(), 1.0, n_top))
        ref = R.logprobs(z, y, 1.0, n_top)
        assert got["status"][0] == 0
        near(got["logprob"], ref["logprob"], 4e-6 + 3e-7 * np.abs(ref["logprob"]))
        near(got["entropy"], ref["entropy"], 8e-6 * (1 + ref["entropy"]))
        assert np.array_equal(got["top_ids"], ref["top_ids"])
        near(got["top_logprob"], ref["top_logprob"], 4e-6 + 3e-7 * np.abs(ref["top_logprob"]))


def test_nonfinite_rows_and_bad_targets():
    import torch
    for dtype in ["bf16", "f32"]:
        z = np.random.default_rng(3).standard_normal((5, 3001)).astype(np.float32)
        z[1, 2999] = np.nan
        z[2, 5] = np.inf
        y = torch.tensor([0, 1, 2, 3001, -5], dtype=torch.int32, device="cuda")
        got = host(forward(R.device_rows(z, dtype), y, 1.0, 4))
        assert got["status"][0] == M.STATUS_NONFINITE_LOGITS | M.STATUS_BAD_TOKEN
        for k in ["logprob", "entropy", "stats", "top_logprob"]:
            assert np.isnan(got[k][1:3]).all(), k
            assert np.isfinite(got[k][[0, 3, 4]]).all(), k
        assert (got["top_ids"][1:3] == -1).all()
        assert got["logprob"][3] == 0 and got["logprob"][4] == 0


def test_optional_outputs_and_no_rows():
    import torch
    z = R.device_rows(np.random.default_rng(4).standard_normal((3, 999)).astype(np.float32), "f32")
    y = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    full = host(forward(z, y, 1.0, 3))
    lp, st, en = torch.empty(3, device="cuda"), torch.empty((3, 2), device="cuda"), torch.empty(3, device="cuda")
    M.moe_token_logprobs(z, y, 1.0, 0, lp, None, None)
    M.moe_token_logprobs(z, None, 1.0, 0, None, None, st)
    M.moe_token_logprobs(z, None, 1.0, 0, None, en, None)
    assert np.array_equal(lp.cpu().numpy(), full["logprob"])
    assert np.array_equal(st.cpu().numpy(), full["stats"])
    assert np.array_equal(en.cpu().numpy(), full["entropy"])
    M.moe_token_logprobs(z[:0], y[:0], 1.0, 2, lp[:0], None, None, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                         torch.empty((0, 2), device="cuda"))
    with pytest.raises(M.MoeError) as e:
        M.moe_token_logprobs(z, y, 0.0, 0, lp, None, None)
    assert e.value.code == M.MOE_ERR_SHAPE
    with pytest.raises(ValueError):
        M.moe_token_logprobs(z.t(), y, 1.0, 0, lp, None, None)
    with pytest.raises(ValueError):
        M.moe_token_logprobs(z, y.long(), 1.0, 0, lp, None, None)
    with pytest.raises(ValueError):
        M.moe_token_logprobs(z, y[:2], 1.0, 0, lp, None, None)


@pytest.mark.parametrize("T", [1, 2, 5, 37, 400])
def test_repeats_bit_for_bit_and_on_another_stream(T):
    import torch
    rng = np.random.default_rng(T)
    z = R.device_rows(R.logit_rows(rng, T, 30011, "bf16"), "bf16")
    y = torch.from_numpy(rng.integers(0, 30011, T).astype(np.int32)).cuda()
    a = host(forward(z, y, 1.0, 20))
    b = forward(z, y, 1.0, 20)
    again = host(b)
    for v in b.values():
        v.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    M.moe_token_logprobs(z, y, 1.0, 20, b["logprob"], b["entropy"], b["stats"], b["top_ids"], b["top_logprob"],
                         b["status"], s)
    s.synchronize()
    b = host(b)
    for k in a:
        assert np.array_equal(a[k].view(np.int32), again[k].view(np.int32)), k
        assert np.array_equal(a[k].view(np.int32), b[k].view(np.int32)), k


def backward(zd, y, inv_t, f, g, ge, dlogits):
    import torch
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_token_logprobs_backward(zd, y, inv_t, f["stats"], f["entropy"], g, ge, dlogits, st)
    return int(st.item())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (6, 2), (7, 13), (6, 1000), (9, 4099), (6, 50001), (2, 131072), (70, 8192)])
def test_backward(T, V, dtype):
    import torch
    rng = np.random.default_rng(T * 7 + V)
    for inv_t, pad, lead, dpad, dlead, with_ent in [(1.0, 0, 0, 0, 0, True), (1 / 0.6, 3, 1, 3, 1, True),
                                                    (0.5, 3, 0, 6, 2, False), (1.0, 8, 2, 1, 0, True)]:
        z = R.logit_rows(rng, T, V, dtype)
        y = rng.integers(-1, V, T).astype(np.int32)
        g = rng.standard_normal(T).astype(np.float32)
        ge = (rng.standard_normal(T) * (0.3 if with_ent else 0)).astype(np.float32)
        if T > 6:
            g[6] = ge[6] = 0
        zd, yd = R.device_rows(z, dtype, pad, lead), torch.from_numpy(y).cuda()
        f = forward(zd, yd, inv_t, 0)
        dl = R.device_rows(np.full((T, V), 55.0, np.float32), dtype, dpad, dlead, fill=66.0)
        gd, ged = torch.from_numpy(g).cuda(), torch.from_numpy(ge).cuda()
        assert backward(zd, yd, inv_t, f, gd, ged if with_ent else None, dl) == 0
        ref = R.logprobs_grad(z, y, inv_t, g.astype(float), ge.astype(float))
        r = R.logprobs(z, y, inv_t, 0)
        p, H = np.exp(r["lp"]), r["entropy"][:, None]
        with np.errstate(invalid="ignore"):
            lpH = np.where(p > 0, np.abs(r["lp"]) + H, 0)
        A = np.abs(np.where(y >= 0, g, 0))[:, None]
        B = np.abs(ge)[:, None]
        rel = 6e-6 + 4e-7 * np.where(p > 0, -r["lp"], 0)
        tol = inv_t * (rel * p * (A + B * lpH) + B * p * 2e-5 * (1 + H) + 2e-7 * A) + 1e-37
        if dtype == "bf16":
            tol = tol + 2.0 ** -7.99 * np.abs(ref)
        near(dl.float().cpu().numpy(), ref, tol)
        if dpad:  # the gaps between the rows stay
            flat = dl.as_strided((T, V + dpad), (V + dpad, 1), dl.storage_offset())[:-1, V:] if T > 1 else dl[:, :0]
            assert (flat == 66).all()
        if not with_ent:
            continue
        z2 = R.device_rows(z, dtype, pad, lead)  # in place
        assert backward(z2, yd, inv_t, f, gd, ged, z2) == 0
        assert torch.equal(z2.float(), dl.float())


def test_backward_matches_differences():
    """Central differences of sum(g logprob + ge entropy) in 64 bits: their
    error, h^2 / 6 times a third derivative of order one, is below 1e-8 with h
    = 1e-4, their rounding below 1e-11 / h."""
    import torch
    rng = np.random.default_rng(9)
    T, V, inv_t, h = 3, 37, 1.3, 1e-4
    z = R.round_to(rng.standard_normal((T, V)) * 2, "f32")
    y = np.array([4, -1, 36], np.int32)
    g, ge = rng.standard_normal(T).astype(np.float32), rng.standard_normal(T).astype(np.float32)

    def f(zz):
        r = R.logprobs(zz, y, inv_t, 0)
        return g * r["logprob"] + ge * r["entropy"]
    num = np.zeros((T, V))
    for v in range(V):
        d = np.zeros((T, V))
        d[:, v] = h
        num[:, v] = (f(z.astype(float) + d) - f(z.astype(float) - d)) / (2 * h)
    zd, yd = R.device_rows(z, "f32"), torch.from_numpy(y).cuda()
    dl = torch.empty((T, V), device="cuda")
    backward(zd, yd, inv_t, forward(zd, yd, inv_t, 0), torch.from_numpy(g).cuda(), torch.from_numpy(ge).cuda(), dl)
    near(dl.cpu().numpy(), num, 3e-5)


def test_backward_of_nonfinite_and_skipped_rows():
    import torch
    z = np.random.default_rng(5).standard_normal((4, 2050)).astype(np.float32)
    z[1, 7] = np.nan
    z[3, 9] = np.nan  # no gradient there: not read
    zd = R.device_rows(z, "f32")
    y = torch.tensor([3, 4, 2050, -1], dtype=torch.int32, device="cuda")
    f = forward(zd, y, 1.0, 0)
    dl = torch.full((4, 2050), 5.0, device="cuda")
    st = backward(zd, y, 1.0, f, torch.ones(4, device="cuda"), None, dl)
    assert st == M.STATUS_BAD_TOKEN
    d = dl.cpu().numpy()
    assert np.isnan(d[1]).all() and (d[2:] == 0).all() and np.isfinite(d[0]).all() and d[0, 3] > 0
