"""moe_distill_topk, its gradient and the step that gives both, against the
definitions in 64 bits.

Tolerances.  As for the log-probabilities (test_gpu_logprobs.py): a student's
log-probability and the log of its mass off the list within 6e-6 + 3e-7 |lp|;
the teacher's q_i = exp of a number rounded twice, relative error 1e-6 + 1.2e-7
(|a inv_t| + |lse|) =: eq; so r = 1 - sum q within eq absolutely.  The loss adds q and r
weighted terms, each of those errors times at most (1 + |ln q| + |lp|) or (1 +
|ln r| + |ln s|).  The gradient holds p, q, t s and t r, each with its relative
error; BF16 output adds 2^-8 relative."""
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


def teacher(rng, z, K, tail):
    """K ids a row: mostly the student's likely ones, in any order; a fifth of
    the places empty where K > 4; the teacher near the student."""
    T, V = z.shape
    ids = np.full((T, K), -1, np.int32)
    for t in range(T):
        n = min(K, V)
        top = np.argsort(-z[t], kind="stable")[:max(1, n // 2)]
        rest = rng.permutation(V)[:K]
        c = list(dict.fromkeys(list(top) + list(rest)))[:n]
        rng.shuffle(c)
        ids[t, :n] = c
    if K > 4:
        ids[rng.random((T, K)) < 0.2] = -1
    x = np.take_along_axis(z, np.maximum(ids, 0), 1)
    x = np.where(np.isfinite(x) & (np.abs(x) < 1e30), x, 0)
    a = (x + 0.5 * rng.standard_normal((T, K))).astype(np.float32)
    return ids, a


def teacher_lse(rng, a, ids, inv_t):
    w = np.where(ids >= 0, np.exp(a.astype(float) * inv_t), 0).sum(1)
    return np.log(np.where(w > 0, w, 1) / rng.uniform(0.5, 0.98, len(w))).astype(np.float32)


def dev(a):
    import torch
    return None if a is None else torch.from_numpy(a).cuda()


def step(zd, ids, a, lse, inv_t, g, dlogits=None):
    """Forward, backward and the one-call step; the last two must agree."""
    import torch
    T = zd.shape[0]
    o = dict(loss=torch.full((T,), 7.0, device="cuda"), stats=torch.full((T, 4), 7.0, device="cuda"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (dev(ids), dev(a), dev(lse), inv_t)
    M.moe_distill_topk(zd, *args, o["loss"], o["stats"], st)
    new = lambda: torch.full_like(zd, 55.0) if dlogits is None else dlogits.clone()  # noqa: E731
    o["grad"] = new() if dlogits is None else dlogits
    M.moe_distill_topk_backward(zd, *args, o["stats"], dev(g), o["grad"], st)
    loss2, grad2 = torch.full((T,), 7.0, device="cuda"), new()
    M.moe_distill_topk_train(zd, *args, dev(g), loss2, grad2, st)
    o["status"] = int(st.item())
    return o, loss2, grad2


def tolerances(z, ids, a, lse, inv_t, g):
    """(loss, gradient) tolerances of the module's text."""
    T, V = z.shape
    ok = R.keep_entries(ids, V)
    tl, tg = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        k, at = ids[t][ok[t]], a[t][ok[t]].astype(float) * inv_t
        zz = z[t].astype(float) * inv_t
        if np.isneginf(zz).all():
            continue
        lpa = (zz - zz.max()) - np.log(np.exp(zz - zz.max()).sum())
        on = np.zeros(V, bool)
        on[k] = True
        L = float(lse[t]) if lse is not None else (at.max() + np.log(np.exp(at - at.max()).sum()) if len(k) else 0)
        q = np.exp(at - L)
        r = max(0.0, 1 - q.sum()) if lse is not None else 0.0
        eq = 1e-6 + 1.2e-7 * ((np.abs(at).max() if len(k) else 0) + abs(L))
        s = np.exp(lpa[~on]).sum()
        e = 6e-6 + 3e-7 * np.where(np.isfinite(lpa), -lpa, 0)
        fin = np.isfinite(lpa[k])
        tl[t] = (q * (e[k] + eq * (2 + np.abs(at - L) + np.where(fin, -lpa[k], 0))))[q > 0].sum()
        if r > 0 and s > 0:
            tl[t] += r * (6e-6 + 3e-7 * abs(np.log(s))) + eq * (2 + abs(np.log(r)) + abs(np.log(s)))
        p = np.exp(lpa)
        tt = np.where(on, 0, p) / (s if s > 0 else 1)
        tg[t] = 2 * e * p + tt * (2 * e * r + eq + 1e-6)
        tg[t, k] = 2 * e[k] * p[k] + 2 * eq * q + 1e-7
    return tl, tg * inv_t * np.abs(g)[:, None] + 1e-37


def check(z, dtype, ids, a, lse, inv_t, g, pad=0, lead=0, dpad=None, dlead=0):
    zd = R.device_rows(z, dtype, pad, lead)
    T, V = z.shape
    dl = None if dpad is None else R.device_rows(np.full((T, V), 55.0, np.float32), dtype, dpad, dlead, fill=66.0)
    o, loss2, grad2 = step(zd, ids, a, lse, inv_t, g, dl)
    loss, grad, stats = R.distill(z, ids, a, lse, inv_t)
    grad = grad * g.astype(float)[:, None]
    tl, tg = tolerances(z, ids, a, lse, inv_t, g)
    if dtype == "bf16":
        tg = tg + 2.0 ** -7.99 * np.abs(grad)
    huge = ~(np.abs(loss) < 1e30)  # masked at the lowest value: only the size is checked
    got = o["loss"].cpu().numpy()
    near(np.where(huge, 0, got), np.where(huge, 0, loss), tl + 2e-7 * np.abs(np.where(huge, 0, loss)))
    assert (got[huge] > 1e30).all()
    st = o["stats"].cpu().numpy()
    near(st[:, [0, 2]], stats[:, [0, 2]], 0.0)
    near(st[:, [1, 3]], stats[:, [1, 3]], 4e-6)
    near(o["grad"].float().cpu().numpy(), grad, tg)
    near(loss2.cpu().numpy(), o["loss"].cpu().numpy(), 2 * tl + 4e-7 * np.where(huge, 0, np.abs(loss)) + np.where(huge, 1e33, 0))
    near(grad2.float().cpu().numpy(), grad, tg)
    if dpad and T > 1:
        assert (o["grad"].as_strided((T, V + dpad), (V + dpad, 1), o["grad"].storage_offset())[:-1, V:] == 66).all()
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (6, 2, 2), (7, 9, 4), (8, 33, 40), (6, 1000, 16), (9, 4097, 64), (7, 30011, 256),
                                   (2, 131072, 64), (64, 2048, 8), (1, 262145, 33), (200, 8190, 3), (330, 66000, 16)])
def test_loss_and_gradient(T, V, K, dtype):
    rng = np.random.default_rng(T * 31 + V + K)
    for inv_t, tail, pad, lead, dpad, dlead in [(1.0, True, 0, 0, None, 0), (0.5, False, 3, 1, 3, 1),
                                                (1 / 0.7, True, 5, 2, 2, 0)]:
        z = R.logit_rows(rng, T, V, dtype)
        ids, a = teacher(rng, z, K, tail)
        lse = teacher_lse(rng, a, ids, inv_t) if tail else None
        g = rng.uniform(0.5, 2, T).astype(np.float32)
        g[T // 2] = 0 if T > 2 else 1
        o = check(z, dtype, ids, a, lse, inv_t, g, pad, lead, dpad, dlead)
        assert o["status"] == 0


def test_peaked_student_keeps_its_rest():
    """The student's mass off the list down to e^-80: beyond what 1 minus the
    rest could tell."""
    V, K = 3001, 4
    for off in [5.0, 20.0, 40.0, 80.0]:
        z = np.zeros((3, V), np.float32)
        z[:, :K] = off + np.log(V)
        ids = np.tile(np.arange(K, dtype=np.int32), (3, 1))
        a = np.zeros((3, K), np.float32)
        lse = np.log(K / 0.9).astype(np.float32) * np.ones(3, np.float32)
        check(R.round_to(z, "f32"), "f32", ids, a, lse, 1.0, np.ones(3, np.float32))


def test_empty_lists_repeats_and_bad_ids():
    import torch
    rng = np.random.default_rng(2)
    z = R.round_to(rng.standard_normal((4, 500)), "bf16")
    ids = np.array([[-1, -1, -1, -1], [3, 9, 3, 9], [500, 7, -2, 1 << 30], [4, 5, 6, 7]], np.int32)
    a = rng.standard_normal((4, 4)).astype(np.float32)
    for lse in [None, np.full(4, 3.0, np.float32)]:
        o = check(z, "bf16", ids, a, lse, 1.0, np.ones(4, np.float32))
        assert o["status"] == M.STATUS_BAD_TOKEN
        assert o["loss"][0].item() == 0 if lse is None else abs(o["loss"][0].item()) < 1e-5
        assert torch.count_nonzero(o["grad"][0]).item() == 0 or lse is not None


def test_list_of_the_whole_vocabulary():
    rng = np.random.default_rng(3)
    z = R.round_to(rng.standard_normal((3, 200)) * 2, "f32")
    ids = np.stack([rng.permutation(200) for _ in range(3)]).astype(np.int32)
    a = np.take_along_axis(z, ids, 1) + rng.standard_normal((3, 200)).astype(np.float32) * 0.1
    check(z, "f32", ids, a.astype(np.float32), None, 1.0, np.ones(3, np.float32))
    lse = (np.log(np.exp(a.astype(float)).sum(1)) + 0.5).astype(np.float32)  # r > 0 with nothing off the list
    import torch
    o, loss2, _ = step(R.device_rows(z, "f32"), ids, a.astype(np.float32), lse, 1.0, np.ones(3, np.float32))
    assert torch.isinf(o["loss"]).all() and torch.isinf(loss2).all() and (o["loss"] > 0).all()


def test_nonfinite_numbers():
    rng = np.random.default_rng(4)
    z = rng.standard_normal((6, 700)).astype(np.float32)
    ids = np.tile(np.array([1, 2, 3], np.int32), (6, 1))
    a = np.zeros((6, 3), np.float32)
    lse = np.full(6, 2.0, np.float32)
    z[0, 600] = np.nan
    z[1, 2] = np.inf
    a[2, 0] = np.nan
    lse[3] = np.nan
    a[4, 1] = -np.inf  # the teacher excludes it: no term
    for le in [lse, None]:
        o, loss2, grad2 = step(R.device_rows(z, "f32"), ids, a, le, 1.0, np.ones(6, np.float32))
        assert o["status"] == M.STATUS_NONFINITE_LOGITS
        bad = 4 if le is not None else 3
        for x in [o["loss"], loss2]:
            x = x.cpu().numpy()
            assert np.isnan(x[:bad]).all() and np.isfinite(x[bad:]).all()
        for x in [o["grad"], grad2]:
            x = x.cpu().numpy()
            assert np.isnan(x[:2]).all() and np.isfinite(x[bad:]).all()
            assert all(np.isnan(x[i]).any() for i in range(2, bad))


def test_gradient_matches_differences():
    """Central differences of the 64-bit loss with h = 1e-4: error below 1e-8
    (third derivatives of order one) plus 1e-11 / h."""
    rng = np.random.default_rng(6)
    T, V, K, h, inv_t = 3, 40, 5, 1e-4, 0.8
    z = R.round_to(rng.standard_normal((T, V)) * 2, "f32")
    ids, a = teacher(rng, z, K, True)
    for lse in [teacher_lse(rng, a, ids, inv_t), None]:
        num = np.zeros((T, V))
        for v in range(V):
            d = np.zeros((T, V))
            d[:, v] = h
            num[:, v] = (R.distill(z + d, ids, a, lse, inv_t)[0] - R.distill(z - d, ids, a, lse, inv_t)[0]) / (2 * h)
        o, _, grad2 = step(R.device_rows(z, "f32"), ids, a, lse, inv_t, np.ones(T, np.float32))
        near(o["grad"].cpu().numpy(), num, 3e-5)
        near(grad2.cpu().numpy(), num, 3e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 50001), (5, 131072), (300, 4099)])
def test_in_place_repeats_and_streams(T, V, dtype):
    import torch
    rng = np.random.default_rng(V)
    z = R.logit_rows(rng, T, V, dtype)
    ids, a = teacher(rng, z, 20, True)
    lse = teacher_lse(rng, a, ids, 1.0)
    g = rng.uniform(0.5, 2, T).astype(np.float32)
    for lead in [0, 1]:
        zd = R.device_rows(z, dtype, 3, lead)
        o, loss2, grad2 = step(zd, ids, a, lse, 1.0, g)
        args = (dev(ids), dev(a), dev(lse), 1.0)
        z2 = R.device_rows(z, dtype, 3, lead)
        M.moe_distill_topk_backward(z2, *args, o["stats"], dev(g), z2)
        z3, l3 = R.device_rows(z, dtype, 3, lead), torch.zeros(T, device="cuda")
        gd = dev(g)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        M.moe_distill_topk_train(z3, *args, gd, l3, z3, None, s)
        s.synchronize()
        bits = torch.int16 if dtype == "bf16" else torch.int32
        assert torch.equal(z2.contiguous().view(bits), o["grad"].contiguous().view(bits))
        assert torch.equal(z3.contiguous().view(bits), grad2.contiguous().view(bits))
        assert torch.equal(l3.view(torch.int32), loss2.view(torch.int32))
