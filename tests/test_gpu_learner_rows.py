"""Many rows: groups of threads and blocks that take several rows in turn, by
plans that small tests do not reach.

A period of P rows is repeated over all T rows (P a multiple of 8, so that
equal rows lie alike within 16 bytes for any stride): the first P are compared
with the definitions in 64 bits, with the tolerances of test_gpu_logprobs.py
and test_gpu_distill.py, and every other row has to have the bits of the equal
row among them, whatever came before it in its group.  The sizes give each
group of a launch (152 SMs) two rows or more; the row that a group had before
is never the same one."""
import numpy as np
import pytest

import learner_ref as R
import nvfp4_w4a4_moe_top_gb300 as M
from test_gpu_distill import teacher, teacher_lse, tolerances
from test_gpu_logprobs import near

pytestmark = pytest.mark.gpu
P = 56


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def many(a, T):
    """[P][..] repeated over T rows, on the device."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.repeat((-(-T // P),) + (1,) * (t.dim() - 1))[:T].contiguous()


def many_rows(z, dtype, T, pad, lead):
    """The same for logits, V + pad elements apart, `lead` elements into their
    storage; the gaps hold NaN."""
    import torch
    V, n = z.shape[1], -(-T // P) * P
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    flat = torch.full((n * (V + pad) + lead,), float("nan"), dtype=dt, device="cuda")
    rows = flat[lead:].view(n, V + pad)
    rows.view(n // P, P, V + pad)[:, :, :V] = torch.from_numpy(z).to(dt).cuda()
    return rows[:T, :V]


def same_rows(x, what):
    """Every row of x has the bits of the one P rows before it."""
    import torch
    x = x if x.dim() > 1 else x[:, None]
    size = torch.int16 if x.element_size() == 2 else torch.int32
    for t0 in range(0, len(x) - P, 4096):
        t1 = min(t0 + 4096, len(x) - P)
        a, b = x[t0:t1], x[t0 + P:t1 + P]
        bits = [v.contiguous().view(size) for v in (a, b)]
        if not torch.equal(*bits):
            rows = (bits[0] != bits[1]).any(1).nonzero()[:5, 0] + t0 + P
            raise AssertionError("%s: rows %s differ from those before" % (what, rows.tolist()))


def logits(rng, V, dtype, nan):
    z = R.logit_rows(rng, P, V, dtype)
    if nan:
        z[7, rng.integers(V)] = np.nan
        z[30, V - 1] = np.inf
    return z


BAD = [7, 30]


@pytest.mark.parametrize("T,V,dtype,n_top,pad,nan", [
    (40000, 300, "bf16", 0, 0, True), (40000, 301, "bf16", 20, 0, True), (40000, 70, "f32", 5, 3, False),
    (30000, 24001, "bf16", 20, 1, False),                  # a warp per row, runs of two groups
    (8192, 32768, "bf16", 0, 0, True), (8192, 32771, "bf16", 20, 0, True), (8000, 16384, "f32", 32, 8, False),
    (8000, 70001, "bf16", 3, 2, False),                    # 128 threads, runs of two groups
    (3700, 131101, "bf16", 20, 0, True), (3700, 66000, "f32", 7, 1, False),  # 256 threads
    (8200, 131072, "bf16", 0, 0, False)])
def test_logprobs(T, V, dtype, n_top, pad, nan):
    import torch
    rng = np.random.default_rng(T + V)
    z = logits(rng, V, dtype, nan)
    y = rng.integers(-1, V, P).astype(np.int32)
    f = lambda *s: torch.full(s, 777.0, device="cuda")  # noqa: E731
    o = dict(logprob=f(T), entropy=f(T), stats=f(T, 2),
             top_ids=torch.full((T, n_top), 777, dtype=torch.int32, device="cuda"), top_logprob=f(T, n_top))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_token_logprobs(many_rows(z, dtype, T, pad, 1 if pad else 0), many(y, T), 1 / 0.7, n_top, o["logprob"],
                         o["entropy"], o["stats"], o["top_ids"] if n_top else None, o["top_logprob"] if n_top else None, st)
    assert int(st.item()) == (M.STATUS_NONFINITE_LOGITS if nan else 0)
    for k, v in o.items():
        if v.numel():
            same_rows(v, k)
    got = {k: v[:P].cpu().numpy() for k, v in o.items()}
    if nan:
        for k in ["entropy", "stats", "top_logprob"]:
            assert np.isnan(got[k][BAD]).all(), k
        assert (got["top_ids"][BAD] == -1).all()
    keep = np.setdiff1d(np.arange(P), BAD) if nan else np.arange(P)
    ref = R.logprobs(z[keep], y[keep], 1 / 0.7, n_top)
    got = {k: v[keep] for k, v in got.items()}
    near(got["logprob"], ref["logprob"], 4e-6 + 3e-7 * np.abs(ref["logprob"]))
    near(got["entropy"], ref["entropy"], 8e-6 * (1 + ref["entropy"]))
    near(got["stats"][:, 0], ref["stats"][:, 0], 0.0)
    near(got["stats"][:, 1], ref["stats"][:, 1], 4e-6)
    assert np.array_equal(got["top_ids"], ref["top_ids"])
    near(got["top_logprob"], ref["top_logprob"], 4e-6 + 3e-7 * np.abs(ref["top_logprob"]))


@pytest.mark.parametrize("T,V,dtype,pad", [
    (2000, 4000, "bf16", 0), (2000, 2001, "f32", 3),       # a warp per row
    (600000, 33, "bf16", 0),                               # and more than 65535 blocks of them
    (66000, 4104, "bf16", 0), (66000, 2051, "f32", 1),     # a block per row, more than 65535
    (65600, 16401, "bf16", 0)])                            # two blocks per row
def test_logprobs_backward(T, V, dtype, pad):
    import torch
    rng = np.random.default_rng(T + V)
    z = logits(rng, V, dtype, False)
    y = rng.integers(-1, V, P).astype(np.int32)
    g, ge = rng.standard_normal(P).astype(np.float32), (0.3 * rng.standard_normal(P)).astype(np.float32)
    g[9] = ge[9] = 0
    zd, yd = many_rows(z, dtype, T, pad, 1 if pad else 0), many(y, T)
    st, ent = torch.empty((T, 2), device="cuda"), torch.empty(T, device="cuda")
    M.moe_token_logprobs(zd, None, 0.9, 0, None, ent, st)
    dl = many_rows(np.zeros((P, V), np.float32), dtype, T, pad, 1 if pad else 0)
    M.moe_token_logprobs_backward(zd, yd, 0.9, st, ent, many(g, T), many(ge, T), dl)
    same_rows(dl, "dlogits")
    assert torch.isfinite(dl[:P].float()).all()
    ref = R.logprobs_grad(z, y, 0.9, g.astype(float), ge.astype(float))
    r = R.logprobs(z, y, 0.9, 0)
    p, H = np.exp(r["lp"]), r["entropy"][:, None]
    with np.errstate(invalid="ignore"):
        lpH = np.where(p > 0, np.abs(r["lp"]) + H, 0)
        rel = 6e-6 + 4e-7 * np.where(p > 0, -r["lp"], 0)
    A, B = np.abs(np.where(y >= 0, g, 0))[:, None], np.abs(ge)[:, None]
    tol = 0.9 * (rel * p * (A + B * lpH) + B * p * 2e-5 * (1 + H) + 2e-7 * A) + 1e-37
    near(dl[:P].float().cpu().numpy(), ref, tol + (2.0 ** -7.99 * np.abs(ref) if dtype == "bf16" else 0))
    if pad:
        assert torch.isnan(dl.as_strided((T - 1, pad), (V + pad, 1), dl.storage_offset() + V)).all()
    first = dl[:P].clone()
    M.moe_token_logprobs_backward(zd, yd, 0.9, st, ent, many(g, T), many(ge, T), zd)  # in place
    same_rows(zd, "dlogits in place")
    assert torch.equal(zd[:P], first)


def distill_case(T, V, K, dtype, pad, tail, nan, ops):
    import torch
    rng = np.random.default_rng(T + V + K)
    z = logits(rng, V, dtype, nan)
    ids, a = teacher(rng, np.where(np.isnan(z), 0, z), K, tail)
    # a repeat and ids out of range, among rows without
    if K > 3:
        ids[11, :2] = ids[11, 2] = V // 3
        ids[12, 1] = V
        ids[12, 3] = 1 << 30
    lse = teacher_lse(rng, a, np.where(R.keep_entries(ids, V), ids, -1), 0.8) if tail else None
    g = rng.uniform(0.5, 2, P).astype(np.float32)
    g[13] = 0
    lead = 1 if pad else 0
    zd = many_rows(z, dtype, T, pad, lead)
    args = (many(ids, T), many(a, T), None if lse is None else many(lse, T), 0.8)
    gd, st = many(g, T), torch.zeros(1, dtype=torch.int32, device="cuda")
    empty = lambda: many_rows(np.full((P, V), 55.0, np.float32), dtype, T, pad, lead)  # noqa: E731
    status = (M.STATUS_BAD_TOKEN if K > 3 else 0) | (M.STATUS_NONFINITE_LOGITS if nan else 0)
    keep = np.setdiff1d(np.arange(P), BAD) if nan else np.arange(P)
    zk = z[keep]
    ik, ak, lk, gk = ids[keep], a[keep], None if lse is None else lse[keep], g[keep]
    loss, grad, stats = R.distill(zk, ik, ak, lk, 0.8)
    grad = grad * gk.astype(float)[:, None]
    tl, tg = tolerances(zk, ik, ak, lk, 0.8, gk)
    if dtype == "bf16":
        tg = tg + 2.0 ** -7.99 * np.abs(grad)
    huge = ~(np.abs(loss) < 1e30)

    def check_loss(x):
        same_rows(x, "loss")
        got = x[:P].cpu().numpy()
        assert np.isnan(got[BAD]).all() or not nan
        got = got[keep]
        near(np.where(huge, 0, got), np.where(huge, 0, loss), tl + 2e-7 * np.abs(np.where(huge, 0, loss)))
        assert (got[huge] > 1e30).all()

    def check_grad(x, what):
        same_rows(x, what)
        got = x[:P].float().cpu().numpy()
        assert np.isnan(got[BAD]).all() or not nan
        assert (got[13] == 0).all()
        near(got[keep], grad, tg)
    l1, s1 = torch.full((T,), 7.0, device="cuda"), torch.full((T, 4), 7.0, device="cuda")
    M.moe_distill_topk(zd, *args, l1, s1, st)
    assert int(st.item()) == status
    check_loss(l1)
    same_rows(s1, "stats")
    s = s1[:P].cpu().numpy()[keep]
    near(s[:, [0, 2]], stats[:, [0, 2]], 0.0)
    near(s[:, [1, 3]], stats[:, [1, 3]], 4e-6)
    if "gradient" in ops:
        d = empty()
        M.moe_distill_topk_backward(zd, *args, s1, gd, d, st)
        check_grad(d, "gradient")
        del d
    if "step" in ops:
        d, l2 = empty(), torch.full((T,), 7.0, device="cuda")
        M.moe_distill_topk_train(zd, *args, gd, l2, d, st)
        check_loss(l2)
        check_grad(d, "gradient of the step")
        first, lost = d[:P].clone(), l2.clone()
        M.moe_distill_topk_train(zd, *args, gd, l2, zd, st)  # in place
        same_rows(zd, "gradient in place")
        assert torch.equal(zd[:P].nan_to_num(9), first.nan_to_num(9)) and torch.equal(l2.nan_to_num(9), lost.nan_to_num(9))


@pytest.mark.parametrize("T,V,K,dtype,pad,tail,nan", [
    (20000, 1000, 40, "bf16", 0, True, True), (20000, 61, 3, "bf16", 3, False, False),
    (20000, 501, 64, "f32", 0, False, True), (20000, 6000, 16, "bf16", 1, True, False),   # a warp per row
    (6000, 20001, 33, "bf16", 0, True, True), (6000, 10002, 200, "f32", 2, False, False),  # 128 threads
    (2600, 40000, 64, "bf16", 8, False, False), (2600, 70001, 5, "bf16", 0, True, True),   # 256
    (2000, 131072, 64, "bf16", 0, True, False),              # the gradient alone in two parts per row
    (1300, 100003, 50, "bf16", 1, False, False), (1300, 50001, 256, "f32", 0, True, False),  # 512
    (700, 140001, 16, "bf16", 0, True, True), (700, 70007, 33, "f32", 5, False, False)])     # 1024 in the step
def test_distill(T, V, K, dtype, pad, tail, nan):
    distill_case(T, V, K, dtype, pad, tail, nan, ["gradient", "step"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [400003, 700001, M.DISTILL_MAX_V])
@pytest.mark.parametrize("T", [3, 40])
def test_distill_of_long_rows(T, V, dtype):
    """Up to the longest row: one bit per id takes 49, 85 and 128 KB beside the
    ring.  Rows by themselves against the definitions (no repeats here)."""
    import torch
    rng = np.random.default_rng(V + T)
    n, K = 3, 100
    z = R.logit_rows(rng, 6, V, dtype)[[0, 4, 5]]
    ids, a = teacher(rng, z, K, True)
    lse = teacher_lse(rng, a, ids, 1.0)
    g = rng.uniform(0.5, 2, n).astype(np.float32)
    at = np.arange(T) % n
    zd = torch.empty((T, V + 3), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")[:, :V]
    zd.copy_(torch.from_numpy(z).cuda()[at])
    d = lambda x: torch.from_numpy(x[at]).cuda()  # noqa: E731
    args = (d(ids), d(a), d(lse), 1.0)
    loss, stats, l2 = torch.empty(T, device="cuda"), torch.empty((T, 4), device="cuda"), torch.empty(T, device="cuda")
    g1, g2, st = torch.empty_like(zd), torch.empty_like(zd), torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_distill_topk(zd, *args, loss, stats, st)
    M.moe_distill_topk_backward(zd, *args, stats, d(g), g1, st)
    M.moe_distill_topk_train(zd, *args, d(g), l2, g2, st)
    assert int(st.item()) == 0
    rl, rg, rs = R.distill(z, ids, a, lse, 1.0)
    rg = rg * g.astype(float)[:, None]
    tl, tg = tolerances(z, ids, a, lse, 1.0, g)
    if dtype == "bf16":
        tg = tg + 2.0 ** -7.99 * np.abs(rg)
    huge = ~(np.abs(rl) < 1e30)
    for t in sorted({0, 1, 2, T - 2, T - 1}):
        i = at[t]
        for x in [loss, l2]:
            if huge[i]:
                assert x[t].item() > 1e30
            else:
                near(x[t:t + 1].cpu().numpy(), rl[i:i + 1], tl[i] + 2e-7 * abs(rl[i]))
        s = stats[t].cpu().numpy()
        near(s[[0, 2]], rs[i, [0, 2]], 0.0)
        near(s[[1, 3]], rs[i, [1, 3]], 4e-6)
        for x in [g1, g2]:
            near(x[t].float().cpu().numpy(), rg[i], tg[i])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_of_a_very_long_row(dtype):
    """2^26 logits and a few: runs of many groups, ties (BF16 has few values)
    that no list of candidates holds.  Tolerances: a thread of the 2048 adds at
    most 2^26 / 2048 / 16 batches one by one, 2048 roundings of its sums, and
    some 20 more within a batch and between threads: 2100 * 2^-24 of a sum."""
    far = 2100 * 2.0 ** -24
    import torch
    T, V, n = 2, (1 << 26) + 3, 20
    gen = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn((T, V), generator=gen, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    y = torch.tensor([5, V - 1], dtype=torch.int32, device="cuda")
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    lp, ent, st, tl = f(T), f(T), f(T, 2), f(T, n)
    ti = torch.empty((T, n), dtype=torch.int32, device="cuda")
    M.moe_token_logprobs(z, y, 1.0, n, lp, ent, st, ti, tl)
    for t in range(T):
        x = z[t].double()
        ref = torch.log_softmax(x, 0)
        H = -(ref.exp() * ref).sum().item()
        best, order = torch.sort(z[t].float(), descending=True, stable=True)
        assert torch.equal(ti[t].long(), order[:n])
        near(tl[t].cpu().numpy(), ref[order[:n]].cpu().numpy(), far + 4e-6 + 3e-7 * ref[order[:n]].abs().cpu().numpy())
        near(lp[t:t + 1].cpu().numpy(), [ref[y[t].long()].item()], far + 4e-6 + 3e-7 * abs(ref[y[t].long()].item()))
        near(ent[t:t + 1].cpu().numpy(), [H], (2 * far + 8e-6) * (1 + H))
        assert st[t, 0].item() == x.max().item()
        near(st[t, 1:].cpu().numpy(), [(torch.logsumexp(x, 0) - x.max()).item()], far + 4e-6)
