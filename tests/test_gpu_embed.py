"""Embedding and its gradient against their definitions in 64 bits.

Tolerances.  Forward: the FP32 product is rounded once to BF16, both sides by
the same rule: equal bits.  Gradient: a sum of n BF16 values in FP32, in some
order, is off by at most (n - 1) 2^-24 of the sum of magnitudes in the first
order; with the product by the scale and, accumulating, the final addition n + 1
roundings.  2^-24 (n + 2) of the magnitudes covers the higher orders for n below
2^20."""
import numpy as np
import pytest

import nvfp4_w4a4_moe_top_gb300 as M
import tokens_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def rows(a, dtype, pad, fill=float("nan")):
    """A device tensor of a's rows, `pad` elements apart."""
    import torch
    n, d = a.shape
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    flat = torch.full((n, d + pad), fill, dtype=dt, device="cuda")
    v = flat[:, :d]
    v.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(dt))
    return v


def draw_ids(rng, T, V, kind):
    if kind == "same":
        return np.full(T, V // 2, np.int32)
    if kind == "each":
        return rng.permutation(np.arange(T) % V).astype(np.int32)
    ids = np.minimum(np.exp(rng.random(T) * np.log(V)).astype(np.int64), V) - 1
    if kind == "padded":
        ids[rng.random(T) < 0.3] = -1
    if kind == "out of range":
        ids[rng.random(T) < 0.2] = V
        ids[rng.random(T) < 0.1] = 2 ** 31 - 1
        ids[rng.random(T) < 0.1] = -2 ** 31
    if kind == "none":
        ids[:] = -1
    return ids.astype(np.int32)


KINDS = ["often", "same", "each", "padded", "out of range", "none"]


@pytest.mark.parametrize("T,V,d,pad", [(1, 1, 8, 0), (1, 50, 2048, 0), (7, 1000, 24, 8), (33, 300, 1000, 0),
                                       (500, 129, 264, 16), (1003, 5000, 1024, 0), (5, 40, 16384, 8), (300, 70, 2056, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_embed(T, V, d, pad, dtype):
    import torch
    rng = np.random.default_rng(T * 31 + d)
    table = rows(rng.standard_normal((V, d)).astype(np.float32), dtype, pad)
    back = table.float().cpu().numpy()
    for kind in KINDS:
        ids = draw_ids(rng, T, V, kind)
        for scale in [1.0, d ** 0.5, -0.3]:
            out = rows(np.full((T, d), 3.0, np.float32), "bf16", pad)
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            M.moe_embed_tokens(torch.from_numpy(ids).cuda(), table, scale, out, status)
            want = torch.from_numpy(R.embed(ids, back, scale)).to(torch.bfloat16)
            assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16)), (kind, scale)
            assert int(status.item()) == (M.STATUS_BAD_TOKEN if (ids >= V).any() else 0)
            gap = torch.as_strided(out, (T, d + pad), (d + pad, 1))[:, d:]
            assert torch.isnan(gap).all()  # between the rows nothing is written


@pytest.mark.parametrize("T,V,d,pad", [
    (1, 1, 8, 0), (1, 1000, 64, 0), (2, 3, 16384, 8), (31, 70, 24, 0), (33, 32, 1000, 8), (257, 513, 264, 0),
    (1003, 50, 1024, 0), (2500, 3000, 128, 16), (4099, 20000, 72, 0), (3000, 300000, 8, 0), (20011, 7, 40, 0)])
def test_gradient(T, V, d, pad):
    import torch
    rng = np.random.default_rng(T * 17 + d)
    dy = rows(rng.standard_normal((T, d)).astype(np.float32), "bf16", pad)
    h = dy.float().cpu().numpy()
    n = M.embed_tokens_backward_workspace_bytes(T, V, d)
    for kind in KINDS:
        ids = draw_ids(rng, T, V, kind)
        for accumulate, scale in [(False, 1.0), (True, 1.7), (False, -0.25)]:
            start = rng.standard_normal((V, d)).astype(np.float32)
            dtable = torch.from_numpy(start).cuda() if accumulate else torch.full((V, d), float("nan"), device="cuda")
            ws = torch.full((n + 64,), 0xAB, dtype=torch.uint8, device="cuda")  # of no use before the call
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            M.moe_embed_tokens_backward(dy, torch.from_numpy(ids).cuda(), scale, dtable, ws[:n], accumulate, status)
            got = dtable.cpu().numpy()
            want, mag, count = R.embed_grad(h, ids, V, np.float64(np.float32(scale)), start if accumulate else None)
            off = np.abs(got.astype(np.float64) - want)
            assert (off <= 2.0 ** -24 * (count[:, None] + 2) * mag).all(), (kind, accumulate, scale)
            still = count == 0
            assert np.array_equal(got[still], start[still] if accumulate else np.zeros_like(start[still]))
            assert int(status.item()) == (M.STATUS_BAD_TOKEN if (ids >= V).any() else 0)
            assert (ws[n:] == 0xAB).all()


def test_gradient_by_differences():
    """d/dE of the sum of out * g, with power-of-two steps that BF16 holds: the
    forward is linear, so the difference is the derivative."""
    import torch
    rng = np.random.default_rng(3)
    T, V, d, scale = 40, 12, 16, 2.0
    ids = torch.from_numpy(draw_ids(rng, T, V, "padded")).cuda()
    g = torch.from_numpy(rng.integers(-4, 5, (T, d)).astype(np.float32)).cuda()
    table = torch.from_numpy(rng.integers(-8, 9, (V, d)).astype(np.float32)).cuda()
    dtable = torch.empty((V, d), device="cuda")
    ws = torch.empty(M.embed_tokens_backward_workspace_bytes(T, V, d), dtype=torch.uint8, device="cuda")
    M.moe_embed_tokens_backward(g.to(torch.bfloat16), ids, scale, dtable, ws)

    def total(tab):
        out = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
        M.moe_embed_tokens(ids, tab, scale, out)
        return (out.float() * g).sum().item()
    for v, c in [(0, 0), (3, 7), (11, 15), (5, 1)]:
        up = table.clone()
        up[v, c] += 1.0
        assert total(up) - total(table) == dtable[v, c].item()


@pytest.mark.parametrize("T,V,d", [(700, 900, 256), (9000, 300, 512)])
def test_same_bits_every_time(T, V, d):
    import torch
    rng = np.random.default_rng(T)
    dy = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).cuda().to(torch.bfloat16)
    ids = torch.from_numpy(draw_ids(rng, T, V, "often")).cuda()
    ws = torch.empty(M.embed_tokens_backward_workspace_bytes(T, V, d), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(20):
        out = torch.empty((V, d), device="cuda")
        M.moe_embed_tokens_backward(dy, ids, 1.0, out, ws)
        first = out if first is None else first
        assert torch.equal(out, first)


def test_no_tokens():
    import torch
    table = torch.ones((5, 16), device="cuda")
    none, out = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    M.moe_embed_tokens(none, table, 1.0, out)
    M.moe_embed_tokens_backward(out, none, 1.0, table, None, True)
    assert (table == 1).all()
    M.moe_embed_tokens_backward(out, none, 1.0, table, None)
    assert (table == 0).all()
