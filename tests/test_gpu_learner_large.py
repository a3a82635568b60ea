"""Offsets beyond 32 bits: rows more than 2^31 elements apart, and more than
2^31 elements of contiguous rows.  The same rows close together give the same
bits."""
import numpy as np
import pytest

import learner_ref as R
import nvfp4_w4a4_moe_top_gb300 as M

pytestmark = pytest.mark.gpu
FAR = (1 << 31) + 24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def far_rows(z, ld):
    """z [2][n] as rows ld elements apart (the storage between is not set)."""
    import torch
    v = torch.empty(ld + z.shape[1], dtype=z.dtype, device="cuda").as_strided(z.shape, (ld, 1))
    v.copy_(z)
    return v


def test_far_rows_of_logits():
    import torch
    T, V, K, n = 2, 20011, 24, 8
    rng = np.random.default_rng(0)
    near = R.device_rows(R.logit_rows(rng, T, V, "bf16"), "bf16")
    far = far_rows(near, FAR)
    y = torch.tensor([7, V - 1], dtype=torch.int32, device="cuda")
    ids = torch.from_numpy(np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32)).cuda()
    a, g = torch.randn(T, K, device="cuda"), torch.ones(T, device="cuda")

    def run(z, out):
        f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
        lp, en, st, tl, loss, ds = f(T), f(T), f(T, 2), f(T, n), f(T), f(T, 4)
        ti = torch.zeros((T, n), dtype=torch.int32, device="cuda")
        M.moe_token_logprobs(z, y, 1.0, n, lp, en, st, ti, tl)
        M.moe_token_logprobs_backward(z, y, 1.0, st, en, g, g, out)
        r = [lp, en, st, ti, tl, out.clone()]
        M.moe_distill_topk(z, ids, a, None, 1.0, loss, ds)
        M.moe_distill_topk_backward(z, ids, a, None, 1.0, ds, g, out)
        r += [loss.clone(), ds, out.clone()]
        M.moe_distill_topk_train(z, ids, a, None, 1.0, g, loss, out)
        return r + [loss, out.clone()]
    a1 = run(near, torch.zeros_like(near))
    a2 = run(far, far_rows(torch.zeros_like(near), FAR + 5))
    for i, (p, q) in enumerate(zip(a1, a2)):
        assert torch.equal(p, q), i


def test_far_and_many_rows_of_the_norm():
    import torch
    d = 2048
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((2, d), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    h, y, h2, y2 = (torch.empty_like(x) for _ in range(4))
    M.moe_add_rmsnorm(x, x, w, 1e-6, h, y)
    far = far_rows(x, FAR)
    M.moe_add_rmsnorm(far, far, w, 1e-6, h2, y2)
    assert torch.equal(h, h2) and torch.equal(y, y2)
    del far
    T = (1 << 20) + 300  # T d > 2^31
    block = torch.randn((1 << 12, d), generator=g, device="cuda").to(torch.bfloat16)
    big = block.repeat((T + len(block) - 1) // len(block), 1)[:T]
    hb, yb, r = torch.empty_like(big), torch.empty_like(big), torch.empty(T, device="cuda")
    y8 = torch.empty((T, d), dtype=torch.uint8, device="cuda")
    sf = torch.zeros(M.mx8_sf_bytes(T, d), dtype=torch.uint8, device="cuda")
    M.moe_add_rmsnorm(big, None, w, 1e-6, hb, yb, y8, sf, r)
    tail = 300 % (1 << 12)  # the last rows repeat the block's first
    assert torch.equal(yb[-tail:], yb[:tail]) and torch.equal(y8[-tail:], y8[:tail]) and torch.equal(r[-tail:], r[:tail])
    assert torch.equal(hb, big)
    dx, dw = hb, torch.empty(d, device="cuda")
    ws = torch.empty(M.add_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    M.moe_add_rmsnorm_backward(yb, None, big, r, w, dx, dw, ws)
    assert torch.equal(dx[-tail:], dx[:tail])
    n = big[:tail].double() * r[:tail].double()[:, None]
    dy = yb[:tail].double()
    ref = r[:tail].double()[:, None] * (dy - n * (dy * n).mean(1, keepdim=True))
    assert ((dx[:tail].double() - ref).abs() <= 2.0 ** -7.99 * ref.abs() + 8e-6 * (dy.abs() + n.abs())).all()
