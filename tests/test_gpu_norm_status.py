"""moe_add_rmsnorm_backward's status: a dx that is no finite number."""
import numpy as np
import pytest

import nvfp4_w4a4_moe_top_gb300 as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("d", [16, 48, 1024, 2048, 2176, 4096, 8192, 16384])
@pytest.mark.parametrize("T", [3, 700])
def test_nonfinite_rows_are_reported(T, d):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(d)
    b16 = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    clean = dict(dy=b16(T, d), dh=b16(T, d), h=b16(T, d), w=b16(d))
    clean["rstd"] = (clean["h"].float().square().mean(1) + 1e-6).rsqrt()
    ws = torch.empty(M.add_rmsnorm_backward_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")

    def run(v, with_dw, status):
        dx, dw = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda"), torch.zeros(d, device="cuda")
        M.moe_add_rmsnorm_backward(v["dy"], v["dh"], v["h"], v["rstd"], v["w"], dx, dw if with_dw else None, ws, status)
        return dx
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = run(clean, True, st)
    assert int(st.item()) == 0
    rows = np.arange(T)
    for name, row, col, value in [("dy", 0, 0, np.nan), ("dy", T - 1, d - 1, np.inf), ("h", T // 2, d // 2, -np.inf),
                                  ("dh", T - 1, d - 1, np.nan), ("dh", 0, 3, -np.inf), ("rstd", T // 2, None, np.nan)]:
        v = dict(clean)
        v[name] = v[name].clone()
        if col is None:
            v[name][row] = value
        else:
            v[name][row, col] = value
        for with_dw in [True, False]:
            st = torch.full((1,), M.STATUS_TIMEOUT, dtype=torch.int32, device="cuda")  # other bits stay
            dx = run(v, with_dw, st)
            assert int(st.item()) == M.STATUS_TIMEOUT | M.STATUS_NONFINITE_X, (name, row)
            keep = torch.from_numpy(rows != row).cuda()
            assert torch.equal(dx[keep], ref[keep])
            assert not torch.isfinite(dx[row].float()).all()
            assert torch.equal(run(v, with_dw, None)[keep], ref[keep])  # no status word
