"""The table's gradient for more tokens than one chunk per thread block of the sort
and than 64 chunks: whole numbers, whose FP32 sums are exact in any order."""
import pytest

import nvfp4_w4a4_moe_top_gb300 as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


# one, two and three passes of the sort; 2, 4, 32 tokens per thread; 65 and 129 chunks
@pytest.mark.parametrize("T,V,d", [(32769, 300, 64), (40000, 50001, 72), (100003, 300000, 24), (1048577, 300000, 8),
                                   (1048577, 500, 16), (2100001, 40009, 8)])
def test_many_tokens(T, V, d):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + V)
    r = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda")  # noqa: E731
    often = ((torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * (V + 1.0)) ** 2 / (V + 1.0)).long()
    for ids in [often.clamp(max=V - 1), r(-3, V + 2, T), torch.full((T,), V - 1, device="cuda")]:
        dy = r(-2, 3, T, d).to(torch.bfloat16)
        start = r(-9, 10, V, d).float()
        ok = (ids >= 0) & (ids < V)
        want = torch.zeros((V, d), dtype=torch.float64, device="cuda").index_add_(0, ids[ok], dy[ok].double())
        ws = torch.empty(M.embed_tokens_backward_workspace_bytes(T, V, d), dtype=torch.uint8, device="cuda").fill_(0xAB)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for accumulate in [False, True]:
            dtable = start.clone()
            M.moe_embed_tokens_backward(dy, ids.int(), 2.0, dtable, ws, accumulate, status)
            assert torch.equal(dtable.double(), 2 * want + (start.double() if accumulate else 0))
        assert int(status.item()) == (M.STATUS_BAD_TOKEN if bool((ids >= V).any()) else 0)
