"""The learner operators captured in one CUDA graph and replayed on new inputs
in the captured buffers: every replay equals the calls made outside it, bit for
bit."""
import pytest

import nvfp4_w4a4_moe_top_gb300 as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("T,d,V,K,n", [(3, 256, 70001, 16, 5), (700, 1024, 9000, 33, 20)])
def test_replays(T, d, V, K, n):
    import torch
    b16, i32 = torch.bfloat16, torch.int32
    e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    x, res, dy, w = e(T, d, t=b16), e(T, d, t=b16), e(T, d, t=b16), torch.ones(d, dtype=b16, device="cuda")
    z, y, ids, a, g = e(T, V, t=b16), e(T, t=i32), e(T, K, t=i32), e(T, K), torch.ones(T, device="cuda")

    def draw(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for v in (x, res, dy, z):
            v.copy_(torch.randn(v.shape, generator=gen, device="cuda"))
        y.copy_(torch.randint(-1, V, (T,), generator=gen, device="cuda"))
        a.copy_(torch.randn(a.shape, generator=gen, device="cuda"))
        ids.copy_((torch.randint(0, V, (T, 1), generator=gen, device="cuda") + 7 * torch.arange(K, device="cuda")) % V)

    def outputs():
        return dict(h=e(T, d, t=b16), y=e(T, d, t=b16), y8=e(T, d, t=torch.uint8),
                    sf=torch.zeros(M.mx8_sf_bytes(T, d), dtype=torch.uint8, device="cuda"), rstd=e(T), dx=e(T, d, t=b16),
                    dw=e(d), ws=e(M.add_rmsnorm_backward_workspace_bytes(T, d), t=torch.uint8), lp=e(T), ent=e(T),
                    st=e(T, 2), ti=e(T, n, t=i32), tl=e(T, n), dz=e(T, V, t=b16), loss=e(T), ds=e(T, 4),
                    dq=e(T, V, t=b16), loss2=e(T), dr=e(T, V, t=b16))

    def calls(o):
        M.moe_add_rmsnorm(x, res, w, 1e-6, o["h"], o["y"], o["y8"], o["sf"], o["rstd"])
        M.moe_add_rmsnorm_backward(dy, None, o["h"], o["rstd"], w, o["dx"], o["dw"], o["ws"])
        M.moe_token_logprobs(z, y, 1.0, n, o["lp"], o["ent"], o["st"], o["ti"], o["tl"])
        M.moe_token_logprobs_backward(z, y, 1.0, o["st"], o["ent"], g, g, o["dz"])
        M.moe_distill_topk(z, ids, a, None, 1.0, o["loss"], o["ds"])
        M.moe_distill_topk_backward(z, ids, a, None, 1.0, o["ds"], g, o["dq"])
        M.moe_distill_topk_train(z, ids, a, None, 1.0, g, o["loss2"], o["dr"])

    draw(0)
    captured, plain = outputs(), outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls(captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls(captured)
    for seed in [1, 2]:
        draw(seed)
        graph.replay()
        calls(plain)
        torch.cuda.synchronize()
        for k in captured:
            if k != "ws":
                assert torch.equal(captured[k].view(torch.uint8), plain[k].view(torch.uint8)), (seed, k)
