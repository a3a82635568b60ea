"""The learner operators' C ABI without a GPU: every function of its header is
exported, sizes are what the header says, and bad arguments are refused on the
host before any CUDA call."""
import ctypes

import pytest

import nvfp4_w4a4_moe_top_gb300 as M

FAKE = ctypes.c_void_p(1 << 20)        # aligned, never dereferenced
NAN, INF = float("nan"), float("inf")


def at(off):
    return ctypes.c_void_p((1 << 20) + off)


@pytest.fixture(scope="module")
def L():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()
    return M.lib()


def test_exports_every_header_function(L):
    names = M.header_functions(M.LEARNER_HEADER)
    assert names == ["moe_add_rmsnorm", "moe_add_rmsnorm_backward", "moe_add_rmsnorm_backward_workspace_bytes",
                     "moe_distill_topk", "moe_distill_topk_backward", "moe_distill_topk_train", "moe_mx8_sf_bytes",
                     "moe_token_logprobs", "moe_token_logprobs_backward"]
    for n in names:
        assert hasattr(L, n), n


def test_sizes(L):
    assert M.mx8_sf_bytes(128, 128) == 512
    assert M.mx8_sf_bytes(129, 2048) == 2 * 16 * 512
    assert M.mx8_sf_bytes(0, 128) == 0 and M.mx8_sf_bytes(4, 96) == 0 and M.mx8_sf_bytes(-1, 128) == 0
    assert M.add_rmsnorm_backward_workspace_bytes(1, 2048) >= 2048 * 4
    assert M.add_rmsnorm_backward_workspace_bytes(8, 100) == 0
    assert M.add_rmsnorm_backward_workspace_bytes(-1, 128) == 0


def call(f, args, **change):
    """f on the dict `args` with some replaced, by name."""
    assert set(change) <= set(args), change
    return f(*{**args, **change}.values())


def refuses(f, args, code, **change):
    assert call(f, args, **change) == code, change


def test_add_rmsnorm_refusals(L):
    a = dict(x=FAKE, ldx=256, res=FAKE, ldr=256, w=FAKE, eps=1e-6, T=4, d=256, h=FAKE, y=FAKE, y8=FAKE, sf=FAKE,
             rstd=FAKE, status=None, stream=None)
    f = L.moe_add_rmsnorm
    for c in [dict(d=0), dict(d=250), dict(d=16400), dict(ldx=255), dict(ldx=260), dict(ldr=128), dict(T=-1),
              dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(d=144), dict(ldx=1 << 50), dict(ldr=1 << 46)]:
        refuses(f, a, M.MOE_ERR_SHAPE, **c)
    for c in [dict(x=None), dict(w=None), dict(x=at(2)), dict(res=at(8)), dict(h=at(2)), dict(y=at(2)), dict(y8=at(4)),
              dict(sf=at(4)), dict(rstd=at(2)), dict(y8=None), dict(sf=None), dict(h=None), dict(status=at(1))]:
        refuses(f, a, M.MOE_ERR_POINTER, **c)


def test_add_rmsnorm_backward_refusals(L):
    a = dict(dy=FAKE, dh=FAKE, h=FAKE, rstd=FAKE, w=FAKE, T=4, d=256, dx=FAKE, dw=FAKE, ws=FAKE, ws_bytes=1 << 30,
             status=None, stream=None)
    f = L.moe_add_rmsnorm_backward
    for c in [dict(T=-1), dict(d=8), dict(d=20000), dict(d=1000)]:
        refuses(f, a, M.MOE_ERR_SHAPE, **c)
    for c in [dict(dy=None), dict(h=None), dict(rstd=None), dict(w=None), dict(dx=None), dict(ws=None), dict(dy=at(2)),
              dict(dh=at(2)), dict(dw=at(2)), dict(ws=at(4))]:
        refuses(f, a, M.MOE_ERR_POINTER, **c)
    refuses(f, a, M.MOE_ERR_WORKSPACE, ws_bytes=16)


LOGITS = dict(logits=FAKE, dtype=0, ld=1000, T=4, V=1000)
BAD_LOGITS = [dict(dtype=2), dict(dtype=-1), dict(ld=999), dict(V=0), dict(T=-1), dict(ld=1 << 45),
              dict(V=(1 << 30) + 1, ld=1 << 31), dict(inv_t=0.0),
              dict(inv_t=-1.0), dict(inv_t=NAN), dict(inv_t=INF), dict(inv_t=1e7)]


def test_token_logprobs_refusals(L):
    a = dict(LOGITS, targets=FAKE, inv_t=1.0, n_top=5, logprob=FAKE, entropy=FAKE, stats=FAKE, top_ids=FAKE,
             top_logprob=FAKE, status=None, stream=None)
    f = L.moe_token_logprobs
    for c in BAD_LOGITS + [dict(n_top=-1), dict(n_top=33)]:
        refuses(f, a, M.MOE_ERR_SHAPE, **c)
    for c in [dict(logits=None), dict(logits=at(1)), dict(logits=at(2), dtype=1), dict(targets=None),
              dict(top_ids=None), dict(top_logprob=None), dict(stats=at(2)), dict(targets=at(2))]:
        refuses(f, a, M.MOE_ERR_POINTER, **c)


def test_token_logprobs_backward_refusals(L):
    a = dict(LOGITS, targets=FAKE, inv_t=1.0, stats=FAKE, entropy=FAKE, g=FAKE, ge=FAKE, dlogits=at(1 << 24), ldd=1000,
             status=None, stream=None)
    f = L.moe_token_logprobs_backward
    for c in BAD_LOGITS + [dict(ldd=900), dict(dlogits=FAKE, ldd=1001), dict(ldd=1 << 45)]:
        refuses(f, a, M.MOE_ERR_SHAPE, **c)
    for c in [dict(logits=None), dict(dlogits=None), dict(dlogits=at(1)), dict(stats=None), dict(targets=None),
              dict(entropy=None), dict(g=None, ge=None), dict(g=at(2))]:
        refuses(f, a, M.MOE_ERR_POINTER, **c)


def test_distill_refusals(L):
    head = dict(LOGITS, ids=FAKE, teacher=FAKE, lse=None, K=8, inv_t=1.0)
    fwd = dict(head, loss=FAKE, stats=FAKE, status=None, stream=None)
    bwd = dict(head, stats=FAKE, g=FAKE, dlogits=at(1 << 24), ldd=1000, status=None, stream=None)
    train = dict(head, g=FAKE, loss=FAKE, dlogits=at(1 << 24), ldd=1000, status=None, stream=None)
    for f, a in [(L.moe_distill_topk, fwd), (L.moe_distill_topk_backward, bwd), (L.moe_distill_topk_train, train)]:
        for c in BAD_LOGITS + [dict(K=0), dict(K=257), dict(V=(1 << 20) + 1, ld=1 << 21)]:
            refuses(f, a, M.MOE_ERR_SHAPE, **c)
        for c in [dict(logits=None), dict(logits=at(1)), dict(ids=None), dict(teacher=None), dict(ids=at(2)),
                  dict(lse=at(2)), dict(status=at(2))]:
            refuses(f, a, M.MOE_ERR_POINTER, **c)
        if "dlogits" in a:
            refuses(f, a, M.MOE_ERR_SHAPE, ldd=999)
            refuses(f, a, M.MOE_ERR_SHAPE, dlogits=FAKE, ldd=1001)
            refuses(f, a, M.MOE_ERR_POINTER, dlogits=None)
            refuses(f, a, M.MOE_ERR_POINTER, g=None)
        if "loss" in a:
            refuses(f, a, M.MOE_ERR_POINTER, loss=None)
        if "stats" in a:
            refuses(f, a, M.MOE_ERR_POINTER, stats=at(8))
    refuses(L.moe_distill_topk_backward, bwd, M.MOE_ERR_POINTER, stats=None)


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 64), dtype=torch.bfloat16)  # on the CPU
    with pytest.raises(ValueError):
        M.moe_token_logprobs(x, None, 1.0, 0, None, None, torch.zeros(4, 2))
    with pytest.raises(ValueError):
        M.moe_add_rmsnorm(x, None, x[0], 1e-6, None, x)
    with pytest.raises(ValueError):
        M.moe_distill_topk(x, torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 2), None, 1.0, torch.zeros(4), None)
