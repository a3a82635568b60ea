"""The C ABI of the operators at the token ends without a GPU: every function of
its header is exported, sizes are what the header says, and bad arguments are
refused on the host before any CUDA call."""
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
    names = M.header_functions(M.TOKENS_HEADER)
    assert names == ["moe_embed_tokens", "moe_embed_tokens_backward", "moe_embed_tokens_backward_workspace_bytes",
                     "moe_sample_tokens"]
    for n in names:
        assert hasattr(L, n), n


def test_constants():
    src = open(M.TOKENS_HEADER).read()
    for line in ["MOE_STATUS_BAD_SAMPLING 0x%x" % M.STATUS_BAD_SAMPLING, "MOE_EMBED_MAX_V  (1 << 24)",
                 "MOE_EMBED_MAX_D  %d" % M.EMBED_MAX_D, "MOE_SAMPLE_MAX_V (1 << 20)"]:
        assert "#define " + line in src
    assert (M.EMBED_MAX_V, M.SAMPLE_MAX_V) == (1 << 24, 1 << 20)


def test_workspace_sizes(L):
    f = M.embed_tokens_backward_workspace_bytes
    for T, V, d in [(1, 1, 8), (512, 32768, 1024), (65536, 131072, 2048), (1 << 24, 1 << 24, 8), (3, 1 << 24, 16384)]:
        assert f(T, V, d) >= 8 * T  # the sorted tokens at least
    for T, V, d in [(-1, 8, 8), (4, 0, 8), (4, (1 << 24) + 1, 8), (4, 8, 0), (4, 8, 12), (4, 8, 16392), ((1 << 24) + 1, 8, 8)]:
        assert f(T, V, d) == 0


def call(f, args, **change):
    """f on the dict `args` with some replaced, by name."""
    assert set(change) <= set(args), change
    return f(*{**args, **change}.values())


def refuses(f, args, code, **change):
    assert call(f, args, **change) == code, change


def test_embed_refusals(L):
    a = dict(ids=FAKE, table=FAKE, dtype=0, ldt=256, T=4, V=100, d=256, scale=1.0, out=FAKE, ldo=256, status=None,
             stream=None)
    f = L.moe_embed_tokens
    for c in [dict(dtype=2), dict(dtype=-1), dict(ldt=255), dict(ldt=260), dict(ldt=248), dict(T=-1), dict(V=0),
              dict(V=(1 << 24) + 1), dict(d=0), dict(d=252), dict(d=16392), dict(ldo=248), dict(ldo=257),
              dict(ldt=1 << 46), dict(ldo=1 << 46), dict(scale=NAN), dict(scale=INF)]:
        refuses(f, a, M.MOE_ERR_SHAPE, **c)
    for c in [dict(ids=None), dict(table=None), dict(out=None), dict(ids=at(2)), dict(table=at(8)), dict(out=at(2)),
              dict(status=at(1))]:
        refuses(f, a, M.MOE_ERR_POINTER, **c)


def test_embed_backward_refusals(L):
    a = dict(dy=FAKE, ldy=256, ids=FAKE, T=4, V=100, d=256, scale=1.0, accumulate=0, dtable=FAKE, ws=FAKE,
             ws_bytes=1 << 30, status=None, stream=None)
    f = L.moe_embed_tokens_backward
    for c in [dict(ldy=255), dict(ldy=260), dict(T=-1), dict(T=(1 << 24) + 1), dict(V=0), dict(V=(1 << 24) + 1),
              dict(d=12), dict(d=16392), dict(scale=NAN), dict(scale=-INF), dict(accumulate=2), dict(accumulate=-1),
              dict(ldy=1 << 46)]:
        refuses(f, a, M.MOE_ERR_SHAPE, **c)
    for c in [dict(dy=None), dict(ids=None), dict(dtable=None), dict(ws=None), dict(dy=at(2)), dict(ids=at(2)),
              dict(dtable=at(4)), dict(ws=at(4)), dict(status=at(2)), dict(T=0, dtable=None)]:
        refuses(f, a, M.MOE_ERR_POINTER, **c)
    n = M.embed_tokens_backward_workspace_bytes(4, 100, 256)
    refuses(f, a, M.MOE_ERR_WORKSPACE, ws_bytes=n - 1)
    refuses(f, a, M.MOE_ERR_WORKSPACE, ws_bytes=0)


def test_sample_refusals(L):
    a = dict(logits=FAKE, dtype=0, ld=1000, T=4, V=1000, inv_t=FAKE, top_k=FAKE, top_p=FAKE, min_p=FAKE, u=FAKE,
             tokens=FAKE, logprob=FAKE, kept=FAKE, status=None, stream=None)
    f = L.moe_sample_tokens
    for c in [dict(dtype=2), dict(ld=999), dict(T=-1), dict(V=0), dict(V=(1 << 20) + 1, ld=1 << 21), dict(ld=1 << 45)]:
        refuses(f, a, M.MOE_ERR_SHAPE, **c)
    for c in [dict(logits=None), dict(u=None), dict(tokens=None), dict(logits=at(1)), dict(logits=at(2), dtype=1)] + \
            [{n: at(2)} for n in ["inv_t", "top_k", "top_p", "min_p", "u", "tokens", "logprob", "kept", "status"]]:
        refuses(f, a, M.MOE_ERR_POINTER, **c)
