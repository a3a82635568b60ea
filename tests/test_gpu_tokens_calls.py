"""The operators at the token ends as a program calls them: captured in a CUDA
graph and replayed on new inputs, on several streams and from several threads at
the same time, in a row without a wait between them, and on tensors whose offsets
pass 32 bits."""
import threading

import numpy as np
import pytest

import learner_ref as LR
import nvfp4_w4a4_moe_top_gb300 as M
import tokens_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


class Case:
    """Inputs and outputs of one size, and the calls on them."""

    def __init__(self, T, V, d, dtype):
        import torch
        self.T, self.V = T, V
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.z = e(T, V, t=torch.bfloat16 if dtype == "bf16" else torch.float32)
        self.u, self.p, self.k = e(T), e(T), e(T, t=torch.int32)
        self.ids, self.table, self.dy = e(T, t=torch.int32), e(V, d, t=torch.bfloat16), e(T, d, t=torch.bfloat16)

    def draw(self, seed):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda t: t.copy_(torch.randn(t.shape, generator=g, device="cuda"))  # noqa: E731
        for t in (self.z, self.table, self.dy):
            r(t)
        self.z[::3] *= 4
        self.u.copy_(torch.rand(self.T, generator=g, device="cuda"))
        self.p.copy_(0.5 + 0.5 * torch.rand(self.T, generator=g, device="cuda"))
        self.k.copy_(torch.randint(0, 60, (self.T,), generator=g, device="cuda"))
        self.ids.copy_(torch.randint(-1, self.V, (self.T,), generator=g, device="cuda") // 7)
        return self

    def outputs(self):
        import torch
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        V, d = self.table.shape
        return dict(tokens=e(self.T, t=torch.int32), lp=e(self.T), kept=e(self.T), free=e(self.T, t=torch.int32),
                    x=e(self.T, d, t=torch.bfloat16), again=e(self.T, d, t=torch.bfloat16), dtable=e(V, d),
                    ws=e(M.embed_tokens_backward_workspace_bytes(self.T, V, d), t=torch.uint8))

    def run(self, o, stream=None):
        M.moe_sample_tokens(self.z, self.u, o["tokens"], None, self.k, self.p, None, o["lp"], o["kept"], stream=stream)
        M.moe_sample_tokens(self.z, self.u, o["free"], stream=stream)
        M.moe_embed_tokens(o["tokens"], self.table, 1.5, o["x"], stream=stream)  # of the tokens just drawn
        M.moe_embed_tokens(self.ids, self.table, 1.0, o["again"], stream=stream)
        M.moe_embed_tokens_backward(self.dy, self.ids, 0.5, o["dtable"], o["ws"], stream=stream)
        M.moe_embed_tokens_backward(self.dy, o["tokens"], 2.0, o["dtable"], o["ws"], True, stream=stream)


def same(a, b):
    import torch
    for k in a:
        if k != "ws":
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


SIZES = [(3, 9001, 64, "bf16"), (40, 20000, 128, "f32"), (700, 3001, 256, "bf16"), (1500, 2000, 128, "f32")]


@pytest.mark.parametrize("T,V,d,dtype", SIZES)
def test_replays(T, V, d, dtype):
    import torch
    c = Case(T, V, d, dtype).draw(0)
    captured, plain = c.outputs(), c.outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run(captured)
    for seed in [1, 2, 3]:
        c.draw(seed)
        for _ in range(seed):  # once, and several times in a row
            graph.replay()
        c.run(plain)
        torch.cuda.synchronize()
        same(captured, plain)


def test_streams_and_threads():
    """Each size from a thread of its own on a stream of its own, many times."""
    import torch
    cases = [Case(*s).draw(i) for i, s in enumerate(SIZES)]
    alone, outs, errors = [c.outputs() for c in cases], [c.outputs() for c in cases], []
    for c, o in zip(cases, alone):
        c.run(o)
    torch.cuda.synchronize()
    gate = threading.Barrier(len(cases))

    def work(c, o):
        s = torch.cuda.Stream()
        gate.wait()
        try:
            for i in range(200):
                c.run(o, s)
                if i % 50 == 49:
                    s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))
        s.synchronize()
    threads = [threading.Thread(target=work, args=a) for a in zip(cases, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert errors == []
    for a, b in zip(alone, outs):
        same(a, b)


def test_inputs_written_just_before():
    """No call may read ahead of the kernel that writes its input."""
    import torch
    c = Case(64, 20000, 256, "bf16").draw(0)
    o, w = c.outputs(), c.outputs()
    for seed in range(1, 30):
        c.draw(seed)
        c.run(o)
        torch.cuda.synchronize()
        c.run(w)
        torch.cuda.synchronize()
        same(o, w)


@pytest.mark.parametrize("T", [4, 24])
def test_logit_rows_far_apart(T):
    """Rows whose offsets pass 2^32 elements."""
    import torch
    V, ld = 5003, (1 << 32) // (T - 2) + 1000
    flat = torch.empty(ld * (T - 1) + V, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(flat, (T, V), (ld, 1))
    rng = np.random.default_rng(T)
    h = LR.round_to(rng.standard_normal((T, V)) * 2, "bf16")
    z.copy_(torch.from_numpy(h))
    for kind in ["", "p"]:
        inv_t, k, p, m, u = R.filters(rng, T, kind)
        f = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        tokens = torch.empty(T, dtype=torch.int32, device="cuda")
        M.moe_sample_tokens(z, f(u), tokens, f(inv_t), None, f(p))
        want = R.sample_rows(h, inv_t, k, p, m, u)
        assert (want[3] > 2.0 ** -33).all() and np.array_equal(tokens.cpu().numpy(), want[0])
    del flat, z
    torch.cuda.empty_cache()


def test_table_beyond_32_bits():
    """A table and a gradient of more than 2^31 elements."""
    import torch
    V, d, T = 1100000, 2048, 1300
    table = torch.zeros((V, d), dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, V, (T,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    ids[:40] = V - 1 - torch.arange(40, device="cuda") // 8
    table[ids] = torch.randn((T, d), device="cuda").to(torch.bfloat16)
    out = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    M.moe_embed_tokens(ids.int(), table, 1.0, out)
    assert torch.equal(out, table[ids])
    del table
    torch.cuda.empty_cache()
    dy = torch.randint(-8, 9, (T, d), device="cuda").float()
    for n in [T, 300]:  # sorted, and few
        dtable = torch.full((V, d), 7.0, device="cuda")
        ws = torch.empty(M.embed_tokens_backward_workspace_bytes(n, V, d), dtype=torch.uint8, device="cuda")
        M.moe_embed_tokens_backward(dy[:n].to(torch.bfloat16), ids[:n].int(), 1.0, dtable, ws)
        some, back = ids[:n].unique(return_inverse=True)
        want = torch.zeros((len(some), d), device="cuda").index_add_(0, back, dy[:n])  # whole numbers: exact
        assert torch.equal(dtable[some], want)
        dtable[some] = 0
        assert int(torch.count_nonzero(dtable)) == 0
        del dtable
        torch.cuda.empty_cache()
