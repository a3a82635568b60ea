"""Workloads of the operators at a model's token ends: the embedding of given
tokens and its gradient, and the draw of the next token from the logits.

run() computes a case with plain torch operations, or, where `own` is true,
with this package's entry points.  exact() states the same results from their
definitions in 64 bits.

Definitions (T tokens or rows, V ids):
  embed      out_t = bf16(scale * table[ids_t]); zeros where ids_t < 0.
  embed_bwd  dtable_v = scale * sum of dy_t over ids_t = v, in FP32, all V rows.
  sample     z = logits * inv_t of the row, w = e^(z - max z), 0 where that is
             below 2^-42.  Kept are the ids among the top_k first in the order
             (logit descending, id ascending), of these the shortest leading
             part with at least top_p of their weight, of these the ones with
             w >= min_p.  The token is the first kept id, in the order of the
             ids, up to which the kept weight is above u times all of it.
             logprob = ln(w / sum of all w), kept_logprob = ln(w / kept weight).
Filters that are off: top_k 0, top_p 1, min_p 0.  The draw's weights, sums and
comparisons are in 64 bits, as a token is one or another.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
OFF = dict(top_k=0, top_p=1.0, min_p=0.0, temp=1.0)
CHUNK = 1 << 26  # logits that the plain draw works on at a time


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _sample(name, T, V, dtype, pad=0, masked=0, mixed=False, **filters):
    return dict(name=name, op="sample", T=T, V=V, dtype=dtype, pad=pad, masked=masked, mixed=mixed, **{**OFF, **filters})


def _embed(name, op, T, V, d, dtype="bf16", scale=1.0, pads=0.0):
    return dict(name=name, op=op, T=T, V=V, d=d, dtype=dtype, scale=scale, pads=pads)


def listed():
    return [
        # one decoding step of two conversations: latency
        _sample("sample_decode", 2, 131072, "bf16", top_p=0.95, temp=0.8),
        # a step of an on-policy rollout: the policy itself, no filter
        _sample("sample_rollout", 512, 131072, "bf16"),
        # a serving batch with the usual filters
        _sample("sample_top_k", 256, 131072, "bf16", top_k=50, top_p=0.95, temp=0.7),
        # the largest rollout step, with a nucleus
        _sample("sample_top_p", 2048, 131072, "bf16", top_p=0.95),
        # hot sampling from a few padded rows of an odd vocabulary
        _sample("sample_min_p", 64, 100003, "bf16", pad=5, min_p=0.05, temp=1.5),
        # requests with filters of their own, FP32 logits, masked ids
        _sample("sample_mixed", 777, 50001, "f32", pad=3, masked=301, mixed=True),
        # the tokens of one decoding step: latency
        _embed("embed_decode", "embed", 16, 131072, 2048),
        # a learner micro-batch of 16 sequences of 4096 tokens
        _embed("embed_micro", "embed", 65536, 131072, 2048),
        # FP32 table, scaled, rows that are no multiple of a cache line, padded batch
        _embed("embed_odd", "embed", 5003, 50001, 1000, dtype="f32", scale=1000 ** 0.5, pads=0.1),
        # the micro-batch's gradient
        _embed("embed_bwd_micro", "embed_bwd", 65536, 131072, 2048),
        # a few sequences and a smaller vocabulary
        _embed("embed_bwd_few", "embed_bwd", 512, 32768, 1024),
        # ragged, scaled, padded batch
        _embed("embed_bwd_odd", "embed_bwd", 16003, 50001, 1000, scale=1000 ** 0.5, pads=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "embed", "embed_bwd"])
    if op == "sample":
        V = _log_int(rng, 1000, 200000)
        if rng.random() < 0.5:
            V = V // 64 * 64
        dtype = rng.choice(["bf16", "bf16", "f32"])
        T = _log_int(rng, 1, 2048 * 131072 // V // (2 if dtype == "f32" else 1))
        kind = rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"])
        c = dict(OFF, op=op, T=T, V=V, dtype=dtype, pad=rng.choice([0, 0, 3, 64]), masked=rng.choice([0, 0, V // 50]),
                 mixed=kind == "mixed", temp=rng.choice([1.0, 1.0, 0.6, 1.5]))
        if kind in ("top_k", "all"):
            c["top_k"] = _log_int(rng, 1, V // 2)
        if kind in ("top_p", "all"):
            c["top_p"] = rng.choice([0.5, 0.8, 0.95, 0.99])
        if kind in ("min_p", "all"):
            c["min_p"] = rng.choice([0.001, 0.02, 0.1])
        return c
    d = 8 * _log_int(rng, 8, 512)
    V = _log_int(rng, 1000, 131072 * 2048 // max(d, 2048))
    T = _log_int(rng, 1, 65536 * 2048 // max(d, 2048))
    dtype = rng.choice(["bf16", "bf16", "f32"]) if op == "embed" else "bf16"
    if dtype == "f32":
        T = max(1, T // 2)
    return dict(op=op, T=T, V=V, d=d, dtype=dtype, scale=rng.choice([1.0, 1.0, d ** 0.5]), pads=rng.choice([0.0, 0.0, 0.2]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _logit_rows(g, T, V, dtype, pad, masked, temp):
    """Rows as a language model gives them: a normal bulk and 64 raised ids of
    falling logits.  How far the row's first is raised varies, so that most rows
    are decided by a few ids and one in seven is left to the bulk.  Returns a
    view of rows V + pad apart."""
    free = V - masked
    z = torch.randn((T, V + pad), generator=g, device="cuda") * 2.0
    start = torch.randint(0, free, (T, 1), generator=g, device="cuda")
    step = 7919 if free % 7919 else 7907  # a prime that does not divide free: different ids
    hot = (start + torch.arange(64, device="cuda") * step) % free
    lift = math.log(V) + 8.2 + 3.0 * torch.randn((T, 1), generator=g, device="cuda")
    lift = lift - 1.5 * torch.arange(1, 65, device="cuda", dtype=F32).log2()
    z.scatter_(1, hot, lift + torch.randn((T, 64), generator=g, device="cuda"))
    if masked:
        z[:, free:V] = -math.inf
    return z.mul_(temp).to(BF16 if dtype == "bf16" else F32)[:, :V]


def _token_ids(g, T, V, pads):
    """Ids whose frequency falls as 1 / (id + 1), as a tokeniser orders them;
    a part of the batch is padding (-1)."""
    r = torch.rand(T, generator=g, device="cuda", dtype=F64)
    ids = (r * math.log(V)).exp().floor().long().clamp(1, V) - 1
    return torch.where(torch.rand(T, generator=g, device="cuda") < pads, -1, ids).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    T, V = case["T"], case["V"]
    s = dict(case)
    if case["op"] != "sample":
        d = case["d"]
        s["ids"] = _token_ids(g, T, V, case["pads"])
        if case["op"] == "embed":
            s["table"] = torch.randn((V, d), generator=g, device="cuda").mul_(0.02)
            if case["dtype"] == "bf16":
                s["table"] = s["table"].to(BF16)
            s["out"] = torch.empty((T, d), dtype=BF16, device="cuda")
        else:
            s["dy"] = (torch.randn((T, d), generator=g, device="cuda") * 1e-3).to(BF16)
            s["dtable"] = torch.empty((V, d), device="cuda")
        return s
    s["logits"] = _logit_rows(g, T, V, case["dtype"], case["pad"], case["masked"], case["temp"])
    full = lambda v, t: torch.full((T,), v, dtype=t, device="cuda")  # noqa: E731
    if case["mixed"]:  # every request its own
        def pick(values, t):
            at = torch.randint(0, len(values), (T,), generator=g, device="cuda")
            return torch.tensor(values, dtype=t, device="cuda")[at]
        s["inv_t"] = 1.0 / pick([0.6, 0.8, 1.0, 1.0, 1.3], F32)
        s["k"] = pick([0, 0, 1, 20, 50, 1000], torch.int32)
        s["p"] = pick([1.0, 1.0, 0.5, 0.9, 0.95, 0.99], F32)
        s["m"] = pick([0.0, 0.0, 0.0, 0.02, 0.1], F32)
    else:
        s["inv_t"] = full(1.0 / case["temp"], F32)
        s["k"] = full(case["top_k"], torch.int32) if case["top_k"] else None
        s["p"] = full(case["top_p"], F32) if case["top_p"] < 1 else None
        s["m"] = full(case["min_p"], F32) if case["min_p"] else None
    s["u"] = torch.rand(T, generator=g, device="cuda")
    s["tokens"] = torch.empty(T, dtype=torch.int32, device="cuda")
    s["logprob"], s["kept_logprob"] = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _embed_plain(s):
    ids = s["ids"].long()
    rows = s["table"][ids.clamp(min=0)].float() * s["scale"]
    return dict(out=torch.where(ids[:, None] >= 0, rows, 0.0).to(BF16))


def _embed_bwd_plain(s):
    ids = s["ids"].long()
    V = s["V"]
    out = torch.zeros((V + 1, s["d"]), device="cuda")  # the last row takes the padding
    out.index_add_(0, torch.where(ids >= 0, ids, V), s["dy"].float())
    return dict(dtable=out[:V] * s["scale"])


def _sample_rows(x, inv_t, k, p, m, u):
    z = x.to(F64) * inv_t.to(F64)[:, None]
    z = z - z.amax(1, keepdim=True)
    w = z.exp()
    w = torch.where(w < 2.0 ** -42, 0.0, w)
    total = w.sum(1)
    kept = w
    if k is not None or p is not None:
        order = x.float().sort(dim=1, descending=True, stable=True).indices
        first = w.gather(1, order)
        if k is not None:
            place = torch.arange(x.shape[1], device=x.device)
            limit = torch.where(k > 0, k, x.shape[1])
            first = torch.where(place < limit[:, None], first, 0.0)
        if p is not None:
            sums = first.cumsum(1)
            before = torch.cat((torch.zeros_like(sums[:, :1]), sums[:, :-1]), 1)
            within = before < p.to(F64)[:, None] * sums[:, -1:]
            within |= p[:, None] >= 1
            first = torch.where(within, first, 0.0)
        kept = torch.zeros_like(w).scatter_(1, order, first)
    if m is not None:
        kept = torch.where(w >= m.to(F64)[:, None], kept, 0.0)
    sums = kept.cumsum(1)
    mass = sums[:, -1]
    token = (sums <= (u.to(F64) * mass)[:, None]).sum(1)
    zt = z.gather(1, token[:, None]).squeeze(1)
    return token.int(), (zt - total.log()).float(), (zt - mass.log()).float()


def _sample_plain(s):
    n = max(1, CHUNK // s["V"])
    parts = [tuple(v[i:i + n] if v is not None else None
                   for v in (s["logits"], s["inv_t"], s["k"], s["p"], s["m"], s["u"])) for i in range(0, s["T"], n)]
    tokens, logprob, kept = (torch.cat(v) for v in zip(*(_sample_rows(*part) for part in parts)))
    return dict(tokens=tokens, logprob=logprob, kept_logprob=kept)


# --------------------------------------------------------------------------
# run
# --------------------------------------------------------------------------
def _run_own(s):
    import nvfp4_w4a4_moe_top_gb300 as M
    if s["op"] == "embed":
        M.moe_embed_tokens(s["ids"], s["table"], s["scale"], s["out"])
        return dict(out=s["out"])
    if s["op"] == "embed_bwd":
        if "ws" not in s:
            s["ws"] = torch.empty(M.embed_tokens_backward_workspace_bytes(s["T"], s["V"], s["d"]), dtype=torch.uint8,
                                  device="cuda")
        M.moe_embed_tokens_backward(s["dy"], s["ids"], s["scale"], s["dtable"], s["ws"])
        return dict(dtable=s["dtable"])
    M.moe_sample_tokens(s["logits"], s["u"], s["tokens"], s["inv_t"], s["k"], s["p"], s["m"], s["logprob"],
                        s["kept_logprob"])
    return dict(tokens=s["tokens"], logprob=s["logprob"], kept_logprob=s["kept_logprob"])


def run(state):
    if own:
        return _run_own(state)
    return dict(embed=_embed_plain, embed_bwd=_embed_bwd_plain, sample=_sample_plain)[state["op"]](state)


def work(case):
    """Each input read once and each output written once (of a table the rows
    that the tokens name); the operations every element needs (an exponential
    counted as one)."""
    T, V = case["T"], case["V"]
    if case["op"] == "sample":
        n = T * V
        return dict(bytes=n * (2 if case["dtype"] == "bf16" else 4) + T * 32, flops=n * 4)
    n = T * case["d"]
    if case["op"] == "embed":
        often = T / math.log(V)  # ids below it are all there, of a later id v one in v / often
        rows = min(T, V, often * (1 + math.log(V / often))) if often < V else V
        return dict(bytes=rows * case["d"] * (2 if case["dtype"] == "bf16" else 4) + n * 2 + 4 * T, flops=n)
    return dict(bytes=n * 2 + 4 * T + V * case["d"] * 4, flops=n + V * case["d"])


# --------------------------------------------------------------------------
# the same from the definitions in 64 bits
# --------------------------------------------------------------------------
def _sample_exact(x, inv_t, k, p, m, u):
    """One row: the ids that remain, filter by filter, and the draw among them."""
    z = x.to(F64) * inv_t
    lse = torch.logsumexp(z, 0)
    ids = torch.nonzero(z >= z.max() - 42 * math.log(2)).squeeze(1)
    left = ids[torch.argsort(-x[ids].to(F64), stable=True)]
    if k > 0:
        left = left[:k]
    if p < 1:
        share = torch.softmax(z[left], 0)
        # ids that the heavier ones before them leave below top_p
        left = left[(share.cumsum(0) - share) < p * share.sum()]
    if m > 0:
        left = left[(z[left] - z.max()).exp() >= m]
    left = left.sort().values
    cdf = torch.softmax(z[left], 0).cumsum(0)
    token = left[torch.searchsorted(cdf, u * cdf[-1], right=True).clamp(max=len(left) - 1)]
    return token, z[token] - lse, z[token] - torch.logsumexp(z[left], 0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = torch.zeros((case["T"], case["d"]), dtype=F64, device="cuda")
        has = s["ids"] >= 0
        out[has] = s["table"].index_select(0, s["ids"][has]).to(F64).mul_(case["scale"])
        return dict(out=out)
    if case["op"] == "embed_bwd":
        has = torch.nonzero(s["ids"] >= 0).squeeze(1)
        out = torch.zeros((case["V"], case["d"]), dtype=F64, device="cuda")
        out.index_put_((s["ids"][has].long(),), s["dy"][has].to(F64).mul_(case["scale"]), accumulate=True)
        return dict(dtable=out)
    if case["T"] > 8192:
        return None  # row by row it would take too long
    f = lambda v, off: [off] * case["T"] if v is None else v.to(F64).tolist()  # noqa: E731
    rows = zip(s["logits"], f(s["inv_t"], 1.0), map(int, f(s["k"], 0)), f(s["p"], 1.0), f(s["m"], 0.0), s["u"].to(F64))
    tokens, logprob, kept = (torch.stack(v) for v in zip(*(_sample_exact(*row) for row in rows)))
    return dict(tokens=tokens, logprob=logprob, kept_logprob=kept)
