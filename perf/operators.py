"""Workloads of the operators around the expert layer: the residual add + RMS
norm in front of it, and the token losses at the learner's other end
(log-probabilities of given tokens, distillation from a teacher's top
logits), each forward and backward.

run() computes a case with plain torch operations in 32 bits, rounded once at
the end, or, where `own` is true, with this package's entry points.  exact()
states the same results from their definitions in 64 bits.

Definitions (T rows; z = logits * inv_t, inv_t the inverse temperature):
  norm      h = bf16(x + res); r = rsqrt(mean h^2 + eps); y = h r w, given in
            BF16 and, with mx8, in E4M3 with one power-of-two scale per 32
            values (the smallest with |y| / scale <= 448), the scales in the
            128 x 4 tile layout.
  norm_bwd  dx = r (dy w - h r mean(dy w h r)) + dh; dw = sum_t dy h r.
  logprobs  logp = z_target - lse(z) (0 without a target); entropy of
            softmax(z); the n_top largest logits, ties to the lower id, with
            their log-probabilities; stats = (max logit, ln sum e^(z - max)).
  logprobs_bwd  dlogits = inv_t (g (1[target] - p) - g_ent p (ln p + H)).
  distill   q_i = e^(a_i inv_t - L) over the listed ids, r = 1 - sum q (L the
            teacher's lse; without it q is normalised over the list, r = 0);
            s = student mass off the list;
            loss = sum q_i (ln q_i - ln p_i) + r (ln r - ln s);
            stats = (max, ln-sum) of the whole row and of its part off the list.
  distill_bwd   dlogits = g inv_t (p - q) on the list, g inv_t t (s - r) off
            it, t = p / s.  distill_train: loss and dlogits in one call.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a small batch: latency
        dict(name="norm_decode", op="norm", T=4, d=2048, mx8=True),
        # a learner micro-batch ahead of the experts
        dict(name="norm_micro", op="norm", T=16384, d=2048, mx8=True),
        # the backward over 16 sequences of 4096 tokens
        dict(name="norm_bwd_micro", op="norm_bwd", T=65536, d=2048),
        # ragged backward of the small layer
        dict(name="norm_bwd_ragged", op="norm_bwd", T=1003, d=1024),
        # one decoding step that reports 20 alternatives
        dict(name="logprobs_decode", op="logprobs", T=2, V=131072, dtype="bf16", n_top=20, pad=0, masked=0, temp=1.0),
        # a learner scoring a rollout
        dict(name="logprobs_score", op="logprobs", T=4096, V=131072, dtype="bf16", n_top=0, pad=0, masked=0, temp=1.0),
        # scoring with alternatives, odd vocabulary, FP32 logits, masked ids, temperature
        dict(name="logprobs_odd", op="logprobs", T=777, V=50001, dtype="f32", n_top=5, pad=0, masked=301, temp=0.7),
        # the policy gradient through log-probabilities and entropy
        dict(name="logprobs_bwd", op="logprobs_bwd", T=4096, V=131072, dtype="bf16", pad=0, masked=0, temp=1.0),
        # distillation loss of a validation batch, FP32 logits
        dict(name="distill_eval", op="distill", T=256, V=32768, dtype="f32", K=32, tail=True, pad=0, masked=0, temp=1.0),
        # its gradient, odd vocabulary in padded rows, list normalised
        dict(name="distill_bwd_odd", op="distill_bwd", T=1024, V=100003, dtype="bf16", K=50, tail=False, pad=5,
             masked=100, temp=2.0),
        # a distillation step: loss and gradient together
        dict(name="distill_train", op="distill_train", T=4096, V=131072, dtype="bf16", K=64, tail=True, pad=0,
             masked=0, temp=1.0),
        # the same on a few rows
        dict(name="distill_train_few", op="distill_train", T=40, V=65536, dtype="bf16", K=16, tail=False, pad=0,
             masked=0, temp=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "logprobs", "logprobs", "logprobs_bwd", "distill", "distill_bwd",
                     "distill_train"])
    if op.startswith("norm"):
        d = 128 * _log_int(rng, 1, 32)
        T = _log_int(rng, 1, 65536 * 2048 // max(d, 2048))
        return dict(op=op, T=T, d=d, mx8=rng.random() < 0.5) if op == "norm" else dict(op=op, T=T, d=d)
    V = _log_int(rng, 1000, 200000)
    if rng.random() < 0.5:
        V = V // 64 * 64
    dtype = rng.choice(["bf16", "bf16", "f32"])
    T = _log_int(rng, 1, 4096 * 131072 // V // (2 if dtype == "f32" else 1))
    c = dict(op=op, T=T, V=V, dtype=dtype, pad=rng.choice([0, 0, 3, 64]), masked=rng.choice([0, 0, V // 50]),
             temp=rng.choice([1.0, 1.0, 0.6, 1.5]))
    if op == "logprobs":
        c["n_top"] = rng.choice([0, 1, 5, 20, 32])
    elif op.startswith("distill"):
        c.update(K=_log_int(rng, 1, 128), tail=rng.random() < 0.5)
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _logit_rows(g, T, V, dtype, pad, masked, n_hot, temp):
    """Peaked rows as a language model gives them: a normal bulk and n_hot ids
    raised by falling amounts.  Returns the logits (a view of rows V + pad
    apart), the raised ids and the raised values' base."""
    free = V - masked
    z = torch.randn((T, V + pad), generator=g, device="cuda") * 2.0
    start = torch.randint(0, free, (T, 1), generator=g, device="cuda")
    step = 7919 if free % 7919 else 7907  # a prime that does not divide free: n_hot different ids
    hot = (start + torch.arange(n_hot, device="cuda") * step) % free
    lift = 11.0 - 1.5 * torch.arange(1, n_hot + 1, device="cuda", dtype=F32).log2()
    lift = lift + torch.randn((T, n_hot), generator=g, device="cuda")
    z.scatter_(1, hot, lift)
    if masked:
        z[:, free:V] = -math.inf
    z = z.mul_(temp).to(BF16 if dtype == "bf16" else F32)
    return z[:, :V], hot, lift


def _full_stats(z, inv_t):
    m = z.amax(1, keepdim=True)
    return m.squeeze(1), ((z - m) * inv_t).exp().sum(1).log()


def _off_list(z, ids):
    return z.scatter(1, ids.long(), -math.inf)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, T = case["op"], case["T"]
    s = dict(case)
    if op in ("norm", "norm_bwd"):
        d = case["d"]
        ch = torch.randint(0, d, (max(1, d // 200),), generator=g, device="cuda")

        def act(std):
            v = torch.randn((T, d), generator=g, device="cuda") * std
            v[:, ch] *= 20.0
            return v.to(BF16)
        s["w"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(BF16)
        s["h"] = act(1.0) if op == "norm_bwd" else torch.empty((T, d), dtype=BF16, device="cuda")
        if op == "norm":
            s["x"], s["res"] = act(0.3), act(1.0)
            s["y"] = torch.empty_like(s["x"])
            s["rstd"] = torch.empty(T, device="cuda")
            if case["mx8"]:
                s["y8"] = torch.empty((T, d), dtype=torch.uint8, device="cuda")
                s["sf"] = torch.zeros((T + 127) // 128 * (d // 128) * 512, dtype=torch.uint8, device="cuda")
        else:
            s["rstd"] = (s["h"].float().square().mean(1) + EPS).rsqrt()
            s["dy"] = (torch.randn((T, d), generator=g, device="cuda") * 1e-3).to(BF16)
            s["dh"] = (torch.randn((T, d), generator=g, device="cuda") * 1e-3).to(BF16)
            s["dx"] = torch.empty((T, d), dtype=BF16, device="cuda")
            s["dw"] = torch.empty(d, device="cuda")
        return s

    V, inv_t = case["V"], 1.0 / case["temp"]
    n_hot = case.get("K", 32)
    s["logits"], hot, lift = _logit_rows(g, T, V, case["dtype"], case["pad"], case["masked"], n_hot, case["temp"])
    s["inv_t"] = inv_t
    if op.startswith("logprobs"):
        pick = torch.randint(0, 8, (T, 1), generator=g, device="cuda")
        s["targets"] = hot.gather(1, pick).squeeze(1).int()
        # one row in ten has no target (prompt tokens)
        s["targets"] = torch.where(torch.rand(T, generator=g, device="cuda") < 0.1, -1, s["targets"]).int()
        s["entropy"] = torch.empty(T, device="cuda")
        s["stats"] = torch.empty((T, 2), device="cuda")
    if op == "logprobs":
        n = case["n_top"]
        s["logprob"] = torch.empty(T, device="cuda")
        s["top_ids"] = torch.empty((T, n), dtype=torch.int32, device="cuda") if n else None
        s["top_logprob"] = torch.empty((T, n), device="cuda") if n else None
    elif op == "logprobs_bwd":
        f = _logprobs_plain(s["logits"], s["targets"], inv_t, 0)
        s["stats"], s["entropy"] = f["stats"], f["entropy"]
        s["g"] = torch.randn(T, generator=g, device="cuda") / T
        s["g_ent"] = torch.full((T,), -0.01 / T, device="cuda")
    else:
        s["ids"] = hot.int()
        # the teacher's logits: near the student's, at the same temperature
        a = (lift + 0.5 * torch.randn((T, n_hot), generator=g, device="cuda")) * case["temp"]
        s["teacher"] = a
        rest = 0.02 + 0.2 * torch.rand(T, generator=g, device="cuda")
        s["teacher_lse"] = torch.logsumexp(a * inv_t, 1) - (1 - rest).log() if case["tail"] else None
        s["loss"] = torch.empty(T, device="cuda")
        s["g"] = (0.5 + torch.rand(T, generator=g, device="cuda")) / T
        if op == "distill_bwd":
            z = s["logits"].float()
            s["stats"] = torch.stack(_full_stats(z, inv_t) + _full_stats(_off_list(z, s["ids"]), inv_t), 1)
        else:
            s["stats"] = torch.empty((T, 4), device="cuda")
    if op in ("logprobs_bwd", "distill_bwd", "distill_train"):
        s["dlogits"] = torch.empty((T, V + case["pad"]), dtype=s["logits"].dtype, device="cuda")[:, :V]
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _tiled_scales(e8, T, d):
    """Scale bytes [T][d/32] into the 128 x 4 tile layout."""
    r = torch.arange(T, device="cuda")[:, None]
    c = torch.arange(d // 32, device="cuda")[None, :]
    at = ((r // 128) * (d // 128) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    out = torch.zeros((T + 127) // 128 * (d // 128) * 512, dtype=torch.uint8, device="cuda")
    out[at.reshape(-1)] = e8.reshape(-1)
    return out


def _norm_plain(s):
    h = (s["x"].float() + s["res"].float()).to(BF16)
    hf = h.float()
    rstd = (hf.square().mean(1) + EPS).rsqrt()
    y = hf * rstd[:, None] * s["w"].float()
    out = dict(h=h, y=y.to(BF16), rstd=rstd)
    if s["mx8"]:
        T, d = y.shape
        b = y.view(T, d // 32, 32)
        f, e = torch.frexp(b.abs().amax(2))  # amax = f 2^e, f in [0.5, 1); 448 = 0.875 * 2^9
        e = torch.where(f > 0.875, e - 8, e - 9).clamp(-127, 127)
        e = torch.where(f == 0, -127, e)
        q = torch.ldexp(b, -e[:, :, None].float()).to(torch.float8_e4m3fn)
        out["y8"] = q.view(T, d)
        out["scales"] = _tiled_scales((e + 127).to(torch.uint8), T, d).view(torch.float8_e8m0fnu)
    return out


def _norm_bwd_plain(s):
    hf, dy, r = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = hf * r
    gy = dy * s["w"].float()
    c = (gy * xhat).mean(1, keepdim=True)
    return dict(dx=(r * (gy - xhat * c) + s["dh"].float()).to(BF16), dw=(dy * xhat).sum(0))


def _logprobs_plain(logits, targets, inv_t, n_top):
    z = logits.float()
    m, l = _full_stats(z, inv_t)
    dist = (z - m[:, None]) * inv_t
    p = (dist - l[:, None]).exp()
    entropy = l - torch.where(p > 0, p * dist, 0.0).sum(1)
    t = targets.long()
    lp = dist.gather(1, t.clamp(min=0)[:, None]).squeeze(1) - l
    out = dict(logprob=torch.where(t >= 0, lp, 0.0), entropy=entropy, stats=torch.stack((m, l), 1))
    if n_top:
        # one whole number per logit, ordered by (value, lower id first)
        b = (z + 0.0).view(torch.int32)
        order = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
        V = z.shape[1]
        key = order * (1 << 24) + (V - 1 - torch.arange(V, device=z.device))
        at = V - 1 - (key.topk(n_top, 1).values & ((1 << 24) - 1))
        out["top_ids"] = at.int()
        out["top_logprob"] = dist.gather(1, at) - l[:, None]
    return out


def _logprobs_bwd_plain(s):
    z, inv_t = s["logits"].float(), s["inv_t"]
    lp = (z - s["stats"][:, :1]) * inv_t - s["stats"][:, 1:]
    p = lp.exp()
    t = s["targets"].long()
    g = torch.where(t >= 0, s["g"], 0.0)
    d = -p * g[:, None] - s["g_ent"][:, None] * torch.where(p > 0, p * (lp + s["entropy"][:, None]), 0.0)
    d.scatter_add_(1, t.clamp(min=0)[:, None], g[:, None])
    return dict(dlogits=(d * inv_t).to(s["logits"].dtype))


def _teacher(s):
    """q over the list, ln q, and the mass r off it."""
    a = s["teacher"] * s["inv_t"]
    if s["teacher_lse"] is None:
        mx = a.amax(1, keepdim=True)
        lq = a - mx - (a - mx).exp().sum(1, keepdim=True).log()
        return lq.exp(), lq, torch.zeros_like(a[:, 0])
    lq = a - s["teacher_lse"][:, None]
    q = lq.exp()
    return q, lq, (1.0 - q.sum(1)).clamp(min=0.0)


def _distill_plain(s, loss, grad):
    z, inv_t, ids = s["logits"].float(), s["inv_t"], s["ids"].long()
    q, lq, r = _teacher(s)
    off = _off_list(z, ids)
    if loss:
        m, l = _full_stats(z, inv_t)
        mt, lt = _full_stats(off, inv_t)
    else:
        m, l, mt, lt = s["stats"].unbind(1)
    lp = (z.gather(1, ids) - m[:, None]) * inv_t - l[:, None]
    ls = (mt - m) * inv_t + lt - l  # ln of the student's mass off the list
    out = {}
    if loss:
        cross = (q * (lq - lp)).sum(1)
        out["loss"] = cross + torch.where(r > 0, r * (r.log() - ls), 0.0)
        if not grad:
            out["stats"] = torch.stack((m, l, mt, lt), 1)
    if grad:
        d = ((off - mt[:, None]) * inv_t - lt[:, None]).exp() * (ls.exp() - r)[:, None]
        d.scatter_(1, ids, lp.exp() - q)
        out["dlogits"] = (d * (s["g"] * inv_t)[:, None]).to(s["logits"].dtype)
    return out


# --------------------------------------------------------------------------
# run
# --------------------------------------------------------------------------
def _run_own(s):
    import nvfp4_w4a4_moe_top_gb300 as M
    op = s["op"]
    if op == "norm":
        mx8 = s["mx8"]
        y8, sf = (s["y8"], s["sf"]) if mx8 else (None, None)
        M.moe_add_rmsnorm(s["x"], s["res"], s["w"], EPS, s["h"], s["y"], y8, sf, s["rstd"])
        out = dict(h=s["h"], y=s["y"], rstd=s["rstd"])
        if mx8:
            out["y8"], out["scales"] = y8.view(torch.float8_e4m3fn), sf.view(torch.float8_e8m0fnu)
        return out
    if op == "norm_bwd":
        if "ws" not in s:
            s["ws"] = torch.empty(M.add_rmsnorm_backward_workspace_bytes(s["T"], s["d"]), dtype=torch.uint8,
                                  device="cuda")
        M.moe_add_rmsnorm_backward(s["dy"], s["dh"], s["h"], s["rstd"], s["w"], s["dx"], s["dw"], s["ws"])
        return dict(dx=s["dx"], dw=s["dw"])
    if op == "logprobs":
        M.moe_token_logprobs(s["logits"], s["targets"], s["inv_t"], s["n_top"], s["logprob"], s["entropy"],
                             s["stats"], s["top_ids"], s["top_logprob"])
        out = dict(logprob=s["logprob"], entropy=s["entropy"], stats=s["stats"])
        if s["n_top"]:
            out.update(top_ids=s["top_ids"], top_logprob=s["top_logprob"])
        return out
    if op == "logprobs_bwd":
        M.moe_token_logprobs_backward(s["logits"], s["targets"], s["inv_t"], s["stats"], s["entropy"], s["g"],
                                      s["g_ent"], s["dlogits"])
        return dict(dlogits=s["dlogits"])
    if op == "distill":
        M.moe_distill_topk(s["logits"], s["ids"], s["teacher"], s["teacher_lse"], s["inv_t"], s["loss"], s["stats"])
        return dict(loss=s["loss"], stats=s["stats"])
    if op == "distill_bwd":
        M.moe_distill_topk_backward(s["logits"], s["ids"], s["teacher"], s["teacher_lse"], s["inv_t"], s["stats"],
                                    s["g"], s["dlogits"])
        return dict(dlogits=s["dlogits"])
    M.moe_distill_topk_train(s["logits"], s["ids"], s["teacher"], s["teacher_lse"], s["inv_t"], s["g"], s["loss"],
                             s["dlogits"])
    return dict(loss=s["loss"], dlogits=s["dlogits"])


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "norm":
        return _norm_plain(state)
    if op == "norm_bwd":
        return _norm_bwd_plain(state)
    if op == "logprobs":
        return _logprobs_plain(state["logits"], state["targets"], state["inv_t"], state["n_top"])
    if op == "logprobs_bwd":
        return _logprobs_bwd_plain(state)
    return _distill_plain(state, loss=op != "distill_bwd", grad=op != "distill")


def work(case):
    """Each input read once and each output written once; the operations
    every element needs (an exponential counted as one)."""
    op, T = case["op"], case["T"]
    if op == "norm":
        n = T * case["d"]
        return dict(bytes=n * 8 + (n + n // 32 if case["mx8"] else 0) + 4 * T + 2 * case["d"],
                    flops=n * (6 + (3 if case["mx8"] else 0)))
    if op == "norm_bwd":
        n = T * case["d"]
        return dict(bytes=n * 8 + 4 * T + 6 * case["d"], flops=n * 11)
    V, size = case["V"], 2 if case["dtype"] == "bf16" else 4
    n = T * V
    if op == "logprobs":
        return dict(bytes=n * size + T * (20 + 8 * case["n_top"]), flops=n * 7)
    if op == "logprobs_bwd":
        return dict(bytes=2 * n * size + T * 24, flops=n * 7)
    lists = T * (8 * case["K"] + (4 if case["tail"] else 0))
    if op == "distill":
        return dict(bytes=n * size + lists + T * 20, flops=n * 5)
    if op == "distill_bwd":
        return dict(bytes=2 * n * size + lists + T * 20, flops=n * 4)
    return dict(bytes=2 * n * size + lists + T * 8, flops=n * 8)


# --------------------------------------------------------------------------
# the same from the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "norm":
        h = (s["x"].to(f64) + s["res"].to(f64))
        hd = h.float().to(BF16).to(f64)
        rstd = 1.0 / torch.sqrt((hd * hd).sum(1) / case["d"] + EPS)
        out = dict(h=h, y=hd * rstd.unsqueeze(1) * s["w"].to(f64), rstd=rstd)
        if case["mx8"]:
            out.update(y8=None, scales=None)
        return out
    if op == "norm_bwd":
        # by the chain rule through y_i = h_i w_i r(h)
        h, w, dy = s["h"].to(f64), s["w"].to(f64), s["dy"].to(f64)
        r = s["rstd"].to(f64).unsqueeze(1)
        inner = torch.einsum("td,td->t", dy * w, h).unsqueeze(1)
        dx = dy * w * r - h * inner * r ** 3 / case["d"] + s["dh"].to(f64)
        return dict(dx=dx, dw=torch.einsum("td,td->d", dy, h * r))
    z = s["logits"].to(f64) * s["inv_t"]
    lse = torch.logsumexp(z, 1)
    if op.startswith("logprobs"):
        lp = z - lse.unsqueeze(1)
        p = torch.exp(lp)
        ent = -torch.special.xlogy(p, p).sum(1)
        t = s["targets"].long()
        has = t >= 0
        rows = torch.arange(len(t), device="cuda")
        if op == "logprobs":
            m = s["logits"].amax(1).to(f64)
            out = dict(logprob=torch.where(has, lp[rows, t.clamp(min=0)], 0.0), entropy=ent,
                       stats=torch.stack((m, lse - m * s["inv_t"]), 1))
            if case["n_top"]:
                out.update(top_ids=None, top_logprob=lp.topk(case["n_top"], 1).values)
            return out
        # d entropy / dz_v = -p_v ln p_v - p_v H
        dz = (-torch.special.xlogy(p, p) - p * ent.unsqueeze(1)) * s["g_ent"].to(f64).unsqueeze(1)
        g = torch.where(has, s["g"].to(f64), 0.0)
        dz -= p * g.unsqueeze(1)
        dz[rows, t.clamp(min=0)] += g
        return dict(dlogits=dz * s["inv_t"])
    ids = s["ids"].long()
    a = s["teacher"].to(f64) * s["inv_t"]
    listed_mask = torch.zeros(z.shape, dtype=torch.bool, device="cuda")
    listed_mask.scatter_(1, ids, True)
    off = z.masked_fill(listed_mask, -math.inf)
    lse_off = torch.logsumexp(off, 1)
    mass = torch.exp(lse_off - lse)
    if case["tail"]:
        q = torch.exp(a - s["teacher_lse"].to(f64).unsqueeze(1))
        r = (1 - q.sum(1)).clamp(min=0)
    else:
        q = torch.softmax(a, 1)
        r = torch.zeros_like(mass)
    out = {}
    if op != "distill_bwd":
        lp = z.gather(1, ids) - lse.unsqueeze(1)
        out["loss"] = (torch.special.xlogy(q, q) - q * lp).sum(1) + torch.special.xlogy(r, r) - r * (lse_off - lse)
    if op == "distill":
        m, mt = s["logits"].amax(1).to(f64), off.amax(1)
        out["stats"] = torch.stack((m, lse - m * s["inv_t"], mt / s["inv_t"], lse_off - mt), 1)
    else:
        dz = torch.exp(off - lse.unsqueeze(1)) * (1 - r / mass).unsqueeze(1)
        dz.scatter_(1, ids, torch.exp(z.gather(1, ids) - lse.unsqueeze(1)) - q)
        out["dlogits"] = dz * (s["g"].to(f64) * s["inv_t"]).unsqueeze(1)
    return out
