"""The learner operators from their definitions in 64-bit numpy (no framework
code), and the inputs of their tests."""
import numpy as np

F64 = np.float64
LOWEST = {"bf16": -3.3895313892515355e38, "f32": -3.4028234663852886e38}


def log_softmax(z):
    """Rows of log p; a row of nothing but -inf gives -inf throughout."""
    m = z.max(1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        return z - m - np.log(np.exp(z - m).sum(1, keepdims=True)) if z.size else z


def xlogx(p):
    return np.where(p > 0, p * np.log(np.where(p > 0, p, 1.0)), 0.0)


def logprobs(logits, targets, inv_t, n_top):
    z = logits.astype(F64) * inv_t
    T, V = z.shape
    none = np.isneginf(z).all(1)
    lp = np.where(none[:, None], -np.inf, log_softmax(z))
    has = (targets >= 0) & (targets < V)
    m = logits.astype(F64).max(1)
    with np.errstate(invalid="ignore", over="ignore"):
        l = np.log(np.exp((logits.astype(F64) - np.where(none, 0, m)[:, None]) * inv_t).sum(1) + none)
    order = np.argsort(-logits.astype(F64), axis=1, kind="stable")[:, :n_top]  # ties: lower id first
    ids = np.full((T, n_top), -1)
    top = np.full((T, n_top), -np.inf)
    ids[:, :order.shape[1]] = order
    top[:, :order.shape[1]] = np.take_along_axis(lp, order, 1)
    ids = np.where(np.isneginf(top), np.where(np.isneginf(np.take_along_axis(
        logits.astype(F64), np.maximum(ids, 0), 1)) | (ids < 0), -1, ids), ids)
    return dict(logprob=np.where(has, lp[np.arange(T), np.where(has, targets, 0)], 0.0),
                entropy=np.where(none, 0.0, -xlogx(np.exp(lp)).sum(1)),
                stats=np.stack((np.where(none, -np.inf, m), np.where(none, 0.0, l)), 1), top_ids=ids,
                top_logprob=top, lp=lp)


def logprobs_grad(logits, targets, inv_t, g, ge):
    f = logprobs(logits, targets, inv_t, 0)
    T, V = logits.shape
    p = np.exp(f["lp"])
    has = (targets >= 0) & (targets < V)
    g = np.where(has, g, 0.0)
    d = -p * g[:, None] - ge[:, None] * (xlogx(p) + p * f["entropy"][:, None])
    d[np.arange(T), np.where(has, targets, 0)] += g
    return np.where(np.isneginf(f["lp"]).all(1)[:, None], 0.0, d * inv_t)


def keep_entries(ids, V):
    """Entries that count: in range, and the first of their id in the row."""
    ok = (ids >= 0) & (ids < V)
    for t in range(ids.shape[0]):
        seen = set()
        for j in range(ids.shape[1]):
            ok[t, j] &= ids[t, j] not in seen
            seen.add(ids[t, j])
    return ok


def distill(logits, ids, a, lse, inv_t):
    """loss, d loss / d logits and stats, row by row."""
    z = logits.astype(F64) * inv_t
    T, V = z.shape
    ok = keep_entries(ids, V)
    loss, grad, stats = np.zeros(T), np.zeros((T, V)), np.zeros((T, 4))
    for t in range(T):
        k = ids[t][ok[t]]
        at = a[t][ok[t]].astype(F64) * inv_t
        if lse is None:
            e = np.exp(at - at.max()) if len(at) else at
            q, r = (e / e.sum() if len(e) else e), 0.0
        else:
            q = np.exp(at - float(lse[t]))
            r = max(0.0, 1.0 - q.sum())
        Q = q.sum() + r
        on = np.zeros(V, bool)
        on[k] = True
        none = np.isneginf(z[t]).all()
        w = np.exp(z[t] - (0 if none else z[t].max()))
        p = w / w.sum() if not none else w
        off_empty = np.isneginf(z[t][~on]).all()
        if off_empty:
            ls, tt = -np.inf, np.zeros(V)
        else:
            zo = np.where(on, -np.inf, z[t])
            wo = np.exp(zo - zo.max())
            tt = wo / wo.sum()
            ls = zo.max() - z[t].max() + np.log(wo.sum()) - np.log(w.sum())
        with np.errstate(divide="ignore", invalid="ignore"):
            lp = z[t][k] - (0 if none else z[t].max()) - (0 if none else np.log(w.sum()))
            terms = np.where(q > 0, q * (np.log(np.where(q > 0, q, 1)) - lp), 0.0)
            loss[t] = terms.sum() + (r * (np.log(r) - ls) if r > 0 else 0.0)
        if none:
            loss[t] = np.inf if Q > 0 else 0.0
        else:
            g = tt * (np.exp(ls) * Q - r)
            g[k] = p[k] * Q - q
            grad[t] = g * inv_t
        x = logits[t].astype(F64)
        stats[t] = [-np.inf if none else x.max(), 0.0 if none else np.log(np.exp((x - x.max()) * inv_t).sum()),
                    -np.inf if off_empty else x[~on].max(),
                    0.0 if off_empty else np.log(np.exp((x[~on] - x[~on].max()) * inv_t).sum())]
    return loss, grad, stats


def round_to(x, dtype):
    """Values as the type holds them (bf16 by torch's cast), in float32."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    return (t.to(torch.bfloat16).float() if dtype == "bf16" else t).numpy()


def logit_rows(rng, T, V, dtype, ties=False):
    """Peaked rows, with the rows that masks make special: everything masked
    but one id, nothing left, everything at the type's lowest value, a third
    masked by -inf, a third by the lowest value."""
    z = rng.standard_normal((T, V)) * 2
    for t in range(T):
        hot = rng.integers(0, V, 6)
        z[t, hot] = 9 - np.arange(6) + rng.standard_normal(6)
    if ties:
        z = np.round(z)
    z = round_to(z, dtype)
    if T > 5:
        z[1] = -np.inf
        z[1, rng.integers(V)] = 1.5
        z[2] = -np.inf
        z[3] = LOWEST[dtype]
        z[4, rng.random(V) < 0.33] = -np.inf
        z[5, rng.random(V) < 0.33] = LOWEST[dtype]
    return z


def device_rows(z, dtype, pad=0, lead=0, fill=float("nan")):
    """z as a device tensor whose rows lie V + pad elements apart and start
    `lead` elements into their storage; the gaps hold `fill`."""
    import torch
    T, V = z.shape
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    flat = torch.full((T * (V + pad) + lead,), fill, dtype=dt, device="cuda")
    v = flat[lead:].view(T, V + pad)[:, :V] if T else flat[:0].view(0, V)
    v.copy_(torch.from_numpy(z).to(dt))
    return v
