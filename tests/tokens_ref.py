"""The operators at the token ends from their definitions in 64-bit numpy (no
framework code), and the inputs of their tests."""
import numpy as np

F64 = np.float64
CUT = 2.0 ** -42


def embed(ids, table, scale):
    """Rows in FP32 before the rounding to BF16."""
    ok = (ids >= 0) & (ids < len(table))
    rows = table[np.where(ok, ids, 0)].astype(np.float32) * np.float32(scale)
    return np.where(ok[:, None], rows, np.float32(0))


def embed_grad(dy, ids, V, scale, start=None):
    """(the gradient, the sum of the magnitudes that went into each value, the
    number of them)."""
    ok = (ids >= 0) & (ids < V)
    g, mag = np.zeros((V, dy.shape[1]), F64), np.zeros((V, dy.shape[1]), F64)
    np.add.at(g, ids[ok], dy[ok].astype(F64))
    np.add.at(mag, ids[ok], np.abs(dy[ok].astype(F64)))
    n = np.bincount(ids[ok], minlength=V)
    if start is not None:
        return start.astype(F64) + g * scale, mag * abs(scale) + np.abs(start), n
    return g * scale, mag * abs(scale), n


def sample(x, inv_t, k, p, m, u, moved=0):
    """One row: (token, logprob, kept_logprob, margin).  margin is the least
    distance of a decision from its border, as a part of the weight in question;
    inf where that is of equal logits only, w = 1, whose sums are exact.  An end of
    the top_p part that is close to its border does not count where one id more
    and one id less (moved) give the same token."""
    given, x = x, x.astype(F64)
    V = len(x)
    if np.isnan(x).any() or np.isposinf(x).any():
        return -1, np.nan, np.nan, np.inf
    if np.isneginf(x).all():
        return -1, -np.inf, -np.inf, np.inf
    x = x + 0.0  # -0 is 0
    with np.errstate(over="ignore"):
        z = (x - x.max()) * float(inv_t)
        w = np.exp(z)
    w[w < CUT] = 0.0
    order = np.argsort(-x, kind="stable")
    order = order[np.isfinite(x[order])]
    margin = np.inf
    flat = lambda ids: bool(((w[ids] == 0) | (w[ids] == 1)).all())  # noqa: E731
    if 0 < k < V:
        order = order[:k]
    if p < 1:
        c = np.cumsum(w[order])
        edge = max(float(p), 0.0) * c[-1]
        n = int(np.searchsorted(c, edge, side="left")) + 1  # the first part that holds the edge
        n = max(1, min(n + moved, len(order)))
        if not flat(order) and p > 0 and not moved:
            margin = np.abs(c - edge).min() / c[-1]
            if margin <= 2.0 ** -33 and len({sample(given, inv_t, k, p, m, u, i)[0] for i in (-2, -1, 1, 2)}) == 1:
                margin = np.inf
        order = order[:n]
    if m > 0:
        with np.errstate(divide="ignore"):
            order = order[z[order] >= np.log(min(float(m), 1.0))]
    kept = np.zeros(V)
    kept[order] = w[order]
    c = np.cumsum(kept)
    edge = float(u) * c[-1]
    token = int(np.searchsorted(c, edge, side="right"))
    if not flat(order) and u > 0:
        margin = min(margin, np.abs(c - edge).min() / c[-1])
    return token, z[token] - np.log(w.sum()), z[token] - np.log(c[-1]), margin


def sample_rows(z, inv_t, k, p, m, u):
    return [np.array(v) for v in zip(*(sample(z[t], inv_t[t], k[t], p[t], m[t], u[t]) for t in range(len(z))))]


def filters(rng, T, kind):
    """Per-row filters of a kind, as float32 / int32 vectors."""
    f32 = np.float32
    inv_t = (1 / rng.choice([0.5, 0.8, 1.0, 1.7], T)).astype(f32)
    k, p, m = np.zeros(T, np.int32), np.ones(T, f32), np.zeros(T, f32)
    if "k" in kind:
        k = rng.choice([1, 2, 7, 50, 333, 20000], T).astype(np.int32)
    if "p" in kind:
        p = rng.choice([0.1, 0.5, 0.9, 0.95, 0.999], T).astype(f32)
    if "m" in kind:
        m = rng.choice([1e-6, 0.01, 0.1, 1.0], T).astype(f32)
    return inv_t, k, p, m, rng.random(T).astype(f32)
