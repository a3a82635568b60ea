"""The draw of a token against its definition in 64 bits.

The token has to be the definition's; the inputs (seeded) are such that no
decision of a row lies within 2^-33 of its border, a few thousand times the
64-bit sums' own error.  Log-probabilities: (x - m) inv_t is rounded three
times, 2^-23 of it, and so is the logarithm of the sum, whose FP32 weights are
off by less than 2^-18: 2^-22 (|z| + ln sum) + 2^-18."""
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


def draw(z, dtype, inv_t, k, p, m, u, pad=0, lead=0, status=None):
    """The library's tokens and log-probabilities for host rows z."""
    import torch
    T = len(z)
    f = lambda a, t: None if a is None else torch.from_numpy(np.ascontiguousarray(a, t)).cuda()  # noqa: E731
    tokens = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    lp, kept = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    M.moe_sample_tokens(LR.device_rows(z, dtype, pad, lead), f(u, np.float32), tokens, f(inv_t, np.float32),
                        f(k, np.int32), f(p, np.float32), f(m, np.float32), lp, kept, status)
    return tokens.cpu().numpy(), lp.cpu().numpy().astype(np.float64), kept.cpu().numpy().astype(np.float64)


def check(z, dtype, inv_t, k, p, m, u, pad=0, lead=0):
    T = len(z)
    got = draw(z, dtype, inv_t, k, p, m, u, pad, lead)
    one = lambda a, v: np.full(T, v) if a is None else a  # noqa: E731
    want = R.sample_rows(z, one(inv_t, 1.0), one(k, 0), one(p, 1.0), one(m, 0.0), u)
    assert (want[3] > 2.0 ** -33).all(), "a decision of these inputs lies on its border"
    assert np.array_equal(got[0], want[0]), np.nonzero(got[0] != want[0])
    zt = np.abs(want[1]) + 2 * np.log(z.shape[1] + 1)  # |z| + ln sum, from above
    for g, w in [(got[1], want[1]), (got[2], want[2])]:
        same = np.isneginf(w) | np.isnan(w)
        assert np.array_equal(g[same], w[same], equal_nan=True)
        assert (np.abs(g[~same] - w[~same]) <= (2.0 ** -22 * zt + 2.0 ** -18)[~same]).all()


SIZES = [(3, 1), (4, 2), (9, 7), (8, 33), (12, 257), (16, 1000), (9, 4097), (8, 16384), (12, 50001), (7, 131072)]
FILTERS = ["", "k", "p", "m", "kp", "km", "pm", "kpm"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", SIZES)
def test_rows(T, V, dtype):
    """All filters on peaked rows, among them those that masks make special."""
    rng = np.random.default_rng(V + (dtype == "f32"))
    for i, kind in enumerate(FILTERS):
        z = LR.logit_rows(rng, T, V, dtype, ties=i % 3 == 2)
        check(z, dtype, *R.filters(rng, T, kind), pad=[0, 3, 5][i % 3], lead=[0, 1, 3][(i + 1) % 3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", FILTERS)
def test_flat_rows(kind, dtype):
    """Rows whose weight lies in tens of thousands of ids, and rows of a few
    values each shared by thousands."""
    rng = np.random.default_rng(len(kind) + 10 * (dtype == "f32"))
    T, V = 10, 70001
    z = LR.round_to(rng.standard_normal((T, V)) * rng.choice([0.3, 1.0, 2.5], (T, 1)), dtype)
    z[5:8] = LR.round_to(rng.integers(-3, 4, (3, V)) * 0.75, dtype)
    z[8] = LR.round_to(-5 - rng.random(V) * 3, dtype)  # below zero throughout
    z[9, rng.random(V) < 0.9] = -np.inf
    check(z, dtype, *R.filters(rng, T, kind))


@pytest.mark.parametrize("V", [1, 6, 1000, 40000])
def test_uniform_rows(V):
    """Equal logits: sums are exact, every border is met exactly."""
    T = 8
    u = np.array([0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 2.0 ** -24, 0.125, 0.375], np.float32)
    for value in [0.0, -3.389531389251535e38, 7.5]:
        z = LR.round_to(np.full((T, V), value), "bf16")
        z[3] = -0.0 if value == 0 else value
        z[3, ::2] = value
        check(z, "bf16", None, None, None, None, u)
        check(z, "bf16", None, np.full(T, 3), None, None, u)
        check(z, "bf16", None, None, np.full(T, 0.5), None, u)
        check(z, "bf16", np.full(T, 1e6), np.full(T, V), np.full(T, 0.25), np.ones(T), u)


def test_numbers_at_their_limits():
    """top_k, top_p, min_p and u at and beyond their ranges, extreme
    temperatures."""
    rng = np.random.default_rng(5)
    T, V = 16, 3001
    z = LR.round_to(rng.standard_normal((T, V)) * 3, "f32")
    u = rng.random(T).astype(np.float32)
    u[0], u[1] = 0, 1 - 2.0 ** -24
    inf = np.inf
    for inv_t, k, p, m in [(1.0, -5, 1.0, 0.0), (1.0, V, 1.5, -1.0), (1.0, V - 1, 1.0, 0.0), (1.0, 2 ** 31 - 1, inf, -inf),
                           (1.0, 0, 0.0, 0.0), (1.0, 0, -inf, 0.0), (1.0, 0, 1e-30, 0.0), (1.0, 0, 1 - 2.0 ** -24, 0.0),
                           (1.0, 0, 1.0, 1.0), (1.0, 0, 1.0, inf), (1.0, 0, 1.0, 1e-38), (1e-6, 0, 1.0, 0.0),
                           (1e6, 0, 1.0, 0.0), (1e-6, 0, 0.7, 0.0), (1e6, 5, 0.7, 0.5), (1e-6, 0, 1.0, 0.999)]:
        check(z, "f32", np.full(T, inv_t, np.float32), np.full(T, k), np.full(T, p, np.float32), np.full(T, m, np.float32), u)


def test_bad_rows():
    """NaN, +inf and bad parameters: token -1, NaN, a status bit; the other rows
    as without them."""
    import torch
    rng = np.random.default_rng(6)
    T, V = 12, 2000
    z = LR.round_to(rng.standard_normal((T, V)) * 3, "f32")
    z[1, 77], z[2, V - 1], z[3, 0] = np.nan, np.inf, -np.nan
    z[4, 5], z[4, 6] = np.inf, np.nan
    inv_t, k, p, m, u = R.filters(rng, T, "kpm")
    for change, bit, rows in [({}, M.STATUS_NONFINITE_LOGITS, [1, 2, 3, 4]),
                              (dict(u=[(6, 1.0), (7, -1e-9), (8, np.nan)]), None, [6, 7, 8]),
                              (dict(inv_t=[(6, 0.0), (7, np.inf), (8, np.nan), (9, -1.0), (10, 2e6), (11, 9e-7)]), None,
                               [6, 7, 8, 9, 10, 11]),
                              (dict(p=[(6, np.nan)], m=[(7, np.nan)]), None, [6, 7])]:
        a = dict(inv_t=inv_t.copy(), k=k, p=p.copy(), m=m.copy(), u=u.copy())
        for name, sets in change.items():
            for t, v in sets:
                a[name][t] = v
        y = z if bit else np.where(np.isfinite(z), z, 0.0).astype(np.float32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tokens, lp, kept = draw(y, "f32", status=status, **a)
        assert int(status.item()) == (bit or M.STATUS_BAD_SAMPLING)
        assert (tokens[rows] == -1).all() and np.isnan(lp[rows]).all() and np.isnan(kept[rows]).all()
        rest = [t for t in range(T) if t not in rows]
        want = R.sample_rows(y[rest], *(a[n][rest] for n in ["inv_t", "k", "p", "m", "u"]))
        assert np.array_equal(tokens[rest], want[0])


def test_masked_ids_are_never_drawn():
    """-inf and the type's lowest value, at u = 0 and close to 1."""
    rng = np.random.default_rng(8)
    T, V = 8, 5000
    for mask in [-np.inf, LR.LOWEST["bf16"]]:
        z = LR.round_to(rng.standard_normal((T, V)), "bf16")
        z[:, :1000] = mask
        z[:, 4000:] = mask
        u = np.array([0, 1 - 2.0 ** -24, 0.5, 1e-30, 0, 1 - 2.0 ** -24, 0.3, 0.9], np.float32)
        for k, p, m in [(0, 1.0, 0.0), (4500, 1.0, 0.0), (0, 1 - 2.0 ** -24, 0.0), (0, 1.0, 1e-30)]:
            tokens, lp, _ = draw(z, "bf16", None, np.full(T, k), np.full(T, p), np.full(T, m), u)
            assert ((tokens >= 1000) & (tokens < 4000)).all() and np.isfinite(lp).all()
            assert (tokens[[0, 3, 4]] == 1000).all() or k or p < 1 or m


def test_frequencies():
    """One row drawn at the middles of 2^16 equal parts of [0, 1): each id as
    often as its probability says, to one draw at each of its two ends."""
    import torch
    rng = np.random.default_rng(9)
    V, n = 300, 1 << 16
    z = LR.round_to(rng.standard_normal((1, V)) * 2, "bf16")
    logits = LR.device_rows(z, "bf16").expand(n, V).contiguous()
    u = ((torch.arange(n, device="cuda", dtype=torch.float64) + 0.5) / n).float()
    tokens = torch.empty(n, dtype=torch.int32, device="cuda")
    M.moe_sample_tokens(logits, u, tokens)
    p = np.exp(z[0].astype(np.float64))
    p /= p.sum()
    assert (np.abs(np.bincount(tokens.cpu().numpy(), minlength=V) - p * n) <= 1 + 1e-6 * n * p).all()
    assert (tokens[1:] >= tokens[:-1]).all()


@pytest.mark.parametrize("V,dtype", [(1 << 20, "bf16"), ((1 << 20) - 3, "f32")])
def test_longest_rows(V, dtype):
    rng = np.random.default_rng(10)
    z = LR.logit_rows(rng, 3, V, dtype)
    z[2] = LR.round_to(rng.standard_normal(V) * 0.1, dtype)
    for kind in ["", "kp", "pm"]:
        check(z, dtype, *R.filters(rng, 3, kind))


def test_agrees_with_token_logprobs():
    """The log-probability is the one that the learner's operator gives for the
    drawn token."""
    import torch
    rng = np.random.default_rng(11)
    T, V = 50, 20011
    z = LR.device_rows(LR.round_to(rng.standard_normal((T, V)) * 3, "bf16"), "bf16")
    u = torch.rand(T, device="cuda")
    tokens, lp, again = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    inv = torch.full((T,), 1.25, device="cuda")
    M.moe_sample_tokens(z, u, tokens, inv, top_p=torch.full((T,), 0.9, device="cuda"), logprob=lp)
    M.moe_token_logprobs(z, tokens, 1.25, 0, again, None, None)
    assert ((lp - again).abs() <= 2.0 ** -17 + 2.0 ** -21 * lp.abs()).all()
