"""The draw at the numbers of rows between its launch plans: a cluster per row with
one and with two blocks per SM, one block per SM, open rows of which each cluster
takes one, or all; against the definition in 64 bits.  Tolerances as in
test_gpu_sample.py."""
import numpy as np
import pytest

import learner_ref as LR
import tokens_ref as R
from test_gpu_sample import check, draw
from test_gpu_sample_many import mixed_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


def ends(rng, z, dtype):
    """Among them rows whose maximum is negative, a zero of either sign, or tiny."""
    V = z.shape[1]
    z[0] = -np.abs(rng.standard_normal(V)) - 0.25
    z[1] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    z[2] = np.where(rng.random(V) < 0.5, -0.0, -rng.random(V))
    z[3] = rng.standard_normal(V) * 1e-30
    return LR.round_to(z, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,flat", [(15, 1.0), (16, 0.5), (17, 1.0), (31, 0.2), (35, 1.0), (36, 0.5), (37, 1.0), (70, 1.0),
                                    (151, 0.1), (152, 0.02), (153, 0.3)])
def test_numbers_of_rows(T, flat, dtype):
    rng = np.random.default_rng(100 * T + (dtype == "f32"))
    V = 9001 if T > 64 else 20013
    for i, kind in enumerate(["", "p", "kp", "m", "kpm"]):
        if T > 64 and i % 2 != (dtype == "f32"):
            continue
        z = ends(rng, mixed_rows(rng, T, V, dtype, flat), dtype)
        check(z, dtype, *R.filters(rng, T, kind), pad=[0, 3][i % 2], lead=[0, 1, 5][i % 3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [[4999], [0, 4096, 4999], [100, 4095, 4097, 4500]])
def test_open_rows_far_apart(at, dtype):
    """Few open rows among more than one look at the tokens finds."""
    rng = np.random.default_rng(len(at) + (dtype == "f32"))
    T, V = 5000, 8200
    z = np.full((T, V), -50.0)
    z[np.arange(T), rng.integers(0, V, T)] = 3.0
    z[at] = rng.standard_normal((len(at), V))
    z = LR.round_to(z, dtype)
    args = R.filters(rng, T, "p")
    tokens, lp, kept = draw(z, dtype, *args)
    part = draw(z[at], dtype, *(a[at] for a in args))
    assert np.array_equal(tokens[at], part[0])
    peaked = np.setdiff1d(np.arange(T), at)
    assert np.array_equal(tokens[peaked], z[peaked].argmax(1))
    check(z[at], dtype, *(a[at] for a in args))


FIRST = """
import torch
import nvfp4_w4a4_moe_top_gb300 as M
g = torch.Generator(device="cuda").manual_seed(3)
calls = []
for T in [3, 20, 60, 400]:
    z = (torch.randn((T, 9001), generator=g, device="cuda") * 2).bfloat16()
    u = torch.rand(T, generator=g, device="cuda")
    p = torch.full((T,), 0.9, device="cuda")
    calls.append((z, u, p, torch.full((T,), -7, dtype=torch.int32, device="cuda")))
torch.cuda.synchronize()
graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(graph, stream=s):
    for z, u, p, tokens in calls:
        M.moe_sample_tokens(z, u, tokens, top_p=p)
graph.replay()
torch.cuda.synchronize()
for z, u, p, tokens in calls:
    again = torch.empty_like(tokens)
    M.moe_sample_tokens(z, u, again, top_p=p)
    assert torch.equal(again, tokens) and (tokens >= 0).all()
"""


def test_first_calls_of_a_process_in_a_capture():
    """What a call asks the device for the first time, it may ask while a graph is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr
