"""Sizes at the end of the learner operators' int."""
import pytest

import nvfp4_w4a4_moe_top_gb300 as M


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from nvfp4_w4a4_moe_top_gb300 import build
    build.build()


@pytest.mark.parametrize("d", [16, 128, 1024, 2048, 4096, 8192, 16384])
def test_workspace_of_the_most_rows(d):
    """As many blocks as for any number of rows that fills them."""
    for T in [2 ** 31 - 20, 2 ** 31 - 2, 2 ** 31 - 1]:
        assert M.add_rmsnorm_backward_workspace_bytes(T, d) == M.add_rmsnorm_backward_workspace_bytes(2 ** 30, d)
