"""Refusals of kda_lin_* and kda_pages_* that guard memory and results (no GPU needed): sizes that the kernels' indices
could not hold, and outputs over other arguments.  Pointers are made up; nothing is launched."""
import ctypes

import pytest

import kda_linear_attention_02_b200 as kda
from kda_linear_attention_02_b200 import build as kbuild

vp = ctypes.c_void_p
ARG = -1
TOO_MANY = [(1 << 30) + 1, (1 << 31) - 4096, (1 << 31) - 1]


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda._load()


@pytest.mark.parametrize("n", TOO_MANY)
def test_lists_and_pools_that_wrap_an_index_are_refused(lib, n):
    a, b, c, d, e, f, ws = (vp(i << 40) for i in range(1, 8))
    most = (1 << 31) - 1
    assert lib.kda_pages_copy(a, most, b, most, c, d, n, 16, None) == ARG
    assert lib.kda_pages_copy(a, most, b, most, None, d, n, 16, None) == ARG
    assert lib.kda_pages_fork(a, 1, n, 16, b, c, d, 4, 3, e, f, None, None, 2, 0, ws, 1 << 40, None) == ARG
    assert lib.kda_pages_compact(a, 1, n, 16, b, c, d, 4, 3, e, None, ws, 1 << 40, None) == ARG
    assert lib.kda_pages_compact_workspace_bytes(n) == 0 < lib.kda_pages_compact_workspace_bytes(1 << 30)
    assert lib.kda_pages_free(a, n, b, c, 4, 3, d, 2, None) == ARG
    assert lib.kda_pages_free(a, 8, b, c, 4, 3, d, n, None) == ARG
    assert lib.kda_lin_recurrent_step(a, 8, b, 1, c, c, d, e, 1, n, 1, 1, 64, 64, 0, f, None) == ARG
