"""The widest rows that the losses over a vocabulary take, on the CPU.

A tile of logits is one sum over all of a row, 64 values at a step, and what
waits for it gives up after 4e9 clocks.  A step takes 512 clocks at the tensor
cores' rate, and 1,400 where its 64 KB for each of 76 pairs come from memory: rows
of 10^9 values cannot be awaited, rows of 2^25 take at most 7.4e8 clocks."""
import ctypes

import pytest

from optimizer_state_gb300 import build as z3build
from optimizer_state_gb300 import z3

WIDEST = 1 << 25


@pytest.fixture(scope="module")
def lib():
    z3build.build()
    return z3.load()


@pytest.mark.parametrize("k,grads", [(0, 0), (0, 1), (5, 0), (5, 1)])
@pytest.mark.parametrize("tokens", [1, 300])
def test_the_widest_rows(lib, k, grads, tokens):
    n = ctypes.c_int64(-1)
    assert lib.z3_head_workspace_bytes(tokens, WIDEST, 10, k, grads, ctypes.byref(n)) == z3.Z3_OK
    assert n.value > 0
    n.value = -1
    for dim in (WIDEST + 8, 10 ** 9, 2 ** 31 - 1024):
        st = lib.z3_head_workspace_bytes(tokens, dim, 10, k, grads, ctypes.byref(n))
        assert (st, n.value) == (z3.Z3_ERR_OVERFLOW, -1)
        assert "the sizes do not fit" in z3.last_error()


def test_a_row_of_the_widest_is_awaited():
    clocks_a_step, steps = 1400, WIDEST // 64
    assert clocks_a_step * steps < 4_000_000_000 / 5
    assert 512 * (10 ** 9 // 64) > 4_000_000_000        # what was taken before was not
