"""The expert layer's binding and argument checks, without a GPU."""
import pytest

import bwd_situ_glu_gb300 as sg

A, B, C, D = (k << 40 for k in range(1, 5))   # pointers that a refused call never reads
INVALID = 1


@pytest.fixture(scope="module")
def lib():
    sg.build()
    return sg.load()


@pytest.mark.parametrize("rows", [2 ** 31 - 1024, 2 ** 31 - 1])
def test_linear_row_limit(lib, rows):
    """Rounded-up row numbers are 32-bit too: the largest row counts are refused."""
    assert lib.situ_linear_fwd(A, B, 0, 1, 0, 0, 0, C, 0, 0, 0, rows, 8, 8, 0) == INVALID
    assert lib.situ_linear_dgrad(A, B, 0, 1, C, 0, rows, 8, 8, 0) == INVALID
    assert lib.situ_linear_wgrad(A, B, 0, 1, C, 1, D, 1 << 40, 0, rows, 8, 8, 0) == INVALID
    assert lib.situ_linear_act_bwd(A, 0, 0, 0, 1, 0, B, C, 1 << 40, rows, 8, 0) == INVALID
    assert lib.situ_linear_act_bwd_workspace(rows, 8, 1) == lib.situ_linear_wgrad_workspace(rows, 8, 8, 1) == 0
    assert lib.situ_linear_act_bwd_workspace(2 ** 31 - 1025, 8, 1) > 0
