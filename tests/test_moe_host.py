"""The expert layer's binding and argument checks, without a GPU."""
import os
import subprocess
import sys

import pytest

import bwd_situ_glu_gb300 as sg

A, B, C, D = (k << 40 for k in range(1, 5))   # pointers that a refused call never reads
INVALID = 1
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def without_torch(code):
    """Standard output of the code in a process in which torch cannot be imported."""
    run = subprocess.run([sys.executable, "-c", "import sys; sys.modules['torch'] = None\n" + code], cwd=ROOT, capture_output=True,
                         text=True, timeout=120)
    assert run.returncode == 0, run.stderr[-2000:]
    return run.stdout


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


def test_loads_without_torch(lib):
    """The library and its pointer entry points need ctypes alone."""
    out = without_torch("import bwd_situ_glu_gb300 as sg\n"
                        "lib = sg.load()\n"
                        "print(sg.version(), sg.status_string(1), lib.situ_route_topk(0, 0, 0, 0, 0, 0, 0, 0))\n"
                        "try: sg.situ_glu_fwd_ptr(0, 0, -1, 8)\n"
                        "except sg.SituGluError as e: print(e.status)")
    assert out.split() == [str(sg.version()), *sg.status_string(1).split(), "1", "1"]


def test_star_import_without_torch():
    assert without_torch("from bwd_situ_glu_gb300 import *\nprint(situ_glu_fwd_ptr.__name__, 'situ_linear' in globals())").split() == [
        "situ_glu_fwd_ptr", "False"]


def test_star_import():
    names = {}
    exec("from bwd_situ_glu_gb300 import *", names)
    assert names["situ_linear"] is sg.situ_linear and names["moe"] is sg.moe and names["situ_glu_fwd"] is sg.situ_glu_fwd
