"""The expert layer's binding and argument checks, without a GPU."""
import os
import subprocess
import sys

import pytest
import torch

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


# ---------------------------------------------------------------- which kernels the autograd operators call


@pytest.fixture
def calls(monkeypatch):
    """The kernels' bindings replaced by ones that note their call and return tensors of the right shape."""
    made = []

    def linear(a, w, expert_offsets=None, bias=None, residual=None, act="none", save_pre=False, **kw):
        made.append(("linear", dict(save_pre=save_pre, **kw)))
        out = torch.zeros(a.shape[0], w.shape[-2], dtype=torch.bfloat16)
        return (out, out.clone()) if save_pre else out

    def linear_bwd(dout, a, w, expert_offsets=None, act="none", pre=None, dw_dtype=None, bias=True, need_da=True, need_dw=True, **kw):
        made.append(("linear_bwd", dict(pre=pre is not None, bias=bias, need_da=need_da, need_dw=need_dw, **kw)))
        return (torch.zeros_like(a) if need_da else None, torch.zeros_like(w) if need_dw else None,
                torch.zeros(w.shape[:-1]) if bias else None)

    def combine(o, row_of, weights=None, residual=None, **kw):
        made.append(("combine", {}))
        return torch.zeros(row_of.shape[0], o.shape[1], dtype=o.dtype)

    def combine_bwd(dy, o, row_of, weights, expert_offsets, **kw):
        made.append(("combine_bwd", {}))
        return torch.zeros_like(o), torch.zeros(row_of.shape)

    for name, f in dict(situ_linear=linear, situ_linear_bwd=linear_bwd, situ_combine=combine, situ_combine_bwd=combine_bwd).items():
        monkeypatch.setattr(sg.moe, name, f)
    return made


def linear_inputs(*needed):
    ts = [torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(8),
          torch.zeros(4, 8, dtype=torch.bfloat16)]
    return [t.requires_grad_(i in needed) for i, t in enumerate(ts)]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_linear_without_grad_keeps_nothing(calls, mode):
    """Weights that require gradients, but no grad mode: the value before the activation is not written."""
    ts = linear_inputs(1, 2)
    with mode():
        out = sg.moe.linear(*ts, act="silu")
    assert not out.requires_grad and len(calls) == 1 and calls[0][1]["save_pre"] is False


def test_linear_with_grad_keeps_what_it_needs(calls):
    for needed, act, pre in (((1,), "silu", True), ((3,), "silu", False), ((0, 1, 2), "none", False)):
        calls.clear()
        sg.moe.linear(*linear_inputs(*needed), act=act).sum().backward()
        assert calls[0][0] == "linear" and calls[0][1]["save_pre"] is pre
        assert [c[0] for c in calls[1:]] == (["linear_bwd"] if needed != (3,) else [])


@pytest.mark.parametrize("needed,launches", [((2,), 0), ((0,), 1), ((1,), 1), ((0, 1, 2), 1)])
def test_combine_backward_launches(calls, needed, launches):
    """The residual's gradient is dy itself: no pass over the rows for it alone."""
    o, w, res = (t.requires_grad_(i in needed) for i, t in enumerate((torch.zeros(8, 16), torch.zeros(4, 2), torch.zeros(4, 16))))
    row_of, off = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    dy = torch.rand(4, 16)
    sg.moe.moe_combine(o, w, row_of, off, residual=res).backward(dy)
    assert [c[0] for c in calls] == ["combine"] + ["combine_bwd"] * launches
    assert [t.grad is not None for t in (o, w, res)] == [i in needed for i in range(3)]
    if 2 in needed:
        assert torch.equal(res.grad, dy)


def test_linear_status_reaches_every_kernel(calls):
    """A timed-out wait is reported through the status word, in the forward and in the backward."""
    status = torch.zeros(1, dtype=torch.int32)
    sg.moe.linear(*linear_inputs(0, 1, 2, 3), act="gelu", status=status).sum().backward()
    assert [c[0] for c in calls] == ["linear", "linear_bwd"] and all(c[1]["status"] is status for c in calls)
