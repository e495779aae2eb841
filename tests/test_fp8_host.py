"""What the bindings of the 8-bit operators and of AdamW do without a GPU: lazy modules, refusals, which kernels the autograd
operator calls and what it keeps."""
import pytest
import torch

import bwd_situ_glu_gb300 as sg

BF = torch.bfloat16


def test_names_of_the_package():
    names = {}
    exec("from bwd_situ_glu_gb300 import *", names)
    assert names["situ_quant_fp8"] is sg.fp8.situ_quant_fp8 and names["AdamWPlan"] is sg.adamw.AdamWPlan
    assert names["fp8"] is sg.fp8 and names["adamw"] is sg.adamw
    with pytest.raises(AttributeError):
        sg.situ_no_such_operator


def test_refusals_without_a_gpu():
    x = torch.zeros(4, 128, dtype=BF)
    codes, scales = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8)
    for call, error in ((lambda: sg.situ_quant_fp8(x), ValueError), (lambda: sg.situ_quant_fp8([1.0]), TypeError),
                        (lambda: sg.situ_quant_fp8(x.half()), TypeError), (lambda: sg.situ_dequant_fp8(codes, scales), ValueError),
                        (lambda: sg.fp8._scale_shape((4, 128), 3), ValueError), (lambda: sg.fp8._pair(x, "w"), TypeError),
                        (lambda: sg.fp8._pair((x, None), "w"), TypeError), (lambda: sg.situ_linear_fp8(x, (codes, scales)), ValueError),
                        (lambda: sg.AdamWPlan([x.float()], [x.float()], [x.float()]), ValueError), (lambda: sg.adamw_state([x], "fp16"), ValueError),
                        (lambda: sg.adamw_coefficients(sg.adam_params(), out=torch.zeros(9)), ValueError),
                        (lambda: sg.fp8.linear_fp8(x.float(), x), TypeError), (lambda: sg.fp8.linear_fp8(x, x, wq=(codes[:2], scales)), ValueError)):
        with pytest.raises(error):
            call()


def test_scale_shapes():
    shape = sg.fp8._scale_shape
    assert shape((4, 128), 1) == (4, 1) and shape((4, 129), 1) == (4, 2) and shape((4, 1), 128) == (1, 1)
    assert shape((3, 129, 256), 128) == (3, 2, 2) and shape((3, 0, 7), 1) == (3, 0, 1)


def test_states():
    params = [torch.zeros(3, 100), torch.zeros(0)]
    s = sg.adamw_state(params, "fp8")
    assert [t.shape for t in s["m"]] == [p.shape for p in params] and all(t.dtype == torch.uint8 for ts in s.values() for t in ts)
    assert [t.numel() for t in s["m_scales"]] == [3, 0]
    s = sg.adamw_state(params, "fp32")
    assert set(s) == {"m", "v"} and all(t.dtype == torch.float32 and not t.any() for ts in s.values() for t in ts)


@pytest.fixture
def calls(monkeypatch):
    """The kernels' bindings replaced by ones that note their call and return tensors of the right shape."""
    made = []

    def quant(x, block_rows=1, **kw):
        made.append(("quant", block_rows))
        return torch.zeros(x.shape, dtype=torch.uint8), torch.ones(sg.fp8._scale_shape(tuple(x.shape), block_rows), dtype=torch.uint8)

    def linear(a, w, expert_offsets=None, bias=None, residual=None, act="none", save_pre=False, **kw):
        made.append(("linear", dict(save_pre=save_pre, w=w, **kw)))
        out = torch.zeros(a[0].shape[0], w[0].shape[-2], dtype=BF)
        return (out, out.clone()) if save_pre else out

    def linear_bwd(dout, a, w, expert_offsets=None, act="none", pre=None, dw_dtype=None, bias=True, need_da=True, need_dw=True, **kw):
        made.append(("linear_bwd", dict(pre=pre is not None, a=a is not None, bias=bias, need_da=need_da, need_dw=need_dw, dw_dtype=dw_dtype, w=w, **kw)))
        return (torch.zeros(dout.shape[0], w[0].shape[-1], dtype=BF) if need_da else None, torch.zeros(w[0].shape, dtype=dw_dtype) if need_dw else None,
                torch.zeros(w[0].shape[:-1]) if bias else None)

    for name, f in dict(situ_quant_fp8=quant, situ_linear_fp8=linear, situ_linear_fp8_bwd=linear_bwd).items():
        monkeypatch.setattr(sg.fp8, name, f)
    return made


def inputs(*needed, dtype=BF):
    ts = [torch.zeros(4, 16, dtype=BF), torch.zeros(32, 16, dtype=dtype), torch.zeros(32), torch.zeros(4, 32, dtype=BF)]
    return [t.requires_grad_(i in needed) for i, t in enumerate(ts)]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_without_grad_mode_nothing_is_kept(calls, mode):
    ts = inputs(0, 1, 2)
    with mode():
        out = sg.fp8.linear_fp8(*ts, act="gelu")
    assert not out.requires_grad and [c[0] for c in calls] == ["quant", "quant", "linear"] and calls[2][1]["save_pre"] is False


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("needed", [(0,), (1,), (2,), (3,), (0, 1), (0, 1, 2, 3)])
def test_what_the_backward_asks_for(calls, needed, act, dtype):
    ts = inputs(*needed, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32)
    sg.fp8.linear_fp8(*ts, act=act, status=status).sum().backward()
    assert calls[2][1]["save_pre"] is (act != "none" and needed != (3,)) and calls[2][1]["status"] is status
    if needed == (3,):
        assert len(calls) == 3
    else:
        asked = calls[3][1]
        assert len(calls) == 4 and asked["status"] is status and asked["dw_dtype"] is dtype
        assert (asked["need_da"], asked["need_dw"], asked["bias"]) == tuple(i in needed for i in range(3))
        assert asked["pre"] is (act != "none") and asked["a"] is (1 in needed)
    assert [t.grad is not None for t in ts] == [i in needed for i in range(4)]
    assert all(t.grad is None or t.grad.dtype == t.dtype for t in ts)


def test_given_codes_are_used_as_they_are(calls):
    ts = inputs(0, 1)
    wq = torch.full((32, 16), 3, dtype=torch.uint8), torch.ones(1, 1, dtype=torch.uint8)
    sg.fp8.linear_fp8(*ts, wq=wq).sum().backward()
    assert [c[0] for c in calls] == ["quant", "linear", "linear_bwd"] and calls[1][1]["w"] is wq
    assert all(torch.equal(x, y) for x, y in zip(calls[2][1]["w"], wq))


@pytest.mark.parametrize("needed,act", [((0, 1), "none"), ((0, 1), "gelu"), ((0,), "gelu"), ((1,), "none"), ((0, 2), "silu")])
def test_a_second_derivative_raises(calls, needed, act):
    """Whatever of the inputs a gradient depends on (without an activation a's is constant where w is)."""
    ts = inputs(*needed)
    first = ts[needed[0]]
    (g,) = torch.autograd.grad(sg.fp8.linear_fp8(*ts, act=act).float().sum(), first, create_graph=True)
    with pytest.raises(RuntimeError, match="not\\s+differentiable"):
        (g.float() * first.float()).sum().backward()


def test_the_rows_themselves_are_not_kept(calls):
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t.dtype) or t, lambda t: t):
        out = sg.fp8.linear_fp8(*inputs(0, 1, 2, dtype=torch.float32), act="silu")
    assert out.requires_grad and kept.count(BF) == 1         # the value before the activation
