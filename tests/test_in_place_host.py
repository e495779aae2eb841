"""What the bindings of the 8-bit operators and of AdamW tell autograd of tensors that their kernels write, and when a plan takes a
tensor for what it was: without a GPU, the library replaced by one that notes its calls."""
import pytest
import torch

import bwd_situ_glu_gb300 as sg

BF, U8 = torch.bfloat16, torch.uint8


class Library:
    """Every entry point returns `status` and is noted by name."""

    def __init__(self):
        self.called, self.status = [], 0

    def __getattr__(self, name):
        def call(*args):
            self.called.append(name)
            return self.status
        return call


def need(t, dtype, shape, name):
    """The package's check, of tensors on any device."""
    if t.dtype != dtype:
        raise TypeError(name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    for module in (sg.fp8, sg.adamw):
        monkeypatch.setattr(module, "_lib", lambda: lib)
        monkeypatch.setattr(module, "_raw_stream", lambda device: 0)
        monkeypatch.setattr(module, "_device_now", lambda: None)

    def check(status):
        if status:
            raise sg.SituGluError(status, "refused")
    monkeypatch.setattr(sg.fp8, "_check", check)
    monkeypatch.setattr(sg.adamw, "_check", check)
    monkeypatch.setattr(sg.fp8, "_shape3", lambda x, name: x.shape if x.dim() == 3 else (1, *x.shape))
    monkeypatch.setattr(sg.fp8, "_two", lambda x, name: x.shape)
    monkeypatch.setattr(sg, "_need", need)
    return lib


class Host:
    """The host as a plan's device: its index is what get_device says of a tensor there."""
    index = -1

    def __eq__(self, other):
        return other == torch.device("cpu")


def plan_of(params, work=None, state="fp8"):
    plan = sg.AdamWPlan(params, work=work, **sg.adamw_state(params, state))
    plan._device = Host()
    return plan


@pytest.fixture
def step(monkeypatch):
    monkeypatch.setattr(sg.adamw, "_device_now", lambda: -1)
    return lambda plan, **kw: plan.step([torch.ones(p.shape) for p in plan._params], sg.adam_params(step=1), **kw)


def versions(*tensors):
    return [t._version for t in tensors]


# ---------------------------------------------------------------- autograd's record of what was written

def test_given_outputs_count_as_written(library):
    x, codes, scales = torch.zeros(4, 128, dtype=BF), torch.zeros(4, 128, dtype=U8), torch.ones(4, 1, dtype=U8)
    out, y, w = torch.zeros(4, 128, dtype=BF), torch.zeros(4, 16, dtype=BF), (torch.zeros(16, 128, dtype=U8), torch.ones(1, 1, dtype=U8))
    every = (x, codes, scales, out, y, *w)

    def moved(call):
        before = versions(*every)
        call()
        return [after > b for after, b in zip(versions(*every), before)]
    assert moved(lambda: sg.situ_quant_fp8(x, codes=codes, scales=scales)) == [False, True, True, False, False, False, False]
    assert moved(lambda: sg.situ_quant_fp8(x, scales=scales)) == [False, False, True, False, False, False, False]
    assert moved(lambda: sg.situ_quant_fp8(x)) == [False] * 7
    assert moved(lambda: sg.situ_dequant_fp8(codes, scales, out=out)) == [False, False, False, True, False, False, False]
    assert moved(lambda: sg.situ_linear_fp8((codes, scales), w, out=y)) == [False, False, False, False, True, False, False]
    library.status = 2                                   # refused: nothing was written
    for call in (lambda: sg.situ_quant_fp8(x, codes=codes, scales=scales), lambda: sg.situ_dequant_fp8(codes, scales, out=out),
                 lambda: sg.situ_linear_fp8((codes, scales), w, out=y)):
        before = versions(*every)
        with pytest.raises(sg.SituGluError):
            call()
        assert versions(*every) == before


def test_a_step_counts_as_written(library, step):
    params = [torch.nn.Parameter(torch.zeros(3, 5)), torch.zeros(7)]
    work = [p.detach().to(BF) for p in params]
    plan = plan_of(params, work)
    before = versions(*params, *work)
    step(plan)
    assert all(after > b for after, b in zip(versions(*params, *work), before))
    before, library.status = versions(*params, *work), 1
    with pytest.raises(sg.SituGluError):
        step(plan)
    assert versions(*params, *work) == before


def test_a_stepped_weight_fails_its_backward(library, step):
    """A torch product keeps the master, which the step between its forward and its backward writes."""
    w, x = torch.nn.Parameter(torch.ones(4, 4)), torch.ones(2, 4, requires_grad=True)
    plan = plan_of([w])
    y = (x @ w).sum()
    step(plan)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_requantised_codes_fail_their_backward(library):
    a = torch.zeros(4, 16, dtype=BF, requires_grad=True)
    w = torch.nn.Parameter(torch.zeros(32, 16))
    wq = sg.situ_quant_fp8(w.detach(), block_rows=128)
    for part in (dict(codes=wq[0]), dict(scales=wq[1])):
        y = sg.fp8.linear_fp8(a, w, wq=wq)
        sg.situ_quant_fp8(w.detach(), block_rows=128, **part)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.float().sum().backward()


@pytest.mark.parametrize("act", ["none", "silu"])
def test_masters_may_be_stepped_before_the_backward(library, step, act):
    """linear_fp8's gradients are of the codes: its masters' values are not among what the backward reads."""
    a = torch.zeros(4, 16, dtype=BF, requires_grad=True)
    w, bias = torch.nn.Parameter(torch.zeros(32, 16)), torch.nn.Parameter(torch.zeros(32))
    plan = plan_of([w, bias])
    sg.fp8._autograd()
    made = []
    y = sg.fp8.linear_fp8(a, w, bias, act=act)
    step(plan)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(sg.fp8, "situ_linear_fp8_bwd", lambda *args, **kw: made.append(1) or (torch.zeros(4, 16, dtype=BF), torch.zeros(32, 16), torch.zeros(32)))
        y.float().sum().backward()
    assert made and all(t.grad is not None for t in (a, w, bias))


def test_a_bias_may_be_stepped_before_the_backward_of_linear(library, step, monkeypatch):
    """The bf16 operator does not read the bias again either."""
    a, w = torch.zeros(4, 16, dtype=BF, requires_grad=True), torch.zeros(32, 16, dtype=BF)
    bias = torch.nn.Parameter(torch.zeros(32))
    out = torch.zeros(4, 32, dtype=BF)
    monkeypatch.setattr(sg.moe, "situ_linear", lambda *args, save_pre=False, **kw: (out.clone(), out.clone()) if save_pre else out.clone())
    monkeypatch.setattr(sg.moe, "situ_linear_bwd", lambda *args, **kw: (torch.zeros(4, 16, dtype=BF), None, torch.zeros(32)))
    y = sg.moe.linear(a, w, bias, act="silu")
    step(plan_of([bias]))
    y.float().sum().backward()
    assert bias.grad is not None


# ---------------------------------------------------------------- a plan's tensors changed under it

def test_transposed_data_at_the_same_place(library, step):
    """A square parameter, or working copy, whose .data became its transpose begins where it did, and pairs with other gradients."""
    for which in ("params", "work"):
        p = [torch.zeros(2, 2), torch.zeros(3, 3)]
        plan = plan_of(p, [t.to(BF) for t in p])
        t = plan._lists[which][1]
        t.data = t.data.t()
        with pytest.raises(ValueError, match="contiguous"):
            step(plan)
        t.data = t.data.t()
        step(plan)
        assert library.called.count("situ_adamw_step") == 1
        library.called.clear()


@pytest.mark.parametrize("which", ["params", "work"])
def test_smaller_data_at_the_same_place(library, step, which):
    """As where the old memory was released and came back for a smaller tensor: a step would write past its end."""
    p = [torch.zeros(300), torch.zeros(40)]
    plan = plan_of(p, [t.to(BF) for t in p])
    t = plan._lists[which][0]
    at = t.data_ptr()
    t.data = t.data[:200]
    assert t.data_ptr() == at
    with pytest.raises(ValueError):
        plan.step([torch.ones(300), torch.ones(40)], sg.adam_params(step=1))
    assert "situ_adamw_step" not in library.called


@pytest.mark.parametrize("state", ["fp32", "fp8"])
def test_the_states_memory_is_the_plans(library, step, state):
    """States are not looked at but for their place: their memory stays, whatever becomes of the tensors that were given."""
    p = [torch.zeros(100000)]
    plan = plan_of(p, state=state)
    for name in set(plan._lists) - {"params"}:
        t = plan._lists[name][0]
        n, storage = t.untyped_storage().nbytes(), t.untyped_storage()._cdata
        t.data = t.data[:1]                              # the same place
        assert any(k.untyped_storage()._cdata == storage and k.untyped_storage().nbytes() == n for k in plan._kept)
    step(plan)


# ---------------------------------------------------------------- weights that the backward has no gradient for

def test_a_type_without_weight_gradients_is_refused_before_any_kernel(library):
    dout, a = torch.zeros(4, 32, dtype=BF), (torch.zeros(4, 16, dtype=U8), torch.ones(4, 1, dtype=U8))
    w = torch.zeros(32, 16, dtype=U8), torch.ones(1, 1, dtype=U8)
    for dtype in (torch.float16, torch.float64, U8):
        with pytest.raises(TypeError, match="dw_dtype"):
            sg.situ_linear_fp8_bwd(dout, a, w, dw_dtype=dtype)
        assert not library.called
    assert sg.situ_linear_fp8_bwd(dout, None, w, dw_dtype=torch.float16, need_dw=False)[1] is None
    # through autograd: the forward reads the given codes alone, and is fine with any weight
    x, master = torch.zeros(4, 16, dtype=BF, requires_grad=True), torch.zeros(32, 16, dtype=torch.float16, requires_grad=True)
    y = sg.fp8.linear_fp8(x, master, wq=w)
    library.called.clear()
    with pytest.raises(TypeError, match="dw_dtype"):
        y.backward(dout)
    assert not library.called
