"""What the kernels of the 8-bit operators and of AdamW write in place, as autograd sees it, and plans whose tensors changed under them."""
import pytest
import torch

import bwd_situ_glu_gb300 as sg

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def randn(*s, seed=0, dtype=torch.float32):
    return torch.randn(*s, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dtype)


# ---------------------------------------------------------------- autograd's record of what was written

def test_requantised_codes_fail_their_backward():
    """Refilled between a forward and its backward, in part or through another stream, the given codes are no longer the forward's."""
    a, w = randn(5, 48, dtype=BF).requires_grad_(), torch.nn.Parameter(randn(32, 48, seed=1))
    wq = sg.situ_quant_fp8(w.detach(), block_rows=128)
    for part in (dict(codes=wq[0]), dict(scales=wq[1]), dict(codes=wq[0], stream=torch.cuda.current_stream())):
        y = sg.fp8.linear_fp8(a, w, wq=wq)
        sg.situ_quant_fp8(w.detach(), block_rows=128, **part)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.float().sum().backward()
    sg.fp8.linear_fp8(a, w, wq=wq).float().sum().backward()
    assert a.grad is not None


@pytest.mark.parametrize("state", ["fp32", "fp8"])
def test_a_stepped_working_copy_fails_its_backward(state):
    """The bf16 product keeps the working copy that the step between its forward and its backward writes."""
    master = [randn(32, 48)]
    work = [t.to(BF).requires_grad_() for t in master]
    plan = sg.AdamWPlan(master, work=work, **sg.adamw_state(master, state))
    a = randn(5, 48, seed=1, dtype=BF).requires_grad_()
    y = sg.moe.linear(a, work[0]).float().sum()
    plan.step([randn(32, 48, seed=2)], sg.adam_params(step=1))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    sg.moe.linear(a, work[0]).float().sum().backward()
    assert work[0].grad is not None


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_masters_stepped_before_the_backward_change_no_gradient(act):
    """linear_fp8's gradients are of the codes and the rows that the forward kept."""
    a, dout = randn(5, 48, dtype=BF), randn(5, 32, seed=3, dtype=BF)
    grads = []
    for stepped in (False, True):
        ts = [a.clone().requires_grad_(), torch.nn.Parameter(randn(32, 48, seed=1)), torch.nn.Parameter(randn(32, seed=2))]
        plan = sg.AdamWPlan(ts[1:], **sg.adamw_state(ts[1:]))
        y = sg.fp8.linear_fp8(*ts, act=act)
        if stepped:
            plan.step([torch.ones_like(t) for t in ts[1:]], sg.adam_params(lr=1.0, step=1))
        y.backward(dout)
        grads.append([t.grad for t in ts])
    assert all(torch.equal(x, y) for x, y in zip(*grads))


def test_tensors_of_inference_mode():
    """They have no record of writes: a step and given outputs take them as before."""
    with torch.inference_mode():
        w, x = [randn(300)], randn(4, 128)
        plan = sg.AdamWPlan(w, **sg.adamw_state(w))
        plan.step([randn(300, seed=1)], sg.adam_params(step=1))
        codes, scales = sg.situ_quant_fp8(x)
        sg.situ_quant_fp8(x, codes=codes, scales=scales)
    plan.step([randn(300, seed=1)], sg.adam_params(step=2))
    assert torch.equal(sg.situ_dequant_fp8(codes, scales, out=torch.empty(4, 128, device=DEV)), sg.situ_dequant_fp8(codes, scales, dtype=torch.float32))


# ---------------------------------------------------------------- a plan's tensors changed under it

def test_data_at_the_same_place():
    """A transposed square, a narrower view and memory that came back for a smaller tensor begin where the plan's tensor did: all are
    refused, and nothing is written."""
    p = [torch.zeros(64, 64, device=DEV), torch.zeros(2 ** 22, device=DEV)]
    work = [t.to(BF) for t in p]
    plan = sg.AdamWPlan(p, work=work, **sg.adamw_state(p))
    g, hp = [torch.ones_like(t) for t in p], sg.adam_params(step=1)
    for t in (p[0], work[0]):
        t.data = t.data.t()
        with pytest.raises(ValueError, match="contiguous"):
            plan.step(g, hp)
        t.data = t.data.t()
    for t in (p[1], work[1]):
        whole = t.data
        t.data = whole[:1000]
        with pytest.raises(ValueError, match="shape"):
            plan.step(g, hp)
        t.data = whole
    assert not any(t.any() for t in (*p, *work))
    plan.step(g, hp)
    assert all((t != 0).all() for t in (*p, *work))


@pytest.mark.parametrize("name", ["m", "v", "m_scales", "v_scales"])
def test_states_given_up_by_the_program_stay_the_plans(name):
    """A state whose tensor shrank in its place: the plan goes on with the memory that it was made with."""
    plans = []
    for shrink in (False, True):
        p = [torch.zeros(5000, device=DEV)]
        state = sg.adamw_state(p)
        plan = sg.AdamWPlan(p, **state)
        for k in (1, 2):
            if shrink and k == 2:
                state[name][0].data = state[name][0].data[:10]
            plan.step([randn(5000, seed=k)], sg.adam_params(step=k))
        plans.append((p[0], *plan._kept))
    assert all(torch.equal(a, b) for a, b in zip(*plans))
