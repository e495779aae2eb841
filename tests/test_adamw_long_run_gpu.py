"""What rounding the root of v at random makes of v itself over many steps (states in 8 bits): the figures that the header states.

Written r for the root before the rounding, lo and hi for the codes around it, gap = hi - lo, the step keeps E[root] = r, so
E[v'] = r² + (hi - r)(r - lo). With r moved by d from the code it came from, that gain is at most (gap - d)·d within one code's distance and gap²/4
beyond, while |g² - v|·(1 - beta2) = d·(r + r0): the ratio is at most gap/(2·r0), which is 1/16 for normal numbers and 1/(2k) at
code k below them."""
import numpy as np
import pytest
import torch

import bwd_situ_glu_gb300 as sg
import _fp8_ref as ref8

pytestmark = pytest.mark.gpu

DEV = "cuda"


def roots(plan):
    return ref8.values(plan._lists["v"][0][None], plan._lists["v_scales"][0][None], 1)[0]


def code_of(k):
    """The k-th number from 0, in steps of 2^-9."""
    return float(ref8.code_values(torch.tensor([k], dtype=torch.uint8))[0])


@pytest.mark.parametrize("beta2", [0.95, 0.99])
@pytest.mark.parametrize("live", [1.0, 0.1])
def test_mean_of_v_of_independent_gradients(beta2, live):
    """Normal gradients, in every step or in one of ten: v's mean lies above that of exact states of the same gradients, by at most the
    mean of |g² - v| / 16, and for gradients in every step by more than 1 %. (The mean of 32768 elements, each off by a standard
    deviation below 0.5 of v, is good to 5·0.5/181 = 1.4 % in one step; over the second half, 4/(1 - beta2) steps of a memory of
    1/(1 - beta2), to 0.7 %.)"""
    n, steps = 32768, round(8 / (1 - beta2))
    gen = torch.Generator(device=DEV).manual_seed(round(1000 * beta2 + 10 * live))
    w = torch.zeros(n, device=DEV)
    plan = sg.AdamWPlan([w], **sg.adamw_state([w], "fp8"))
    exact = torch.zeros(n, dtype=torch.float64, device=DEV)
    mean = torch.zeros(3, dtype=torch.float64, device=DEV)       # stored, exact, |g² - v|
    for k in range(1, steps + 1):
        g = 0.01 * torch.randn(n, generator=gen, device=DEV) * (torch.rand(n, generator=gen, device=DEV) < live)
        square = g.double().square()
        if k > steps // 2:
            mean[2] += (square - roots(plan).square()).abs().mean()
        plan.step([g], sg.adam_params(lr=0.0, beta1=0.9, beta2=beta2, step=k))
        exact = beta2 * exact + (1 - beta2) * square
        if k > steps // 2:
            mean[:2] += torch.stack([roots(plan).square().mean(), exact.mean()])
    stored, want, distance = mean.tolist()
    gain = stored / want - 1
    assert -0.007 <= gain <= distance / want / 16 + 0.007
    if live == 1.0:
        assert gain > 0.01


@pytest.mark.parametrize("k", [1, 2, 3, 7, 8, 9, 15, 60, 100])
def test_gain_of_one_step_without_a_gradient(k):
    """Roots at the k-th code, in blocks whose first element holds the scale: E[v'] as the rounding's rule says, above beta2·v by at most
    (1 - beta2)·v / 16, or / 2k below the normal numbers; at code 1 v stays what it is."""
    blocks, beta2 = 4096, 0.95
    n = 128 * blocks
    w = torch.zeros(n, device=DEV)
    state = sg.adamw_state([w], "fp8")
    state["v"][0].fill_(k)
    state["v"][0][::128] = 0x78                                      # 256
    state["v_scales"][0].fill_(127)
    g = torch.zeros(n, device=DEV)
    g[::128] = 256.0
    plan = sg.AdamWPlan([w], **state)
    plan.step([g], sg.adam_params(lr=0.0, beta2=beta2, step=1))
    assert (state["v_scales"][0] == 127).all()
    got = roots(plan).view(-1, 128)[:, 1:].square()
    root, v = code_of(k), code_of(k) ** 2
    # the step's own fp32 numbers: root² and beta2 are fp32, so is their product's root
    r = float(np.sqrt(np.float32(beta2) * (np.float32(root) * np.float32(root))))
    down = max(j for j in range(k + 1) if code_of(j) <= r)
    lo, hi = code_of(down), code_of(down + 1)
    p = (r - lo) / (hi - lo)
    want = lo * lo + p * (hi * hi - lo * lo) if down else hi * hi    # a root above 0 is not rounded to 0
    spread = (hi * hi - lo * lo) * (p * (1 - p)) ** 0.5 if down else 0.0
    assert abs(got.mean().item() - want) <= 5 * spread / got.numel() ** 0.5 + (hi * hi - lo * lo) * 2.0 ** -16
    bound = (1 - beta2) * v / (16 if k >= 8 else 2 * k)
    assert 0 <= want - beta2 * v + 1e-6 * v <= (bound if k > 1 else (1 - beta2) * v) + 2e-6 * v
    if k == 1:
        assert (got == v).all()


def test_small_elements_of_a_block_stop_at_code_one():
    """Beside one large element: roots of elements whose gradient has ended fall to code 1 of the block's scale and no further, gradients
    below it give code 1, elements that never had one stay 0."""
    blocks = 64
    n = 128 * blocks
    gen = torch.Generator(device=DEV).manual_seed(5)
    root = torch.rand(n, generator=gen, device=DEV)
    root[::128], root[1::128], root[2::128] = 1.0, 0.0, 0.0
    codes, scales = sg.situ_quant_fp8(root[None])
    w = torch.zeros(n, device=DEV)
    state = sg.adamw_state([w], "fp8")
    state["v"][0].copy_(codes[0])
    state["v_scales"][0].copy_(scales[0])
    g = torch.zeros(n, device=DEV)
    g[::128], g[1::128] = 1.0, 2.0 ** -21                             # code 1 is 2^-17 or 2^-18
    plan = sg.AdamWPlan([w], **state)
    never = torch.arange(n, device=DEV) % 128 == 2
    for k in range(1, 1201):                                         # 0.95^600 of a root of 1 is 4e-14
        plan.step([g], sg.adam_params(lr=0.0, beta2=0.95, step=k))
        if k % 100 == 0:
            assert ((state["v"][0] == 0) == never).all()
    rest = torch.arange(n, device=DEV) % 128 > 0
    assert (state["v"][0][rest & ~never] == 1).all()
    largest = roots(plan).view(-1, 128)[:, 0]
    floor = roots(plan).view(-1, 128)[:, 3]
    assert (floor >= 2.0 ** -9 / 448 * largest).all() and (floor <= 2.0 ** -9 / 224 * largest).all()
