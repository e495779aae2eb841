"""AdamW over many tensors on the GPU, states in fp32 and in 8 bits.

With states in fp32 every stored value is one stated sequence of single IEEE fp32 operations: numpy's gives the same bits. So it does
with states in 8 bits, whose rounding at random is a stated function of the seed and the element's place. The tests against
64 bits count roundings: 2^-24 each, relative."""
import ctypes
import threading
import time

import numpy as np
import pytest
import torch

import bwd_situ_glu_gb300 as sg
import _fp8_ref as ref8

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16
F = np.float32
HP = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


# ---------------------------------------------------------------- the definition, in single fp32 operations

def mix(x):
    x = x.astype(np.uint32)
    x ^= x >> np.uint32(16)
    x *= np.uint32(0x9E3779B1)
    x ^= x >> np.uint32(15)
    x *= np.uint32(0x6A09E667)
    return x ^ (x >> np.uint32(16))


def random_bits(n, seed):
    with np.errstate(over="ignore"):
        key = mix(np.array([seed * 0x9E3779B1 % 2 ** 32], dtype=np.uint32))[0]
        return mix((np.arange(n, dtype=np.uint64) % 2 ** 32).astype(np.uint32) + key)


def scale_bytes(x):
    """[blocks of 128] of flat fp32 x, by frexp."""
    n = -(-x.size // 128) * 128
    p = np.zeros(n, dtype=np.float64)
    p[:x.size] = np.where(np.isfinite(x), np.abs(x), 0)
    frac, e = np.frexp(p.reshape(-1, 128).max(1) / 448.0)
    e = np.where(frac == 0.5, e - 1, e)
    return np.where(frac == 0, -126, np.maximum(e, -126)) + 127


def e4m3_at_random(x, u16, least):
    """Codes of flat fp32 x: of the two around a value the upper with the probability of its place, in 2^-16; scale bytes."""
    b = scale_bytes(x)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.abs(x).astype(np.float64) * np.exp2(127.0 - np.repeat(b, 128)[:x.size])
        fine = np.isfinite(y)
        y = np.where(fine, y, 0.0)
        _, e = np.frexp(y)
        step = np.exp2(np.maximum(e - 1, -6) - 3.0)
        y = np.minimum(np.floor(y / step + u16 / 65536.0) * step, 448.0)
        _, e = np.frexp(y)
        e = np.maximum(e - 1, -7)
        code = np.where((e < -6) | (y == 0), y * 512, (e + 7) * 8 + (y / np.exp2(np.maximum(e, -6)) - 1) * 8).astype(np.int64)
        code = np.where(least & (x > 0) & (code == 0), 1, code)
        return np.where(fine, code, 0x7F) + np.where(x < 0, 128, 0), b


def constants(hp):
    b1, b2, t = hp.beta1, hp.beta2, hp.step
    return tuple(F(v) for v in (b1, b2, 1 - b1, 1 - b2, hp.lr / (1 - b1 ** t), 1 / np.sqrt(1 - b2 ** t), hp.eps, 1 - hp.lr * hp.weight_decay))


def one_step(w, g, m, v, hp, gs=None, ms=None, vs=None, seed=None):
    """Flat fp32 arrays (m, v as codes with scales where those are given) -> the new w, m, v, ms, vs."""
    b1, b2, c1, c2, s, r, eps, d = constants(hp)
    with np.errstate(all="ignore"):
        if gs is not None:
            g = g * F(gs)
        if ms is not None:
            def value(codes, b):
                x = ref8.code_values(torch.from_numpy(codes)).numpy() * np.exp2(np.repeat(b.astype(np.float64), 128)[:codes.size] - 127)
                return x.astype(F)
            m, root = value(m, ms), value(v, vs)
            v = root * root
        w = w * d if hp.weight_decay > 0 else w
        m = b1 * m + c1 * g
        v = b2 * v + c2 * (g * g)
        root = np.sqrt(v)
        w = w - s * (m / (root * r + eps))
        if ms is None:
            return w, m, v, None, None
        u = random_bits(w.size, seed)
        m, ms = e4m3_at_random(m, u & np.uint32(0xFFFF), False)
        v, vs = e4m3_at_random(root, u >> np.uint32(16), True)
        return w, m, v, ms, vs


# ---------------------------------------------------------------- inputs

def make(sizes, state, grad=torch.float32, work=True, seed=0, offset=0):
    """Lists of tensors; offset: elements that each begins past an allocation's start."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def place(x):
        if not offset:
            return x.clone()
        flat = torch.empty(x.numel() + offset, dtype=x.dtype, device=DEV)
        flat[offset:] = x
        return flat[offset:]
    randn = lambda n, scale: torch.randn(n, generator=g, device=DEV) * scale  # noqa: E731
    t = dict(params=[place(randn(n, 0.02)) for n in sizes], grads=[])
    for n in sizes:
        x = randn(n, 1e-3) * (torch.rand(n, generator=g, device=DEV) > 0.1)
        x[:n // 3] *= (torch.rand((n // 3 + 127) // 128, generator=g, device=DEV) > 0.3).repeat_interleave(128)[:n // 3]
        t["grads"].append(place(x.to(grad)))
    m, root = [randn(n, 3e-4) for n in sizes], [randn(n, 5e-4).abs() for n in sizes]
    if state == "fp8":
        flat = lambda xs: zip(*(sg.situ_quant_fp8(x[None]) if x.numel() else (x[None].to(torch.uint8),) * 2 for x in xs))  # noqa: E731
        (mc, ms), (vc, vs) = flat(m), flat(root)
        t.update(m=[place(c[0]) for c in mc], v=[place(c[0]) for c in vc], m_scales=[s[0].clone() for s in ms], v_scales=[s[0].clone() for s in vs])
    else:
        t.update(m=[place(x) for x in m], v=[place(x * x) for x in root])
    if work:
        t["work"] = [place(torch.zeros(n, dtype=BF, device=DEV)) for n in sizes]
    return t


def plan_of(t):
    return sg.AdamWPlan(**{k: x for k, x in t.items() if k != "grads"})


def host(x):
    return x.float().cpu().numpy() if x.dtype == BF else x.cpu().numpy()


def expected(t, hp, gs=None, seed=None):
    """The tensors after the step, as lists of arrays."""
    out = {k: [] for k in t if k != "grads"}
    for i, p in enumerate(t["params"]):
        eight = "m_scales" in t
        w, m, v, ms, vs = one_step(host(p).ravel(), host(t["grads"][i]).ravel(), host(t["m"][i]).ravel(), host(t["v"][i]).ravel(), hp, gs,
                                   host(t["m_scales"][i]) if eight else None, host(t["v_scales"][i]) if eight else None, seed)
        out["params"].append(w)
        out["m"].append(m)
        out["v"].append(v)
        if eight:
            out["m_scales"].append(ms)
            out["v_scales"].append(vs)
        if "work" in t:
            out["work"].append(torch.from_numpy(w).to(BF).float().numpy())
    return out


def same(t, want):
    for name, xs in want.items():
        for i, x in enumerate(xs):
            got = host(t[name][i]).ravel()
            assert np.array_equal(got.astype(x.dtype), x, equal_nan=x.dtype.kind == "f"), f"{name}[{i}]"


SIZES = [[1], [7, 128, 129], [0, 5, 0], [8192, 8193, 100000, 127], [2048 * 4 + 8, 16, 3], [1] * 500, [130] * 97]


# ---------------------------------------------------------------- tests

@pytest.mark.parametrize("state", ["fp32", "fp8"])
@pytest.mark.parametrize("grad", [torch.float32, BF])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_bits(sizes, grad, state):
    """Every stored value, over three steps, with and without a factor on the gradients and working copies."""
    for work, scale in ((True, None), (False, 0.37)):
        t = make(sizes, state, grad, work)
        plan = plan_of(t)
        gs = None if scale is None else torch.tensor([scale], device=DEV)
        for k in (1, 2, 1000):
            hp = sg.adam_params(step=k, **HP)
            want = expected(t, hp, scale, seed=k)
            plan.step(t["grads"], hp, grad_scale=gs)
            same(t, want)


@pytest.mark.parametrize("state", ["fp32", "fp8"])
@pytest.mark.parametrize("offset", [1, 3, 8])
def test_bases_off_the_vectors(state, offset):
    t = make([5, 129, 9001], state, BF, offset=offset)
    hp = sg.adam_params(step=3, **HP)
    want = expected(t, hp, seed=11)
    plan_of(t).step(t["grads"], hp, seed=11)
    same(t, want)


@pytest.mark.parametrize("state", ["fp32", "fp8"])
def test_against_64_bits(state):
    """From the same states: m1 within 3 roundings of its terms, v1 within 4, w2 within those of its update (12 in all of
    s·m/q) and two of w. 2^-24 each; the constants bring one more a factor."""
    t = make([50000], state)
    hp = sg.adam_params(step=7, **HP)
    w, g = (host(t[k][0]).astype(np.float64) for k in ("params", "grads"))
    if state == "fp8":
        m = ref8.values(t["m"][0][None], t["m_scales"][0][None], 1)[0].cpu().numpy()
        v = ref8.values(t["v"][0][None], t["v_scales"][0][None], 1)[0].cpu().numpy() ** 2
    else:
        m, v = (host(t[k][0]).astype(np.float64) for k in ("m", "v"))
    plan_of(t).step(t["grads"], hp)
    m1 = hp.beta1 * m + (1 - hp.beta1) * g
    v1 = hp.beta2 * v + (1 - hp.beta2) * g * g
    mag = np.abs(hp.beta1 * m) + np.abs((1 - hp.beta1) * g)
    q = np.sqrt(v1 / (1 - hp.beta2 ** 7)) + hp.eps
    s = hp.lr / (1 - hp.beta1 ** 7)
    u = 2.0 ** -24
    tol = s * mag / q * 14 * u + 4 * np.abs(w) * u
    assert (np.abs(host(t["params"][0]) - (w * (1 - hp.lr * hp.weight_decay) - s * m1 / q)) <= tol).all()
    if state == "fp32":
        assert (np.abs(host(t["m"][0]) - m1) <= 4 * mag * u).all()
        assert (np.abs(host(t["v"][0]) - v1) <= 6 * v1 * u).all()
    else:     # one of the two codes around the value: less than a step away, 2^-3 of it or 2^-9 of the scale
        for name, x in (("m", m1), ("v", np.sqrt(v1))):
            got = ref8.values(t[name][0][None], t[name + "_scales"][0][None], 1)[0].cpu().numpy()
            sc = np.exp2(np.repeat(host(t[name + "_scales"][0]).astype(np.float64), 128)[:x.size] - 127)
            assert (np.abs(got - x) <= np.maximum(np.abs(x) / 8, sc / 512) * (1 + 1e-6)).all(), name


def test_rounding_at_random_keeps_the_mean():
    """The same states and gradients under 4096 seeds: the mean of a moment's code is its value to 5 standard errors, a step
    being at most 1/8 of it. And two seeds, or m and v, do not round alike."""
    n, seeds = 256, 4096
    t = make([n], "fp8", work=False, seed=4)
    hp = sg.adam_params(step=50, **{**HP, "lr": 0.0, "weight_decay": 0.0})
    m = ref8.values(t["m"][0][None], t["m_scales"][0][None], 1)[0]
    v = ref8.values(t["v"][0][None], t["v_scales"][0][None], 1)[0].square()
    g = t["grads"][0].double()
    want = dict(m=hp.beta1 * m + (1 - hp.beta1) * g, v=(hp.beta2 * v + (1 - hp.beta2) * g * g).sqrt())
    total, ups = {k: torch.zeros(n, dtype=torch.float64, device=DEV) for k in want}, {k: [] for k in want}
    for seed in range(seeds):
        u = {k: [x.clone() for x in xs] for k, xs in t.items()}
        plan_of(u).step(u["grads"], hp, seed=seed)
        for k in want:
            got = ref8.values(u[k][0][None], u[k + "_scales"][0][None], 1)[0]
            total[k] += got
            if seed < 64:
                ups[k].append((got > want[k]).double())
    for k, x in want.items():
        sc = torch.exp2(t[k + "_scales"][0].double().repeat_interleave(128)[:n] - 126)
        gap = torch.maximum(x.abs() / 8, sc / 512)
        # a code's standard deviation is at most half the gap; 2^-16 of it the granularity; codes of 0 are lifted in v
        tol = gap * (5 * 0.5 / seeds ** 0.5 + 2.0 ** -16) + (sc / 512 * (x < sc / 512) if k == "v" else 0)
        assert ((total[k] / seeds - x).abs() <= tol).all(), k
    a, b = torch.stack(ups["m"]), torch.stack(ups["v"])
    live = (a.mean(0) > 0.1) & (a.mean(0) < 0.9) & (b.mean(0) > 0.1) & (b.mean(0) < 0.9)
    a, b = a[:, live] - a[:, live].mean(0), b[:, live] - b[:, live].mean(0)
    assert live.sum() > 50
    # correlations of 64 draws: below 5 / sqrt(64 · places) on average over the places
    corr = lambda x, y: ((x * y).mean(0) / (x.square().mean(0) * y.square().mean(0)).sqrt()).mean().abs()  # noqa: E731
    assert corr(a, b) < 5 / (64 * int(live.sum())) ** 0.5
    assert corr(a[:-1], a[1:]) < 5 / (63 * int(live.sum())) ** 0.5 + 1 / 63
    assert corr(a[:, :-1], a[:, 1:]) < 5 / (64 * int(live.sum())) ** 0.5


def test_a_small_change_of_a_moment_is_not_lost():
    """v of a steady gradient, from 0: after many steps sqrt(v) is near the gradient's size, though a step moves it by far less
    than a code's distance (rounded to nearest it would stop there)."""
    n = 4096
    w = torch.zeros(n, device=DEV)
    g = torch.full((n,), 0.01, device=DEV)
    s = sg.adamw_state([w], "fp8")
    plan = sg.AdamWPlan([w], **s)
    steps = 400
    for k in range(1, steps + 1):
        plan.step([g], sg.adam_params(lr=0.0, beta1=0.9, beta2=0.99, step=k))
    v = ref8.values(s["v"][0][None], s["v_scales"][0][None], 1)[0].square()
    # The root r keeps its mean; r² then gains (hi - r)(r - lo), at most gap·|r - its last code|: with gap <= r/8 and a move of
    # (c2/2)·|g²/v - 1|·r a step that is (c2/16)·|g² - v|, against the pull c2·(g² - v): in the long run at most 1/16 of
    # the mean |v - g²|. The variance of v gains 4r² times as much a step and loses 2·c2 of itself, so that mean is at most g²/8:
    # less than 1 % off, and 1 % for the scatter of 4096 elements (5 standard errors of 1/8).
    assert abs(v.mean().item() / (1e-4 * (1 - 0.99 ** steps)) - 1) < 0.03


def test_values_that_are_not_finite():
    t = make([300], "fp32")
    t["grads"][0][5], t["grads"][0][200] = float("nan"), float("inf")
    hp = sg.adam_params(step=2, **HP)
    want = expected(t, hp)
    plan_of(t).step(t["grads"], hp)
    same(t, want)
    t = make([300], "fp8")
    t["grads"][0][5], t["grads"][0][200] = float("nan"), float("-inf")
    want = expected(t, hp, seed=2)
    plan_of(t).step(t["grads"], hp)
    same(t, want)
    assert torch.isnan(t["params"][0]).sum() == 2 and (t["v"][0][[5, 200]] == 0x7F).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-19, 1e18, 1e30])
def test_extreme_gradients(scale):
    """Squares that leave fp32 on either side, scales at their ends."""
    for state in ("fp32", "fp8"):
        t = make([1000], state)
        t["grads"][0] *= scale * 1e3
        hp = sg.adam_params(step=2, **HP)
        want = expected(t, hp, seed=2)
        plan_of(t).step(t["grads"], hp)
        same(t, want)


def test_zero_states_and_first_step():
    """The first step from zero: m/(sqrt(v)·r) is the gradient's sign, so w moves by lr; in 8 bits as in fp32."""
    for state in ("fp32", "fp8"):
        w = [torch.zeros(5, 77, device=DEV), torch.zeros(1000, device=DEV)]
        g = [torch.randn_like(x) for x in w]
        sg.AdamWPlan(w, **sg.adamw_state(w, state)).step(g, sg.adam_params(lr=0.01, step=1))
        for x, y in zip(w, g):
            # four factors of at most two roundings each, and eps against the smallest gradient of some 1e-4
            assert torch.allclose(x, -0.01 * torch.sign(y), rtol=1e-3, atol=0)


def test_split_over_calls_order_and_shared_gradients():
    t = make([3000, 3000, 77], "fp8", seed=8)
    t["grads"][1] = t["grads"][0]                       # one gradient of two tensors
    u = {k: [x.clone() for x in xs] for k, xs in t.items()}
    hp = sg.adam_params(step=4, **HP)
    plan_of(t).step(t["grads"], hp)
    for i in (2, 0, 1):
        sg.situ_adamw_step(*([u[k][i]] for k in ("params", "grads", "m", "v")), hp, [u["m_scales"][i]], [u["v_scales"][i]], [u["work"][i]])
    for k in t:
        for a, b in zip(t[k], u[k]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("state", ["fp32", "fp8"])
def test_captured_with_its_coefficients_on_the_device(state):
    t, u = make([5000, 33], state, seed=2), make([5000, 33], state, seed=2)
    coef = sg.adamw_coefficients(sg.adam_params(step=1, **HP)).to(DEV)
    a, b = plan_of(t), plan_of(u)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(t["grads"], coef)
    for k in range(1, 5):
        hp = sg.adam_params(step=k, **HP)
        coef.copy_(sg.adamw_coefficients(hp))
        graph.replay()
        b.step(u["grads"], hp)
    for k in t:
        for x, y in zip(t[k], u[k]):
            assert torch.equal(x, y), k


def test_another_stream_and_replaced_data():
    t, u = make([70000], "fp8", seed=3), make([70000], "fp8", seed=3)
    hp = sg.adam_params(step=9, **HP)
    plan_of(u).step(u["grads"], hp)
    plan = plan_of(t)
    t["params"][0].data = t["params"][0].data.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan.step(t["grads"], hp, stream=s)
    s.synchronize()
    assert torch.equal(t["params"][0], u["params"][0]) and torch.equal(t["m"][0], u["m"][0])
    t["work"][0].data = torch.zeros_like(t["work"][0])
    for x, y in ((t, plan), (u, plan_of(u))):
        y.step(x["grads"], sg.adam_params(step=10, **HP))
    assert torch.equal(t["work"][0], u["work"][0])
    t["v"][0].data = t["v"][0].data.clone()
    with pytest.raises(ValueError):
        plan.step(t["grads"], hp)
    t["params"][0].data = t["params"][0].data[:69999].clone()
    with pytest.raises(ValueError):
        plan.step(t["grads"], hp)


def test_steps_of_one_plan_from_two_threads(monkeypatch):
    """The library reads a step's own gradients, however long it takes, while another thread steps the same plan."""
    params = [torch.ones(64, device=DEV) for _ in range(3)]
    plan = sg.AdamWPlan(params, **sg.adamw_state(params, "fp32"))
    hp, seen, failed = sg.adam_params(step=1, **HP), [], []
    grads = [[torch.full((64,), f, device=DEV) for _ in params] for f in (1.0, -3.0)]

    class Slow:
        def situ_adamw_step(self, table, count, *rest):
            words = (ctypes.c_int64 * (8 * count)).from_address(table)
            first = list(words)[1::8]
            time.sleep(0.05)                             # without Python's lock, as the library's own call
            seen.append((first, list(words)[1::8]))
            return 0
    monkeypatch.setattr(sg.adamw, "_lib", Slow)
    start = threading.Barrier(2)

    def run(gs):
        try:
            start.wait(60)
            plan.step(gs, hp)
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=run, args=(gs,)) for gs in grads]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    own = [[g.data_ptr() for g in gs] for gs in grads]
    assert sorted(seen) == sorted((at, at) for at in own)


def test_elements_past_32_bits():
    """One tensor of 2^32 + 200 elements: indices repeat modulo 2^32, its ends are those of small tensors."""
    n = 2 ** 32 + 200
    w, g = torch.zeros(n, device=DEV), torch.zeros(n, dtype=BF, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.ones(-(-n // 128), dtype=torch.uint8, device=DEV) for _ in range(2))
    t = make([200], "fp32", BF, work=False)
    g[:200] = t["grads"][0]
    g[2 ** 32:] = t["grads"][0]
    hp = sg.adam_params(step=1, **{**HP, "weight_decay": 0.0})
    sg.situ_adamw_step([w], [g], [m], [v], hp, [ms], [vs])
    for x in (w, m, v):
        assert x[:200].any() and torch.equal(x[:200], x[2 ** 32:])
    assert torch.equal(ms[:2], ms[-2:]) and not w[200:2 ** 20].any() and not m[2 ** 31:2 ** 31 + 10000].any()


def test_refusals():
    t = make([300, 20], "fp8")
    hp = sg.adam_params(step=1)
    plan, x = plan_of(t), torch.zeros(300, device=DEV)
    for call, error in ((lambda: plan.step(t["grads"][:1], hp), ValueError), (lambda: plan.step([x, x], hp), ValueError),
                        (lambda: plan.step([x, t["grads"][1].to(BF)], hp), TypeError), (lambda: plan.step([x.half(), x], hp), TypeError),
                        (lambda: plan.step(t["grads"], 3), TypeError), (lambda: plan.step([x.cpu(), x], hp), ValueError),
                        (lambda: plan.step(t["grads"], hp, grad_scale=torch.ones(2, device=DEV)), ValueError),
                        (lambda: plan.step(t["grads"], sg.adamw_coefficients(hp)), ValueError),
                        (lambda: plan.step(t["grads"], sg.adamw_coefficients(hp).to(DEV), seed=3), ValueError),
                        (lambda: sg.AdamWPlan([x], [x.clone()], [x.clone()], [x.to(torch.uint8)]), ValueError),
                        (lambda: sg.AdamWPlan([x.to(BF)], [x.clone()], [x.clone()]), TypeError),
                        (lambda: sg.AdamWPlan([x], [x[:5]], [x.clone()]), ValueError),
                        (lambda: sg.AdamWPlan([x], [x.clone()], []), ValueError), (lambda: sg.adamw_state([x], "int8"), ValueError)):
        with pytest.raises(error):
            call()
    before = {k: [y.clone() for y in ys] for k, ys in t.items()}
    for change, status in ((dict(params=[t["params"][0]] * 2, grads=[t["grads"][0]] * 2, m=[t["m"][0], t["m"][0].clone()], v=[t["v"][0], t["v"][0].clone()],
                                 m_scales=[t["m_scales"][0]] * 2, v_scales=[t["v_scales"][0]] * 2), 2),
                           (dict(grads=[t["params"][0], t["grads"][1]]), 2)):
        u = {**{k: y for k, y in t.items() if k != "work"}, **change}
        with pytest.raises(sg.SituGluError) as e:
            plan_of(u).step(u["grads"], hp)
        assert e.value.status == status
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(weight_decay=-1.0), dict(step=0)):
        with pytest.raises(sg.SituGluError) as e:
            plan.step(t["grads"], sg.adam_params(**bad))
        assert e.value.status == 1
    for k in t:
        for a, b in zip(t[k], before[k]):
            assert torch.equal(a, b)
    sg.AdamWPlan([], [], []).step([], hp)
