"""Products in 8 bits with their gradients as an autograd operator, at the edges of their ranges, and a run of the 8-bit operators
together as a training step uses them: weights quantised from their masters, forward, backward, AdamW with states in 8 bits."""
import numpy as np
import pytest
import torch

import bwd_situ_glu_gb300 as sg
from bwd_situ_glu_gb300 import fp8
import _fp8_ref as ref8

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def offsets_of(counts):
    return torch.tensor([0, *np.cumsum(counts)], dtype=torch.int64, device=DEV)


def data(R, N, K, E, seed, w_dtype=BF):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    lead = (E,) if E else ()
    return [randn(R, K).to(BF), (randn(*lead, N, K) / K ** 0.5).to(w_dtype), randn(*lead, N), randn(R, N).to(BF)], randn(R, N).to(BF)


# ---------------------------------------------------------------- autograd

@pytest.mark.parametrize("w_dtype", [BF, torch.float32])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("counts", [70, [40, 0, 25]], ids=str)
def test_autograd_matches_the_calls(counts, act, w_dtype):
    dense = isinstance(counts, int)
    R, N, K, E = (counts if dense else sum(counts)), 272, 144, (0 if dense else len(counts))
    off = None if dense else offsets_of(counts)
    ins, dout = data(R, N, K, E, 1, w_dtype)
    qa, qw = sg.situ_quant_fp8(ins[0]), sg.situ_quant_fp8(ins[1], block_rows=128)
    want, pre = sg.situ_linear_fp8(qa, qw, off, bias=ins[2], residual=ins[3], act=act, save_pre=True)
    da, dw, db = sg.situ_linear_fp8_bwd(dout, qa, qw, off, act=act, pre=pre, dw_dtype=w_dtype)
    for wq in (None, qw):
        ts = [t.clone().requires_grad_() for t in ins]
        out = fp8.linear_fp8(*ts, expert_offsets=off, act=act, wq=wq)
        assert torch.equal(out, want)
        out.backward(dout)
        for t, g in zip(ts, (da, dw, db, dout)):
            assert t.grad.dtype == t.dtype and torch.equal(t.grad, g)


@pytest.mark.parametrize("needed", [(0,), (1,), (2,), (3,), (0, 3), (1, 2)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_autograd_of_some_inputs(needed, act):
    """Gradients of some of a, w, bias, residual are those of all four, and only they are given."""
    ins, dout = data(37, 80, 48, 0, 2)
    grads = []
    for some in ((0, 1, 2, 3), needed):
        ts = [t.clone().requires_grad_(i in some) for i, t in enumerate(ins)]
        fp8.linear_fp8(*ts, act=act).backward(dout)
        grads.append([t.grad for t in ts])
    for i, (every, some) in enumerate(zip(*grads)):
        assert torch.equal(some, every) if i in needed else some is None


@pytest.mark.parametrize("act", ["none", "relu"])
def test_gradients_are_differences_of_the_quantised_product(act):
    """The function of the operands' own values, in 64 bits, moved along random directions: linear in each (relu: in a step too small
    to cross 0), so central differences are exact. dout is made of numbers that 8 bits hold, so dz has no rounding of its own; what is
    left is a bf16 gradient's half step, 2^-8 of each element."""
    R, N, K = 60, 272, 144
    ins, _ = data(R, N, K, 0, 3)
    g = torch.Generator(device=DEV).manual_seed(4)
    dout = torch.randint(-3, 4, (R, N), generator=g, device=DEV).to(BF)
    ts = [t.clone().requires_grad_() for t in ins]
    fp8.linear_fp8(*ts, act=act).backward(dout)
    at = [ref8.values(*sg.situ_quant_fp8(ins[0]), 1), ref8.values(*sg.situ_quant_fp8(ins[1], block_rows=128), 128), ins[2].double(), ins[3].double()]

    def loss(a, w, b, r):
        z = a @ w.t() + b
        return ((z.clamp(min=0) if act == "relu" else z) + r).mul(dout.double()).sum()
    for i, t in enumerate(ts):
        d = torch.randn(t.shape, generator=g, device=DEV).double()
        h = 1e-7
        moved = [[x + s * h * d if k == i else x for k, x in enumerate(at)] for s in (1, -1)]
        want = (loss(*moved[0]) - loss(*moved[1])).item() / (2 * h)
        got = (t.grad.double() * d).sum().item()
        tol = ((t.grad.double() * d).abs().sum().item() * (2.0 ** -8 + 1e-4) + 1e-4 * abs(want))      # 1e-4: sums and the differences
        assert abs(got - want) <= tol, i


# ---------------------------------------------------------------- as a program uses them

class Step:
    """One training step of two 8-bit layers: experts' product, relu, a dense product; squared error; AdamW in 8 bits."""

    def __init__(self, state="fp8", seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.off = offsets_of([100, 0, 37, 63])
        self.master = [randn(4, 256, 144) / 12, randn(4, 256) * 0.1, randn(80, 256) / 16]
        self.work = [t.to(BF) for t in self.master]
        self.plan = sg.AdamWPlan(self.master, work=self.work, **sg.adamw_state(self.master, state))
        self.x, self.y = randn(200, 144).to(BF), randn(200, 80).to(BF)

    def grads(self):
        w1, b1, w2 = (t.detach().requires_grad_() for t in self.master)
        h = fp8.linear_fp8(self.x, w1, b1, expert_offsets=self.off, act="relu")
        out = fp8.linear_fp8(h, w2)
        loss = (out.float() - self.y.float()).square().mean()
        return loss.detach(), torch.autograd.grad(loss, (w1, b1, w2))


@pytest.mark.parametrize("state", ["fp32", "fp8"])
def test_training_steps_captured_and_replayed(state):
    """Three steps eagerly, and the same three as replays of one captured step whose coefficients come from the device: the same
    bits in weights, states and working copies; and every step has moved the weights."""
    eager, graphed = Step(state), Step(state)
    hp = lambda k: sg.adam_params(lr=1e-2, weight_decay=0.01, step=k)  # noqa: E731
    first = [t.clone() for t in eager.master]
    for k in (1, 2, 3):
        before = eager.master[0].clone()
        _, gs = eager.grads()
        eager.plan.step(gs, hp(k))
        assert not torch.equal(before, eager.master[0])
    coef = sg.adamw_coefficients(hp(1)).to(DEV)
    s = torch.cuda.Stream()                  # warm-up on a side stream, as captures want it
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graphed.grads()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, gs = graphed.grads()
        graphed.plan.step(gs, coef)
    assert all(torch.equal(a, b) for a, b in zip(first, graphed.master))
    for k in (1, 2, 3):
        coef.copy_(sg.adamw_coefficients(hp(k)))
        graph.replay()
    for name in eager.plan._lists:
        for a, b in zip(eager.plan._lists[name], graphed.plan._lists[name]):
            assert torch.equal(a, b), name
    assert all(torch.equal(w, m.to(BF)) for w, m in zip(graphed.work, graphed.master)) and torch.isfinite(loss)


def test_two_streams_at_once():
    """Two products and a quantisation on two streams of their own, many times: each is what it is alone."""
    jobs = []
    for seed, (R, E, counts) in enumerate(((500, 0, None), (420, 3, [200, 0, 220]))):
        ins, _ = data(R, 528, 400, E, seed)
        qw = sg.situ_quant_fp8(ins[1], block_rows=128)
        off = None if counts is None else offsets_of(counts)
        jobs.append((ins[0], qw, off, sg.situ_linear_fp8(ins[0], qw, off), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[sg.situ_linear_fp8(a, qw, off, stream=s) for _ in range(20)] for a, qw, off, _, s in jobs]
    torch.cuda.synchronize()
    for (_, _, _, want, _), got in zip(jobs, outs):
        assert all(torch.equal(want, x) for x in got)


def test_results_repeat():
    ins, dout = data(900, 528, 656, 3, 5)
    off = offsets_of([500, 3, 397])
    qa, qw = sg.situ_quant_fp8(ins[0]), sg.situ_quant_fp8(ins[1], block_rows=128)
    runs = [[sg.situ_linear_fp8(qa, qw, off, bias=ins[2]), *sg.situ_linear_fp8_bwd(dout, qa, qw, off)] for _ in range(3)]
    assert all(torch.equal(x, y) for other in runs[1:] for x, y in zip(runs[0], other))


# ---------------------------------------------------------------- edges

def small_integers(*shape, seed=0):
    """Values that 8 bits hold exactly and whose sums fp32 holds exactly, in any order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device=DEV).to(BF)


@pytest.mark.parametrize("offsets", [[0, 50, 20, 200], [0, 300, 500, 100], [-5, 40, 9000, 200], [200, 100, 0, 150], [0, 0, 0, 0], [7, 60, 60, 150],
                                     [0, 200, 200, -3]], ids=str)
@pytest.mark.parametrize("R", [12, 200])
def test_offsets_out_of_order_are_those_of_the_bf16_product(offsets, R):
    """Malformed offsets give the rows that situ_linear gives them, bit for bit; other rows stay as they were."""
    a, w, dz = small_integers(R, 144), small_integers(3, 272, 144, seed=1), small_integers(R, 272, seed=2)
    off = torch.tensor(offsets, dtype=torch.int64, device=DEV)
    qa, qw = sg.situ_quant_fp8(a), sg.situ_quant_fp8(w, block_rows=128)
    want, got = (torch.full((R, 272), 7.0, dtype=BF, device=DEV) for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    sg.situ_linear(a, w, off, out=want, status=st)
    sg.situ_linear_fp8(qa, qw, off, out=got, status=st)
    assert torch.equal(want, got) and st.item() == 0
    da, dw, db = sg.situ_linear_fp8_bwd(dz, qa, qw, off, status=st)
    wa, ww, wb = sg.situ_linear_bwd(dz, a, w, off)
    live = (got != 7.0).any(1)
    assert torch.equal(da[live], wa[live]) and torch.equal(dw, ww) and torch.equal(db, wb) and st.item() == 0


def test_most_rows():
    """The largest R, 2^31 - 1025, at both ends and in the middle, zeros elsewhere."""
    R, N, K = 2 ** 31 - 1025, 16, 16
    places = [slice(0, 40), slice(2 ** 30 - 20, 2 ** 30 + 20), slice(R - 300, R)]
    w, st = small_integers(N, K), torch.zeros(1, dtype=torch.int32, device=DEV)
    qw = [t[0] for t in sg.situ_quant_fp8(w[None], block_rows=128)]
    a, s = torch.zeros(R, K, dtype=torch.uint8, device=DEV), torch.ones(R, 1, dtype=torch.uint8, device=DEV)
    rows = {}
    for i, r in enumerate(places):
        rows[i] = small_integers(r.stop - r.start, K, seed=i)
        a[r], s[r] = sg.situ_quant_fp8(rows[i])
    out = sg.situ_linear_fp8((a, s), qw, status=st)
    for i, r in enumerate(places):
        assert torch.equal(out[r], (rows[i].float() @ w.float().t()).to(BF))
    for r in (slice(40, 4000), slice(2 ** 30 + 20, 2 ** 30 + 4000), slice(R - 4000, R - 300)):
        assert not out[r].any()
    da = out                                  # the memory of one tensor of 69 GB for both
    lib = sg.load()
    assert lib.situ_linear_fp8_dgrad(a.data_ptr(), s.data_ptr(), qw[0].data_ptr(), qw[1].data_ptr(), None, 1, da.data_ptr(), st.data_ptr(), R, N, K,
                                     torch.cuda.current_stream().cuda_stream) == 0
    for i, r in enumerate(places):
        assert torch.equal(da[r], (rows[i].float() @ w.float()).to(BF))
    assert st.item() == 0


@pytest.mark.parametrize("rows", [3, 100])
def test_weights_past_32_bits(rows):
    """1024 experts of 2064 x 2048: the last one's weights begin past 2^32 bytes."""
    E, N, K = 1024, 2064, 2048
    qw = (torch.zeros(E, N, K, dtype=torch.uint8, device=DEV), torch.ones(E, 17, 16, dtype=torch.uint8, device=DEV))
    w = small_integers(1, N, K)
    qw[0][E - 1:], qw[1][E - 1:] = sg.situ_quant_fp8(w, block_rows=128)
    a, dz = small_integers(rows, K, seed=1), small_integers(rows, N, seed=2)
    off = torch.full((E + 1,), rows, dtype=torch.int64, device=DEV)
    off[:E] = 0
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sg.situ_linear_fp8(a, qw, off, status=st)
    da, _, _ = sg.situ_linear_fp8_bwd(dz, None, qw, off, bias=False, need_dw=False, status=st)
    assert torch.equal(out, (a.double() @ w[0].double().t()).to(BF)) and torch.equal(da, (dz.double() @ w[0].double()).to(BF)) and st.item() == 0


def test_rows_are_empty():
    a, w = torch.zeros(0, 32, dtype=BF, device=DEV), torch.ones(2, 48, 32, device=DEV)
    off = torch.zeros(3, dtype=torch.int64, device=DEV)
    qw = sg.situ_quant_fp8(w, block_rows=128)
    assert sg.situ_linear_fp8(a, qw, off).shape == (0, 48)
    da, dw, db = sg.situ_linear_fp8_bwd(torch.zeros(0, 48, dtype=BF, device=DEV), sg.situ_quant_fp8(a), qw, off)
    assert da.shape == (0, 32) and not dw.any() and not db.any() and dw.shape == (2, 48, 32)


def test_refusals():
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    a, w = (z(4, 32), z(4, 1)), (z(16, 32), z(1, 1))
    off = z(3, dtype=torch.int64)
    lin, bwd = sg.situ_linear_fp8, sg.situ_linear_fp8_bwd
    for bad, error in ((lambda: lin(a, w[0]), TypeError), (lambda: lin(a, (z(16, 48), z(1, 1))), ValueError), (lambda: lin(a, (w[0], z(1, 2))), ValueError),
                       (lambda: lin((a[0], z(4, 2)), w), ValueError), (lambda: lin(a, w, off), ValueError), (lambda: lin(a, (z(3, 16, 32), z(3, 1, 1)), off), ValueError),
                       (lambda: lin(a, w, act="tanh"), ValueError), (lambda: lin(a, w, bias=z(16)), TypeError), (lambda: lin(a, w, residual=z(4, 32, dtype=BF)), ValueError),
                       (lambda: lin((a[0].float(), a[1]), w), TypeError), (lambda: lin(z(4, 32, dtype=torch.float16), w), TypeError),
                       (lambda: lin((z(4, 64)[:, ::2], a[1]), w), ValueError), (lambda: lin(a, w, out=z(4, 16, dtype=torch.float16)), TypeError),
                       (lambda: lin((a[0].cpu(), a[1]), w), ValueError), (lambda: bwd(z(4, 16, dtype=BF), a, w, act="silu"), ValueError),
                       (lambda: bwd(z(4, 16, dtype=torch.float32), a, w), TypeError), (lambda: bwd(z(4, 16, dtype=BF), a[0], w), TypeError),
                       (lambda: fp8.linear_fp8(z(4, 32, dtype=torch.float32), z(16, 32, dtype=BF)), TypeError)):
        with pytest.raises(error):
            bad()
    for bad in (lambda: lin((z(4, 24), z(4, 1)), (z(16, 24), z(1, 1))), lambda: lin(a, (z(24, 32), z(1, 1))),
                lambda: lin((z(4 * 32 + 8)[8:].view(4, 32), a[1]), w)):        # off a 16-byte boundary
        with pytest.raises(sg.SituGluError) as err:
            bad()
        assert err.value.status == 1
    buf = z(4, 16, dtype=BF)
    with pytest.raises(sg.SituGluError) as err:
        lin((buf.view(torch.uint8).view(-1)[:128].view(4, 32), a[1]), w, out=buf)
    assert err.value.status == 2


@pytest.mark.parametrize("R,N,K", [(3, 272, 4096), (700, 272, 4096), (4000, 80, 400)])
def test_a_product_right_behind_its_quantiser(R, N, K):
    """The product's launch overlaps the end of the kernel before it, whatever that is: the same buffers again and again, filled by a
    copy and quantised in front of each product, the weights too; eagerly and replayed."""
    w, xs = small_integers(N, K, seed=9), [small_integers(R, K, seed=i) for i in range(8)]
    want = [(x.double() @ w.double().t()).to(BF) for x in xs]
    x, codes, scales = torch.empty_like(xs[0]), *sg.situ_quant_fp8(xs[0])
    wq = [t[0] for t in sg.situ_quant_fp8(w[None], block_rows=128)]
    outs = [torch.empty(R, N, dtype=BF, device=DEV) for _ in xs]

    def go():
        for y, out in zip(xs, outs):
            x.copy_(y)
            sg.situ_quant_fp8(x, codes=codes, scales=scales)
            sg.situ_quant_fp8(w, block_rows=128, codes=wq[0], scales=wq[1])
            sg.situ_quant_fp8(x, codes=codes, scales=scales)
            sg.situ_linear_fp8((codes, scales), wq, out=out)
            sg.situ_linear_fp8((codes, scales), wq, out=out)
    for _ in range(20):
        go()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for out in outs:
        out.zero_()
    for _ in range(20):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
