"""Expert offsets that are negative, decreasing, far beyond R or overlapping, given to the expert layer's operators: nothing
outside the buffers is written (guard bands around every output and workspace, the workspaces at exactly the size the
library asks for), the calls return promptly, and in the products every expert has the rows of its offsets clamped into
[0, R], but none where it begins before an earlier one ends; tolerances as in test_linear_gpu.py."""
import math
import time

import numpy as np
import pytest
import torch

import bwd_situ_glu_gb300 as sg
import _moe_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16
GUARD = 1 << 16
BAD = {
    "mixed": lambda R: [0, -5, 1 << 40, 100, 50, R],
    "overlapping": lambda R: [0, R] * 5,
    "many overlapping": lambda R: [0, R] * 512,
    "decreasing": lambda R: [R, R // 2, 7, 0],
    "negative": lambda R: [-9, -3, -1],
    "beyond": lambda R: [R + 1, R + 2, 1 << 62],
    "extremes": lambda R: [-(1 << 63), (1 << 63) - 1, -(1 << 63), 5],
    "starts late, ends early": lambda R: [3, 3, R - 2, R - 5],
}


class Guarded:
    """A zeroed buffer of nbytes with guard bands of 0xFF bytes before and after it."""
    made = []

    def __init__(self, nbytes):
        self.n = nbytes
        self.buf = torch.full((nbytes + 2 * GUARD,), 255, dtype=torch.uint8, device=DEV)
        self.buf[GUARD:GUARD + nbytes] = 0
        self.made.append(self)

    def view(self, dtype, *shape):
        return self.buf[GUARD:GUARD + self.n].view(dtype).view(*shape)

    @property
    def ptr(self):
        return self.buf.data_ptr() + GUARD

    def intact(self):
        return bool((self.buf[:GUARD] == 255).all()) and bool((self.buf[GUARD + self.n:] == 255).all())


@pytest.fixture(autouse=True)
def guards():
    Guarded.made = []
    t0 = time.time()
    yield
    torch.cuda.synchronize()
    assert time.time() - t0 < 30.0
    assert Guarded.made and all(g.intact() for g in Guarded.made)


def ok(status):
    assert status == sg.STATUS_OK


def ranges(raw, R):
    """(begin, end) of the experts that keep rows, by expert."""
    kept, last = {}, 0
    for e, (a, b) in enumerate(zip(raw[:-1], raw[1:])):
        a = min(max(a, 0), R)
        b = min(max(b, a), R)
        if a >= last:
            last = b
            if b > a:
                kept[e] = slice(a, b)
    return kept


def near(got, want, tol, what):
    assert ((got.double() - want).abs() <= tol).all(), what


def steps_tol(n, mag):
    return (n / 16 + 2) * 2.0 ** -22 * mag


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("name", BAD)
@pytest.mark.parametrize("R", [40, 200, 2100])
def test_products(R, name, act):
    lib, N, K = sg.load(), 264, 72
    raw = BAD[name](R)
    E = len(raw) - 1
    off = torch.from_numpy(np.array(raw, dtype=np.int64)).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    new = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    a, w, dout, z, res = new(R, K), new(E, N, K), new(R, N), new(R, N), new(R, N)
    bias = torch.randn(E, N, generator=g, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    code = sg.moe.ACTIVATIONS[act]
    out, pre, dz, da = Guarded(R * N * 2), Guarded(R * N * 2), Guarded(R * N * 2), Guarded(R * K * 2)
    dw, db = Guarded(E * N * K * 4), Guarded(E * N * 4)
    ok(lib.situ_linear_fwd(a.data_ptr(), w.data_ptr(), off.data_ptr(), E, bias.data_ptr(), res.data_ptr(), code, out.ptr, 0,
                           pre.ptr, status.data_ptr(), R, N, K, s))
    nb = lib.situ_linear_act_bwd_workspace(R, N, E)
    ws = Guarded(nb)
    ok(lib.situ_linear_act_bwd(dout.data_ptr(), z.data_ptr(), code, off.data_ptr(), E, dz.ptr, db.ptr, ws.ptr, nb, R, N, s))
    ok(lib.situ_linear_dgrad(dout.data_ptr(), w.data_ptr(), off.data_ptr(), E, da.ptr, status.data_ptr(), R, N, K, s))
    nb = lib.situ_linear_wgrad_workspace(R, N, K, E)
    ws = Guarded(nb)
    ok(lib.situ_linear_wgrad(dout.data_ptr(), a.data_ptr(), off.data_ptr(), E, dw.ptr, 1, ws.ptr if nb else 0, nb,
                             status.data_ptr(), R, N, K, s))
    torch.cuda.synchronize()
    assert status.item() == 0
    # the definitions in float64; what no expert owns stays the zero that it was, and so do its gradients
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device=DEV)  # noqa: E731
    want = dict(out=zeros(R, N), pre=zeros(R, N), dz=zeros(R, N), da=zeros(R, K), dw=zeros(E, N, K), db=zeros(E, N))
    tol = {k: v.clone() for k, v in want.items()}
    half = 1.01 * ref.BF16_HALF
    for e, r in ranges(raw, R).items():
        A, W, G, Z = a[r].double(), w[e].double(), dout[r].double(), z[r].double()
        y = A @ W.t() + bias[e]
        mag = A.abs() @ W.abs().t() + bias[e].abs()
        sig, y_sig = torch.sigmoid(Z), torch.sigmoid(y)
        slope = sig * (1 + Z * (1 - sig)) if code else torch.ones_like(Z)
        want["pre"][r], tol["pre"][r] = y, steps_tol(K, mag) + half * y.abs()
        want["out"][r] = (y * y_sig if code else y) + res[r].double()
        tol["out"][r] = 1.13 * steps_tol(K, mag) + 2e-6 * (1 + y.abs()) + half * want["out"][r].abs()
        if code:
            want["dz"][r], tol["dz"][r] = G * slope, 4e-6 * G.abs() + half * (G * slope).abs()
        want["da"][r], tol["da"][r] = G @ W, steps_tol(N, G.abs() @ W.abs()) + half * (G @ W).abs()
        want["dw"][e], tol["dw"][e] = G.t() @ A, steps_tol(r.stop - r.start, G.abs().t() @ A.abs()) + 2 * ref.U24 * (G.t() @ A).abs()
        want["db"][e], tol["db"][e] = (G * slope).sum(0), (2 * math.sqrt(R) * 1.13 * ref.U24 + 4e-6 * (code > 0)) * G.abs().sum(0)
    for k, (buf, dtype) in dict(out=(out, BF), pre=(pre, BF), dz=(dz, BF), da=(da, BF), dw=(dw, torch.float32), db=(db, torch.float32)).items():
        near(buf.view(dtype, *want[k].shape), want[k], tol[k], k)


@pytest.mark.parametrize("name", BAD)
def test_dispatch_and_combine(name):
    T, K, D = 50, 4, 72
    R = T * K
    g = torch.Generator(device=DEV).manual_seed(4)
    off = torch.from_numpy(np.array(BAD[name](R), dtype=np.int64)).to(DEV)
    x, o, p = torch.randn(T, D, generator=g, device=DEV).to(BF), torch.randn(R, D, generator=g, device=DEV).to(BF), torch.rand(T, K, generator=g, device=DEV)
    row_of = torch.randperm(R, generator=g, device=DEV).to(torch.int32).view(T, K)
    h, do, dp = Guarded(R * D * 2), Guarded(R * D * 2), Guarded(T * K * 4)
    sg.situ_dispatch(x, row_of, off, h=h.view(BF, R, D))
    sg.situ_combine_bwd(x, o, row_of, p, off, do=do.view(BF, R, D), dweights=dp.view(torch.float32, T, K))
    want = torch.einsum("td,tkd->tk", x.double(), o.double()[row_of.long()])     # does not depend on the offsets
    # some 20 fp32 additions in a chain, of products whose absolute values sum to less than 80
    assert (dp.view(torch.float32, T, K).double() - want).abs().max() < 20 * 2.0 ** -24 * 80


@pytest.mark.parametrize("call", ["gateup", "dgrad"])
def test_fused_products_stay_bounded(call):
    """Overlapping offsets are no more work for the fused products than orderly ones over the same rows (ceil(R/128) + E
    row tiles; every second expert owning every row would be 300 times that)."""
    R, H, D, E = 100_000, 256, 64, 1023
    g = torch.Generator(device=DEV).manual_seed(5)
    new = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    h, w, x, p = new(R, D), new(E, 2 * H, D), new(R, 2 * H), torch.rand(R, generator=g, device=DEV)
    xo, out, dx = Guarded(R * 2 * H * 2), Guarded(R * H * 2), Guarded(R * 2 * H * 2)
    dp = torch.empty(R, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)

    def ms(off):
        best = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            if call == "gateup":
                sg.situ_glu_fwd_gateup(h, w, off, xo.view(BF, R, 2 * H), out.view(BF, R, H), status=st)
            else:
                sg.situ_glu_bwd_router_dgrad(x, h, w[:, :H].contiguous(), off, p, dx.view(BF, R, 2 * H), dp, status=st)
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        return min(best)

    orderly = torch.linspace(0, R, E + 1, device=DEV).long()
    overlapping = torch.tensor([0, R] * 512, device=DEV)
    t = ms(orderly), ms(overlapping)
    assert st.item() == 0
    assert t[1] < 5 * t[0], t


def test_rows_without_a_token():
    """Rows past the plan's last are zeroed; one before it that row_of does not name (a pair dropped after the plan) is not
    written; dropped by its id before the plan, the pair has no row at all."""
    T, K, D = 6, 2, 40
    g = torch.Generator(device=DEV).manual_seed(6)
    x, w = torch.randn(T, D, generator=g, device=DEV), torch.rand(T, K, generator=g, device=DEV)
    ids = torch.tensor([[0, 2], [1, -1], [2, 0], [0, 1], [-1, -1], [1, 2]], dtype=torch.int32, device=DEV)
    offsets, row_of, _, _ = sg.situ_dispatch_plan(ids, 3)
    n, R = int(offsets[-1]), T * K
    assert n == 9
    lost = int(row_of[3, 0])
    dropped = row_of.clone()
    dropped[3, 0] = -1
    h, do = Guarded(R * D * 4), Guarded(R * D * 4)
    hv, dv = h.view(torch.float32, R, D), do.view(torch.float32, R, D)
    hv.fill_(7.0)
    dv.fill_(7.0)
    sg.situ_dispatch(x, dropped, offsets, h=hv)
    sg.situ_combine_bwd(x, torch.ones(R, D, device=DEV), dropped, w, offsets, do=dv)
    for buf in (hv, dv):
        assert (buf[n:] == 0).all() and (buf[lost] == 7.0).all()
    for t in range(T):
        for k in range(K):
            if dropped[t, k] >= 0:
                assert torch.equal(hv[dropped[t, k]], x[t]) and torch.equal(dv[dropped[t, k]], w[t, k] * x[t])
    ids[3, 0] = -1
    offsets, row_of, _, _ = sg.situ_dispatch_plan(ids, 3)
    hv.fill_(7.0)
    sg.situ_dispatch(x, row_of, offsets, h=hv)
    assert int(offsets[-1]) == n - 1 and (hv[n - 1:] == 0).all() and not (hv == 7.0).any()
