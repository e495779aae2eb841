"""Expert offsets that are negative, decreasing, far beyond R or overlapping, given to the expert layer's operators: nothing
outside the buffers is written (guard bands around every output and workspace, the workspaces at exactly the size the
library asks for), the calls return promptly, and the products read the offsets as the largest one so far, clamped into
[0, R]: bit for bit what those offsets give."""
import time

import numpy as np
import pytest
import torch

import bwd_situ_glu_gb300 as sg

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


def everything(off, R, N, K, act):
    """All products and gradients for these offsets, through the C entry points."""
    lib, E = sg.load(), off.numel() - 1
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
    return [out.view(BF, R, N), pre.view(BF, R, N), dz.view(BF, R, N), da.view(BF, R, K), dw.view(torch.float32, E, N, K),
            db.view(torch.float32, E, N)]


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("name", BAD)
@pytest.mark.parametrize("R", [40, 200, 2100])
def test_products(R, name, act):
    raw = np.array(BAD[name](R), dtype=np.int64)
    repaired = np.maximum.accumulate(np.clip(raw, 0, R))
    got, want = (everything(torch.from_numpy(o).to(DEV), R, 264, 72, act) for o in (raw, repaired))
    for g, w, what in zip(got, want, ("out", "pre", "dz", "da", "dw", "dbias")):
        assert torch.equal(g, w), what


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
