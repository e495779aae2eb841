"""The per-expert / dense product and its gradients at the edges of their ranges on the GPU."""
import math

import numpy as np
import pytest
import torch

import bwd_situ_glu_gb300 as sg
from bwd_situ_glu_gb300 import moe
import _moe_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def test_most_rows():
    """The largest R, 2^31 - 1025 (34 GB a tensor): rows at both ends and in the middle, zeros elsewhere. Eighths up to 1
    make every product and sum exact in fp32, whatever its order; a bf16 result is that sum rounded once."""
    R, N, K = 2 ** 31 - 1025, 8, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    new = lambda *s: (torch.randint(-8, 9, s, generator=g, device=DEV) / 8).to(BF)  # noqa: E731
    places = [slice(0, 40), slice(2 ** 30 - 20, 2 ** 30 + 20), slice(R - 300, R)]
    w, a, dz = new(N, K), torch.zeros(R, K, dtype=BF, device=DEV), torch.zeros(R, N, dtype=BF, device=DEV)
    for r in places:
        a[r], dz[r] = new(r.stop - r.start, K), new(r.stop - r.start, N)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sg.situ_linear(a, w, status=st)
    da, dw, db = sg.situ_linear_bwd(dz, a, w, status=st)
    assert st.item() == 0
    for r in places:
        assert torch.equal(out[r], (a[r].float() @ w.float().t()).to(BF)) and torch.equal(da[r], (dz[r].float() @ w.float()).to(BF))
    for r in (slice(40, 4000), slice(2 ** 30 + 20, 2 ** 30 + 4000), slice(R - 4000, R - 300)):
        assert not out[r].any() and not da[r].any()
    assert torch.equal(dw, sum(dz[r].float().t() @ a[r].float() for r in places))
    assert torch.equal(db, sum(dz[r].float().sum(0) for r in places))


# gelu on the left side: fp32 evaluation of Φ(z) = t·P(t)·e^{-z²/2} is good to 8e-7 (the fit), some ten roundings and the
# approximate exp2 and reciprocal (2^-22 each): below 3e-6, and the exponent z²/2 is rounded twice: z²·1.2e-7
def gelu_rel(z):
    return 3e-6 + z * z * 1.2e-7


@pytest.mark.parametrize("R", [1, 256])                # streamed weights, and tiles
def test_gelu_relative_accuracy(R):
    """fp32 outputs down to z = -9, where gelu is -1e-18, keep their digits."""
    N = 1024
    z = torch.cat([-torch.linspace(0, 9, N - 8), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3.0, 9.0, 40.0, 3e38])])
    out = sg.situ_linear(torch.zeros(R, 8, dtype=BF, device=DEV), torch.ones(N, 8, dtype=BF, device=DEV), bias=z.to(DEV), act="gelu",
                         out_dtype=torch.float32)
    zd = z.double().numpy()
    want = ref.act(zd, "gelu")[0]
    ref.near(out, np.broadcast_to(want, (R, N)), gelu_rel(np.minimum(np.abs(zd), 9)) * np.abs(want), "out")


def test_gelu_gradient_accuracy():
    """The bias gradient of one row is act'(pre) in fp32: Φ(z) + z·φ(z), each term to the same relative accuracy."""
    z = torch.cat([-torch.linspace(0, 9, 1016), torch.linspace(0, 40, 8)]).to(BF)
    N = z.numel()
    pre = z[None].to(DEV)
    _, _, db = sg.situ_linear_bwd(torch.ones(1, N, dtype=BF, device=DEV), None, torch.zeros(N, 8, dtype=BF, device=DEV), act="gelu",
                                  pre=pre, need_da=False, need_dw=False)
    zd = z.double().numpy()
    cdf = 0.5 * torch.special.erfc(-z.double() / math.sqrt(2)).numpy()
    zphi = np.abs(zd) * np.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    ref.near(db, ref.act(zd, "gelu")[1], gelu_rel(np.abs(zd)) * (cdf + zphi), "dbias")


@pytest.mark.parametrize("R", [2 ** 25, 2 ** 25 - 77])
def test_bias_gradient_of_many_rows(R):
    """Equal values make roundings add up: 1 + 2^-7 summed over 2^25 rows in one chain of 128-row pieces loses 2^-8 of the
    sum. Chains of at most 2·sqrt(R) additions stay within 2·sqrt(R)·2^-24."""
    N = 8
    dout = torch.full((R, N), 1 + 2.0 ** -7, dtype=BF, device=DEV)
    _, _, db = sg.situ_linear_bwd(dout, None, torch.zeros(N, 8, dtype=BF, device=DEV), need_da=False, need_dw=False)
    want = np.full(N, R * (1 + 2.0 ** -7))
    ref.near(db, want, 2 * math.sqrt(R) * ref.U24 * want, "dbias")


def test_bias_gradient_of_many_ragged_rows():
    """Experts of 0 to 400000 rows, 1.1 million in all: pieces of more than 128 rows that end inside an expert."""
    counts = [400_000, 0, 1, 299_999, 128, 400_001]
    R, N = sum(counts), 40
    g = torch.Generator(device=DEV).manual_seed(2)
    dout = torch.randn(R, N, generator=g, device=DEV).to(BF)
    off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int64, device=DEV)
    _, _, db = sg.situ_linear_bwd(dout, None, torch.zeros(len(counts), N, 8, dtype=BF, device=DEV), off, need_da=False, need_dw=False)
    for e in range(len(counts)):
        x = dout[off[e]:off[e + 1]].double()
        ref.near(db[e], x.sum(0).cpu().numpy(), (2 * math.sqrt(R) * ref.U24 * x.abs().sum(0)).cpu().numpy(), f"dbias {e}")


def np64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("counts", [[5, 0, 11], [140, 3, 130]], ids=str)
@pytest.mark.parametrize("of", ["a", "w"])
def test_gradient_by_differences_along_its_signs(counts, act, of):
    """Central differences of <out, dout> (fp32 out) along the signs of the float64 gradient, where its entries add up to
    some thirty times the tolerance: a gradient without act', or a zero one, does not pass.

    d = dz/d(step). Differences: third derivative below 2, times d^3 eps^2 / 6, and the rounding of out over eps. Gradient:
    act' off by act'' (below 1.2) times half an ulp of pre, dz by half an ulp, da by half an ulp."""
    R, N, K, E = sum(counts), 40, 24, 3
    g = torch.Generator().manual_seed(12)
    a = (torch.randint(-8, 9, (R, K), generator=g) / 8).to(BF)
    w = (torch.randint(-8, 9, (E, N, K), generator=g) / 32).to(BF)
    bias, dout = torch.randn(E, N, generator=g) * 0.1, torch.randn(R, N, generator=g).to(BF)
    offs = np.array([0, *np.cumsum(counts)])
    off = torch.from_numpy(offs).to(DEV)
    A, W, B, G = np64(a), np64(w), np64(bias), np64(dout)
    _, z, smag = ref.linear(A, W, offs, B, None, "none")
    want, flat = (ref.linear_bwd(G, A, W, offs, z, name)["d" + of] for name in (act, "none"))
    v = np.where(want < 0, -1.0, 1.0)
    eps = 2.0 ** -5 if of == "a" else 2.0 ** -6         # a ± eps and w ± eps are bf16 values
    step = torch.from_numpy(v * eps)
    _, pre = sg.situ_linear(a.to(DEV), w.to(DEV), off, bias=bias.to(DEV), act=act, save_pre=True)
    da, dw, _ = sg.situ_linear_bwd(dout.to(DEV), a.to(DEV), w.to(DEV), off, act=act, pre=pre)

    def loss(sign):
        x, y = (a.double() + sign * step, w) if of == "a" else (a, w.double() + sign * step)
        out = sg.situ_linear(x.to(BF).to(DEV), y.to(BF).to(DEV), off, bias=bias.to(DEV), act=act, out_dtype=torch.float32)
        return (np64(out) * G).sum()

    num = (loss(1) - loss(-1)) / (2 * eps)
    d = np.abs(ref.linear(v, W, offs, None, None, "none")[0] if of == "a" else ref.linear(A, v, offs, None, None, "none")[0])
    dabs, az = np.abs(G), np.abs(z)
    tol = (dabs * (((K / 16 + 2) * 2.0 ** -22 * smag * 1.13 + 2e-6 * (1 + az)) / eps)).sum()
    tol += (np.abs(want) * ref.BF16_HALF).sum() if of == "a" else 1e-5 * (dabs * d).sum()
    if act != "none":
        tol += (dabs * (d ** 3 * eps ** 2 / 3 + d * (1.2 * ref.BF16_HALF * az + 1.13 * ref.BF16_HALF + 4e-6))).sum()
        assert abs((flat * v).sum() - num) > 10 * tol
    assert tol < 0.05 * abs(num)
    assert abs(num - (np64(da if of == "a" else dw) * v).sum()) <= tol
