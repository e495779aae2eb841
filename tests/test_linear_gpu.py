"""The per-expert / dense product with bias, activation and residual and its gradients on the GPU against the
plain float64 definitions.

Tolerances (derived, not fitted). Tensor-core sums in fp32 may cut each 16-wide step's result towards
zero: n steps stay within (n + 2)·2^-22·Σ|terms|. An activation multiplies that by at most 1.13 (gelu' <
1.129, silu' < 1.1) and is itself evaluated to 2e-6·(1 + |z|) absolute; a bf16 result adds half an ulp,
2^-8 relative. dz is rounded to bf16 before the products, half an ulp of every term: 2^-8·Σ|terms|."""
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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def np64(t):
    return t.detach().cpu().double().numpy()


def dev(t):
    return None if t is None else t.to(DEV)


def steps_tol(n, mag):
    return (n / 16 + 2) * 2.0 ** -22 * mag


def offsets_of(counts):
    return torch.tensor([0, *np.cumsum(counts)], dtype=torch.int64)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def inputs(R, N, K, E, seed):
    g = gen(seed)
    a = torch.randn(R, K, generator=g).to(BF)
    w = (torch.randn(E, N, K, generator=g) / math.sqrt(K)).to(BF)
    return g, a, w, torch.randn(E, N, generator=g), torch.randn(R, N, generator=g).to(BF)


def check_fwd(counts, N, K, act, with_bias, with_res, out_dtype, save_pre, seed=0, tail=0):
    """counts: rows per expert, or an int: dense. tail: rows past the last expert's."""
    dense = isinstance(counts, int)
    counts = [counts] if dense else counts
    R, E = sum(counts) + tail, len(counts)
    g, a, w, bias, res = inputs(R, N, K, E, seed)
    off = offsets_of(counts)
    want, z, mag = ref.linear(np64(a), np64(w), off, np64(bias) if with_bias else None, np64(res) if with_res else None, act)
    out = torch.full((R, N), math.nan, dtype=out_dtype, device=DEV)
    st = status_word()
    got = sg.situ_linear(dev(a), dev(w[0] if dense else w), None if dense else dev(off),
                         bias=dev((bias[0] if dense else bias) if with_bias else None), residual=dev(res if with_res else None),
                         act=act, save_pre=save_pre, out=out, status=st)
    assert st.item() == 0
    if save_pre:
        got, pre = got
        live = ~np.isnan(z)
        ref.near(pre[torch.from_numpy(live).to(DEV)], z[live], (steps_tol(K, mag) + 1.01 * ref.BF16_HALF * np.abs(z))[live], "pre")
    tol = 1.13 * steps_tol(K, mag) + 2e-6 * (1 + np.abs(np.nan_to_num(z)))
    tol = tol + (1.01 * ref.BF16_HALF if out_dtype == BF else 2 * ref.U24) * np.abs(np.nan_to_num(want))
    ref.near(got, want, tol, "out")                    # NaN, as it was, where no expert owns the row


# few rows (weights streamed), tiles of 128 rows, ragged and empty experts, sizes off every tile
LAYOUTS = [1, 7, 8, 9, 33, 64, 65, 200, 300, [0, 1, 0], [3, 0, 12, 1], [40, 17, 9], [128, 129, 0, 1, 255], [1] * 40, [0] * 3,
           [500, 0, 2]]


@pytest.mark.parametrize("counts", LAYOUTS, ids=str)
@pytest.mark.parametrize("N,K", [(8, 8), (264, 72), (1000, 136), (512, 1024)])
def test_forward_shapes(counts, N, K):
    check_fwd(counts, N, K, "none", True, False, BF, False)


@pytest.mark.parametrize("act", list(moe.ACTIVATIONS))
@pytest.mark.parametrize("counts", [5, 150, [3, 0, 12, 1], [128, 0, 129, 7]], ids=str)
@pytest.mark.parametrize("with_bias,with_res,out_dtype,save_pre",
                         [(True, True, BF, True), (False, True, BF, False), (True, False, torch.float32, True),
                          (False, True, torch.float32, False), (False, False, BF, True)])
def test_forward_epilogue(counts, act, with_bias, with_res, out_dtype, save_pre):
    check_fwd(counts, 328, 200, act, with_bias, with_res, out_dtype, save_pre, seed=len(act))


@pytest.mark.parametrize("counts", [[5, 0, 9], [130, 2, 200]], ids=str)
def test_rows_of_no_expert_are_untouched(counts):
    check_fwd(counts, 264, 72, "silu", True, True, BF, False, tail=37)


@pytest.mark.parametrize("R", [37, 400])
def test_no_expert_has_rows(R):
    """Rows, but every expert empty: nothing is written, the weights' gradients are zero."""
    check_fwd([0, 0, 0], 264, 72, "none", True, False, BF, False, tail=R)
    off = torch.zeros(4, dtype=torch.int64, device=DEV)
    z = lambda *s: torch.ones(s, dtype=BF, device=DEV)  # noqa: E731
    for dtype in (torch.float32, BF):
        _, dw, db = sg.situ_linear_bwd(z(R, 264), z(R, 72), z(3, 264, 72), off, dw_dtype=dtype)
        assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("R,E,owner", [(64, 100, 57), (150, 100, 99), (300, 20, 0), (700, 3, 1)])
def test_one_expert_has_all_rows(R, E, owner):
    """The choice of kernel and chunk goes by the average: the worst case against it is still right."""
    counts = [0] * E
    counts[owner] = R
    check_fwd(counts, 72, 136, "silu", True, True, BF, True)
    check_bwd(counts, 72, 136, "none", torch.float32)


def test_more_experts_than_rows():
    counts = ([0, 1, 0, 2, 0, 0, 3] * 147)[:1024]
    check_fwd(counts, 40, 24, "none", True, False, BF, False)
    check_bwd(counts, 40, 24, "none", torch.float32)


def near_rows(got, want, tol):
    assert ((got.double() - want).abs() <= tol).all()


def test_offsets_past_32_bits():
    """out, the weights and the weight gradient each larger than 2^31 elements: places at both ends are right."""
    g = torch.Generator(device=DEV).manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=BF)  # noqa: E731
    R, N, K = 2_200_000, 1000, 8                        # 2.2e9 outputs and residuals
    a, w, res = new(R, K), new(N, K), new(R, N)
    out = sg.situ_linear(a, w, residual=res)
    for rows in (slice(0, 50), slice(R - 50, R), slice(2 ** 31 // N - 25, 2 ** 31 // N + 25)):
        z = a[rows].double() @ w.double().t()
        near_rows(out[rows], z + res[rows].double(), steps_tol(K, a[rows].double().abs() @ w.double().abs().t()) + 1.01 * ref.BF16_HALF * (z + res[rows].double()).abs())
    del a, w, res, out
    E, N, K = 600, 1024, 3584                           # 2.2e9 weights
    w = new(E, N, K)
    for per in (1, 5):                                   # streamed, and tiled
        off = (torch.arange(E + 1, device=DEV) * per)
        a = new(E * per, K)
        out = sg.situ_linear(a, w, off)
        dz = new(E * per, N)
        da, dw, _ = sg.situ_linear_bwd(dz, a, w, off, bias=False)
        for e in (0, 1, 585, E - 1):
            r = slice(e * per, (e + 1) * per)
            W, A, Z = w[e].double(), a[r].double(), dz[r].double()
            near_rows(out[r], A @ W.t(), steps_tol(K, A.abs() @ W.abs().t()) + 1.01 * ref.BF16_HALF * (A @ W.t()).abs())
            near_rows(da[r], Z @ W, steps_tol(N, Z.abs() @ W.abs()) + 1.01 * ref.BF16_HALF * (Z @ W).abs())
            near_rows(dw[e], Z.t() @ A, steps_tol(per, Z.abs().t() @ A.abs()) + 2 * ref.U24 * (Z.t() @ A).abs())


def test_large_values_and_saturation():
    """Activations far from zero: gelu and silu go to 0 on the left and z on the right, nothing turns NaN."""
    K = N = 64
    a = torch.eye(64).to(BF)
    w = torch.linspace(-3e4, 3e4, 64).repeat(64, 1).t().contiguous().to(BF)
    for R in (64, 256):
        x = a.repeat(R // 64, 1)
        for act in ("relu", "silu", "gelu"):
            out = sg.situ_linear(dev(x), dev(w), act=act, out_dtype=torch.float32)
            want = ref.act(np64(x) @ np64(w).T, act)[0]
            ref.near(out, want, 1e-5 * np.abs(want) + 1e-4, act)


def test_nan_stays_in_its_expert():
    """A NaN or inf row, weight or ragged edge of one expert does not reach another's rows or gradients."""
    for counts in ([3, 5, 2], [130, 70, 200]):
        R, N, K = sum(counts), 136, 72
        g, a, w, bias, _ = inputs(R, N, K, 3, 4)
        off = offsets_of(counts)
        rows = slice(int(off[1]), int(off[2]))
        a[rows] = math.nan
        w[1] = math.inf
        dout = torch.randn(R, N, generator=g).to(BF)
        dout[rows] = math.nan
        out = sg.situ_linear(dev(a), dev(w), dev(off), bias=dev(bias))
        da, dw, db = sg.situ_linear_bwd(dev(dout), dev(a), dev(w), dev(off))
        keep = torch.ones(R, dtype=torch.bool)
        keep[rows] = False
        assert torch.isfinite(out[keep.to(DEV)]).all() and torch.isfinite(da[keep.to(DEV)]).all()
        for t in (dw, db):
            assert torch.isfinite(t[0]).all() and torch.isfinite(t[2]).all() and torch.isnan(t[1]).all()


# ---------------------------------------------------------------- gradients

def check_bwd(counts, N, K, act, dw_dtype, seed=0, tail=0):
    dense = isinstance(counts, int)
    counts = [counts] if dense else counts
    R, E = sum(counts) + tail, len(counts)
    g, a, w, _, dout = inputs(R, N, K, E, seed)
    pre = torch.randn(R, N, generator=g).to(BF)
    off = offsets_of(counts)
    want = ref.linear_bwd(np64(dout), np64(a), np64(w), off, np64(pre), act)
    st = status_word()
    da, dw, db = sg.situ_linear_bwd(dev(dout), dev(a), dev(w[0] if dense else w), None if dense else dev(off), act=act,
                                    pre=dev(pre) if act != "none" else None, dw_dtype=dw_dtype, status=st)
    assert st.item() == 0
    dz_off = 1.02 * ref.BF16_HALF + 4e-6 if act != "none" else 0.0     # dz rounded; act' good to 4e-6 of dout
    n = int(off[-1])
    tol = steps_tol(N, want["dam"]) + dz_off * want["dam"] + 1.01 * ref.BF16_HALF * np.abs(np.nan_to_num(want["da"]))
    extra = 0.0
    if act != "none":                                  # act' is good to 4e-6 absolute: of |dout|, not of |dz|
        extra = 4e-6
        W = np.abs(np64(w))
        for e in range(E):
            r = slice(int(off[e]), int(off[e + 1]))
            tol[r] += extra * (np.abs(np64(dout))[r] @ W[e])
    ref.near(da[:n], want["da"][:n], tol[:n], "da")
    rows = max(counts)
    tol = steps_tol(rows, want["dwm"]) + dz_off * want["dwm"] + (1.01 * ref.BF16_HALF if dw_dtype == BF else 2 * ref.U24) * np.abs(want["dw"])
    if extra:
        for e in range(E):
            r = slice(int(off[e]), int(off[e + 1]))
            tol[e] += extra * (np.abs(np64(dout))[r].T @ np.abs(np64(a))[r])
    ref.near(dw[None] if dense else dw, want["dw"], tol, "dw")
    chain = 128 / 8 + 8 + max(64, rows / 128) + 2      # a warp's rows of a piece, the warps, the pieces
    ref.near(db[None] if dense else db, want["db"], (chain * ref.U24 * 1.13 + 4e-6 * (act != "none")) * want["dbm"], "dbias")


@pytest.mark.parametrize("counts", [1, 15, 16, 17, 63, 64, 65, 300, [0, 1, 0], [3, 0, 12, 1], [64, 65, 0, 127, 200], [0, 0],
                                    [1] * 20], ids=str)
@pytest.mark.parametrize("N,K", [(8, 8), (136, 264), (520, 72)])
@pytest.mark.parametrize("dw_dtype", [torch.float32, BF])
def test_gradients(counts, N, K, dw_dtype):
    check_bwd(counts, N, K, "none", dw_dtype)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("counts", [70, [3, 0, 140, 1]], ids=str)
@pytest.mark.parametrize("dw_dtype", [torch.float32, BF])
def test_gradients_through_the_activation(counts, act, dw_dtype):
    check_bwd(counts, 200, 136, act, dw_dtype, tail=9 if not isinstance(counts, int) else 0)


@pytest.mark.parametrize("counts", [4099, [1500, 0, 2600]], ids=str)
def test_long_contraction(counts):
    """Many rows to one weight: the row axis is cut into pieces that are joined in fp32."""
    check_bwd(counts, 136, 264, "none", torch.float32)
    check_bwd(counts, 72, 64, "gelu", BF)


def test_weight_gradient_precision_over_rows():
    """The weight gradient's error does not grow with the rows: below 1e-6 of its norm at 500 and at 9000 rows
    (a sum cut towards zero at each of 560 tensor-core steps would be ten times that)."""
    g = gen(11)
    for R, N, K in ((500, 512, 512), (9000, 2048, 2048)):
        dz, a = torch.randn(R, N, generator=g).to(BF).to(DEV), torch.randn(R, K, generator=g).to(BF).to(DEV)
        _, dw, _ = sg.situ_linear_bwd(dz, a, torch.zeros(N, K, dtype=BF, device=DEV), bias=False, need_da=False)
        want = dz.double().t() @ a.double()
        assert ((dw.double() - want).norm() / want.norm()).item() < 1e-6


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("counts", [[5, 0, 11], [140, 3, 130]], ids=str)
def test_gradient_by_differences(counts, act):
    """Central differences of <out, dout> (fp32 out) in a and w along sign patterns that bf16 holds exactly."""
    R, N, K, E = sum(counts), 40, 24, 3
    g = gen(12)
    a = (torch.randint(-8, 9, (R, K), generator=g) / 8).to(BF)
    w = (torch.randint(-8, 9, (E, N, K), generator=g) / 32).to(BF)
    bias, off = torch.randn(E, N, generator=g) * 0.1, dev(offsets_of(counts))
    dout = torch.randn(R, N, generator=g).to(BF)
    f = lambda a, w: (np64(sg.situ_linear(dev(a.to(BF)), dev(w.to(BF)), off, bias=dev(bias), act=act,  # noqa: E731
                                          out_dtype=torch.float32)) * np64(dout)).sum()
    _, pre = sg.situ_linear(dev(a), dev(w), off, bias=dev(bias), act=act, save_pre=True)
    da, dw, _ = sg.situ_linear_bwd(dev(dout), dev(a), dev(w), off, act=act, pre=pre)
    va, vw = torch.randint(0, 2, (R, K), generator=g) * 2.0 - 1, torch.randint(0, 2, (E, N, K), generator=g) * 2.0 - 1
    offs = off.cpu().numpy()
    _, z, smag = ref.linear(np64(a), np64(w), offs, np64(bias), None, "none")
    adout = np.abs(np64(dout))
    for grad, v, eps, d, plus in (
            (da, va, 2.0 ** -5, ref.linear(np64(va), np64(w), offs, None, None, "none")[0], lambda s: (a.float() + s * va, w.float())),
            (dw, vw, 2.0 ** -6, ref.linear(np64(a), np64(vw), offs, None, None, "none")[0], lambda s: (a.float(), w.float() + s * vw))):
        num = (f(*plus(eps)) - f(*plus(-eps))) / (2 * eps)
        # d = dz/d(step). Differences: third derivative below 2, times d^3 eps^2 / 6; the rounding of out (over eps).
        # Gradient: act' off by act'' (below 1.2) times half an ulp of pre, dz by half an ulp, da by half an ulp
        d, az = np.abs(d), np.abs(z)
        tol = (adout * ((steps_tol(K, smag) * 1.13 + 2e-6 * (1 + az)) / eps)).sum()
        tol += (np.abs(np64(grad)) * ref.BF16_HALF).sum() if grad is da else 1e-5 * (adout * d).sum()
        if act != "none":
            tol += (adout * (d ** 3 * eps ** 2 / 3 + d * (1.2 * ref.BF16_HALF * az + 1.13 * ref.BF16_HALF + 4e-6))).sum()
        assert abs(num - float((np64(grad) * np64(v)).sum())) <= tol


def test_no_rows():
    off = torch.zeros(4, dtype=torch.int64, device=DEV)
    a, w = torch.empty(0, 16, dtype=BF, device=DEV), torch.ones(3, 8, 16, dtype=BF, device=DEV)
    assert sg.situ_linear(a, w, off).shape == (0, 8)
    da, dw, db = sg.situ_linear_bwd(torch.empty(0, 8, dtype=BF, device=DEV), a, w, off)
    assert da.shape == (0, 16) and (dw == 0).all() and (db == 0).all() and dw.shape == (3, 8, 16) and db.shape == (3, 8)


def test_results_repeat():
    counts, N, K = [700, 3, 1500], 200, 264
    g, a, w, bias, dout = inputs(sum(counts), N, K, 3, 1)
    off = dev(offsets_of(counts))
    runs = [[sg.situ_linear(dev(a), dev(w), off, bias=dev(bias)), *sg.situ_linear_bwd(dev(dout), dev(a), dev(w), off)]
            for _ in range(3)]
    assert all(torch.equal(x, y) for other in runs[1:] for x, y in zip(runs[0], other))


def test_another_stream():
    counts, N, K = [70, 3, 150], 200, 264
    g, a, w, bias, dout = inputs(sum(counts), N, K, 3, 1)
    off, a, w, dout = dev(offsets_of(counts)), dev(a), dev(w), dev(dout)
    want = [sg.situ_linear(a, w, off), *sg.situ_linear_bwd(dout, a, w, off)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = torch.zeros_like(a)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(5):
            big = big @ big * 1e-2
        late.copy_(a)
    got = [sg.situ_linear(late, w, off, stream=s), *sg.situ_linear_bwd(dout, late, w, off, stream=s.cuda_stream)]
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_autograd_matches_the_calls():
    g = gen(13)
    counts, N, K = [40, 0, 25], 72, 48
    R = sum(counts)
    off = dev(offsets_of(counts))
    a, w = torch.randn(R, K, generator=g).to(BF).to(DEV).requires_grad_(), (torch.randn(3, N, K, generator=g) / 7).to(BF).to(DEV).requires_grad_()
    bias, res = torch.randn(3, N, generator=g).to(DEV).requires_grad_(), torch.randn(R, N, generator=g).to(BF).to(DEV).requires_grad_()
    dout = torch.randn(R, N, generator=g).to(BF).to(DEV)
    out = moe.linear(a, w, bias, res, off, act="silu")
    out.backward(dout)
    _, pre = sg.situ_linear(a.detach(), w.detach(), off, bias=bias.detach(), act="silu", save_pre=True)
    da, dw, db = sg.situ_linear_bwd(dout, a.detach(), w.detach(), off, act="silu", pre=pre, dw_dtype=BF)
    for got, want in ((a.grad, da), (w.grad, dw), (bias.grad, db), (res.grad, dout)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("needed", [(0,), (1,), (2,), (3,), (0, 3), (1, 2)])
def test_autograd_of_some_inputs(needed, act):
    """Gradients of some of a, w, bias, residual are those of all four, and only they are given."""
    g = gen(14)
    R, N, K = 37, 72, 48
    data = [torch.randn(R, K, generator=g).to(BF), (torch.randn(N, K, generator=g) / 7).to(BF), torch.randn(N, generator=g),
            torch.randn(R, N, generator=g).to(BF)]
    dout = torch.randn(R, N, generator=g).to(BF).to(DEV)
    grads = []
    for some in ((0, 1, 2, 3), needed):
        ins = [t.to(DEV).requires_grad_(i in some) for i, t in enumerate(data)]
        moe.linear(*ins, act=act).backward(dout)
        grads.append([t.grad for t in ins])
    for i, (every, some) in enumerate(zip(*grads)):
        assert torch.equal(some, every) if i in needed else some is None


def test_bounded_waits_time_out_report_and_return():
    """The pair kernels' waits run out on barriers nothing completes, say so, and leave the context usable."""
    status, elapsed = status_word(), torch.zeros(1, dtype=torch.int64, device=DEV)
    moe.selftest_wait_timeout(status, elapsed)
    torch.cuda.synchronize()
    assert status.item() == 1 and 1.5e9 <= elapsed.item() <= 20e9
    check_fwd([200, 3], 264, 72, "none", True, False, BF, False)


def test_refusals():
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    off = torch.zeros(3, dtype=torch.int64, device=DEV)
    for bad in (lambda: sg.situ_linear(z(4, 16, dtype=torch.float32), z(8, 16)), lambda: sg.situ_linear(z(4, 16), z(8, 16), bias=z(8)),
                lambda: sg.situ_linear(z(4, 16), z(2, 8, 16), off.int())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: sg.situ_linear(z(4, 16), z(2, 8, 16)), lambda: sg.situ_linear(z(4, 16), z(8, 16), off),
                lambda: sg.situ_linear(z(4, 16), z(8, 24)), lambda: sg.situ_linear(z(4, 16), z(16, 8).t()),
                lambda: sg.situ_linear(z(4, 16), z(8, 16), act="tanh"), lambda: sg.situ_linear(z(4, 32)[:, ::2], z(8, 16)),
                lambda: sg.situ_linear(z(4, 16), z(8, 16), residual=z(4, 16)), lambda: sg.situ_linear(z(4, 16), z(3, 8, 16), off),
                lambda: sg.situ_linear_bwd(z(4, 8), z(4, 16), z(8, 16), act="gelu")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sg.situ_linear(z(4, 12), z(8, 12)), lambda: sg.situ_linear(z(4, 16), z(12, 16)),
                lambda: sg.situ_linear_bwd(z(4, 12), z(4, 16), z(12, 16)),
                lambda: sg.situ_linear(z(65)[1:].view(4, 16), z(8, 16))):     # off a 16-byte boundary
        with pytest.raises(sg.SituGluError) as err:
            bad()
        assert err.value.status == 1
    a = z(4, 16)
    with pytest.raises(sg.SituGluError) as err:
        sg.situ_linear(a, z(16, 16), out=a)
    assert err.value.status == 2
