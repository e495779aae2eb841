"""The per-expert / dense product of rows and weights in 8 bits with bias, activation and residual, and its gradients, on
the GPU against float64 sums of the values that the codes stand for.

Tolerances (derived, not fitted). Products of codes and their scales are exact. In the tensor cores' fp32 sums every
addend may be cut at the 23rd bit below the running sum's magnitude: a sum of n terms stays within
(n + 64)·2^-23·Σ|terms|. An activation multiplies that by at most 1.13 (gelu' < 1.129, silu' < 1.1) and is itself
evaluated to 2e-6·(1 + |z|) absolute; a bf16 result adds half a step, 2^-8 relative. dz behind an activation is a bf16
tensor: the products are compared with those of the one that the step back through the activation gives. The bias gradient
is a sum in fp32 of values good to 2e-6 of the gradient that came in."""
import math

import numpy as np
import pytest
import torch

import bwd_situ_glu_gb300 as sg
from bwd_situ_glu_gb300 import fp8, moe
import _fp8_ref as ref8
import _moe_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def np64(t):
    return t.detach().cpu().double().numpy()


def dev(t):
    return None if t is None else t.to(DEV)


def tol_of(n, mag):
    return (n + 64) * 2.0 ** -23 * mag


def offsets_of(counts):
    return torch.tensor([0, *np.cumsum(counts)], dtype=torch.int64)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def inputs(R, N, K, E, seed):
    """Rows and weights whose blocks have scales of their own, over some 20 binades."""
    g = torch.Generator().manual_seed(seed)
    spread = lambda *s: torch.exp2(torch.randint(-10, 11, s, generator=g).float())  # noqa: E731
    a = torch.randn(R, K, generator=g)
    a = (a * spread(R, ref8.blocks(K)).repeat_interleave(128, 1)[:, :K]).to(BF)
    w = torch.randn(E, N, K, generator=g) / math.sqrt(K)
    w = w * spread(E, ref8.blocks(N), ref8.blocks(K)).repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :N, :K]
    return g, a, w.to(BF), torch.randn(E, N, generator=g), torch.randn(R, N, generator=g).to(BF)


def quantised(a, w):
    """(codes and scales of both on the GPU, the values they stand for as float64 arrays)."""
    qa, qw = sg.situ_quant_fp8(dev(a)), sg.situ_quant_fp8(dev(w), block_rows=128)
    return qa, qw, np64(ref8.values(*qa, 1)), np64(ref8.values(*qw, 128))


def check_fwd(counts, N, K, act="none", with_bias=True, with_res=False, out_dtype=BF, save_pre=False, seed=0, tail=0):
    """counts: rows per expert, or an int: dense. tail: rows past the last expert's."""
    dense = isinstance(counts, int)
    counts = [counts] if dense else counts
    R, E = sum(counts) + tail, len(counts)
    g, a, w, bias, res = inputs(R, N, K, E, seed)
    qa, qw, av, wv = quantised(a, w)
    off = offsets_of(counts)
    want, z, mag = ref.linear(av, wv, off, np64(bias) if with_bias else None, np64(res) if with_res else None, act)
    out = torch.full((R, N), math.nan, dtype=out_dtype, device=DEV)
    st = status_word()
    got = sg.situ_linear_fp8(qa, [t[0] for t in qw] if dense else qw, None if dense else dev(off),
                             bias=dev((bias[0] if dense else bias) if with_bias else None), residual=dev(res if with_res else None),
                             act=act, save_pre=save_pre, out=out, status=st)
    assert st.item() == 0
    if save_pre:
        got, pre = got
        live = ~np.isnan(z)
        ref.near(pre[torch.from_numpy(live).to(DEV)], z[live], (tol_of(K, mag) + 1.01 * ref.BF16_HALF * np.abs(z))[live], "pre")
    tol = 1.13 * tol_of(K, mag) + 2e-6 * (1 + np.abs(np.nan_to_num(z)))
    tol = tol + (1.01 * ref.BF16_HALF if out_dtype == BF else 2 * ref.U24) * np.abs(np.nan_to_num(want))
    ref.near(got, want, tol, "out")                    # NaN, as it was, where no expert owns the row


# few rows (weights streamed), tiles of rows, ragged and empty experts, sizes off every tile and scale block
LAYOUTS = [1, 7, 8, 9, 33, 64, 65, 200, 300, 500, [0, 1, 0], [3, 0, 12, 1], [40, 17, 9], [128, 129, 0, 1, 255], [1] * 40, [0] * 3,
           [500, 0, 2], [224, 225, 223]]


@pytest.mark.parametrize("counts", LAYOUTS, ids=str)
@pytest.mark.parametrize("N,K", [(16, 16), (272, 80), (1008, 144), (512, 1024), (400, 2000)])
def test_forward_shapes(counts, N, K):
    check_fwd(counts, N, K)


@pytest.mark.parametrize("act", list(moe.ACTIVATIONS))
@pytest.mark.parametrize("counts", [5, 150, [3, 0, 12, 1], [128, 0, 129, 7]], ids=str)
@pytest.mark.parametrize("with_bias,with_res,out_dtype,save_pre",
                         [(True, True, BF, True), (False, True, BF, False), (True, False, torch.float32, True),
                          (False, True, torch.float32, False), (False, False, BF, True)])
def test_forward_epilogue(counts, act, with_bias, with_res, out_dtype, save_pre):
    check_fwd(counts, 336, 208, act, with_bias, with_res, out_dtype, save_pre, seed=len(act))


@pytest.mark.parametrize("counts", [[5, 0, 9], [130, 2, 200]], ids=str)
def test_rows_of_no_expert_are_untouched(counts):
    check_fwd(counts, 272, 80, "silu", True, True, BF, False, tail=37)


@pytest.mark.parametrize("R", [3, 300])
@pytest.mark.parametrize("ea,ew", [(100, -100), (-100, 100), (120, -126), (-126, 120), (-60, -60), (0, 0), (50, 60)])
def test_scales_far_from_one(R, ea, ew):
    """Scales over the whole range whose products stay in fp32's: 2^(ea + ew) times the same sums, exactly."""
    g = torch.Generator(device=DEV).manual_seed(1)
    codes = lambda *s: torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.int32).to(torch.uint8) & 0xB7  # noqa: E731
    aq, wq = codes(R, 256), codes(272, 256)             # |values| below 2, no NaN
    fill = lambda b, *s: torch.full(s, b + 127, dtype=torch.uint8, device=DEV)  # noqa: E731
    one = sg.situ_linear_fp8((aq, fill(0, R, 2)), (wq, fill(0, 3, 2)), out_dtype=torch.float32)
    got = sg.situ_linear_fp8((aq, fill(ea, R, 2)), (wq, fill(ew, 3, 2)), out_dtype=torch.float32)
    assert torch.equal(got, one * 2.0 ** (ea + ew)) and one.any()


@pytest.mark.parametrize("counts", [6, 300, [3, 2, 4], [130, 2, 200]], ids=str)
def test_nan_stays_in_its_row_or_column(counts):
    """A NaN code or scale of a row reaches that row alone, one of the weights their columns (of their expert)."""
    dense = isinstance(counts, int)
    counts = [counts] if dense else counts
    R, E, N, K = sum(counts), len(counts), 272, 336
    _, a, w, _, _ = inputs(R, N, K, E, 3)
    (aq, as_), (wq, ws), _, _ = quantised(a, w)
    off = offsets_of(counts)
    run = lambda a, w: sg.situ_linear_fp8(a, [t[0] for t in w] if dense else w, None if dense else dev(off))  # noqa: E731
    clean = run((aq, as_), (wq, ws))
    for place, bad in (("row code", (aq.clone(), as_, wq, ws)), ("row scale", (aq, as_.clone(), wq, ws)),
                       ("weight code", (aq, as_, wq.clone(), ws)), ("weight scale", (aq, as_, wq, ws.clone()))):
        nan = torch.zeros(R, N, dtype=torch.bool, device=DEV)
        rows = slice(int(off[-2]), int(off[-1]))
        if place == "row code":
            bad[0][R - 2, K - 1] = 0x7F
            nan[R - 2] = True
        elif place == "row scale":
            bad[1][1, 2] = 255
            nan[1] = True
        elif place == "weight code":
            bad[2][E - 1, 5, 129] = 0xFF
            nan[rows, 5] = True
        else:
            bad[3][E - 1, 2, 1] = 255
            nan[rows, 256:] = True
        got = run(bad[:2], bad[2:])
        assert torch.equal(torch.isnan(got), nan), place
        assert torch.equal(got[~nan], clean[~nan]), place


def check_bwd(counts, N, K, act="none", dw_dtype=torch.float32, seed=0, tail=0):
    dense = isinstance(counts, int)
    counts = [counts] if dense else counts
    R, E = sum(counts) + tail, len(counts)
    g, a, w, _, _ = inputs(R, N, K, E, seed)
    qa, qw, av, wv = quantised(a, w)
    off = offsets_of(counts)
    dout, pre = torch.randn(R, N, generator=g).to(BF), torch.randn(R, N, generator=g).to(BF)
    st = status_word()
    one = lambda t: [x[0] for x in t] if dense else t  # noqa: E731
    da, dw, db = sg.situ_linear_fp8_bwd(dev(dout), qa, one(qw), None if dense else dev(off), act=act,
                                        pre=dev(pre) if act != "none" else None, dw_dtype=dw_dtype, status=st)
    assert st.item() == 0
    full = ref.linear_bwd(np64(dout), av, wv, off, np64(pre), act)
    dz = dev(dout)
    if act != "none":              # the bf16 tensor that both products take
        dz = torch.zeros(R, N, dtype=BF, device=DEV)
        d_pre, d_off, d_out = dev(pre), dev(off), dev(dout)
        assert sg.load().situ_linear_act_bwd(d_out.data_ptr(), d_pre.data_ptr(), moe.ACTIVATIONS[act], d_off.data_ptr(), E,
                                             dz.data_ptr(), None, None, 0, R, N, 0) == 0
        torch.cuda.synchronize()
    dq = np64(ref8.values(*sg.situ_quant_fp8(dz), 1))
    want = ref.linear_bwd(dq, av, wv, off, None, "none")
    live = ~np.isnan(want["da"]).any(1)
    ref.near(da[torch.from_numpy(live).to(DEV)], want["da"][live],
             (tol_of(N, want["dam"]) + 1.01 * ref.BF16_HALF * np.abs(want["da"]))[live], "da")
    want = ref.linear_bwd(np64(dz), av, wv, off, None, "none")
    tol = tol_of(R, want["dwm"]) + (1.01 * ref.BF16_HALF if dw_dtype == BF else 2 * ref.U24) * np.abs(want["dw"])
    ref.near(dw.reshape(E, N, K), want["dw"], tol, "dw")
    ref.near(db.reshape(E, N), full["db"], (R + 8) * 2 * ref.U24 * full["dbm"] * 1.2 + 2e-6 * full["dbm"], "db")


@pytest.mark.parametrize("counts", LAYOUTS, ids=str)
@pytest.mark.parametrize("N,K", [(16, 16), (272, 80), (144, 1008), (1024, 512)])
def test_backward_shapes(counts, N, K):
    check_bwd(counts, N, K)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("counts", [5, 150, [128, 0, 129, 7]], ids=str)
def test_backward_through_activations(counts, act):
    check_bwd(counts, 336, 208, act, BF)


def test_plain_rows_are_quantised_first():
    _, a, w, bias, _ = inputs(70, 272, 400, 1, 5)
    qw = [t[0] for t in sg.situ_quant_fp8(dev(w), block_rows=128)]
    want = sg.situ_linear_fp8(sg.situ_quant_fp8(dev(a)), qw)
    assert torch.equal(sg.situ_linear_fp8(dev(a), qw), want)
    assert torch.equal(sg.situ_linear_fp8(dev(a.float()), qw), want)
