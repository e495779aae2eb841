"""Routing, the row plan, dispatch, combine and their gradients on the GPU against the plain float64
definitions.

Tolerances (derived from the arithmetic, not from runs): p is exp(v - m)/Σ in fp32, whose argument is
rounded (|v - m|·2^-24, |v - m| < 40 here), exp and the division are good to 2 ulp, the sum of at most 32
positive terms to 32·2^-24: together below 8e-6 relative. A sum of n products in fp32 is good to
n·2^-24·Σ|terms| whatever its order (n: the longest chain of additions), and storing as bf16 adds half
an ulp, 2^-8 relative (of a value already off by the former: 1 % more is left for it)."""
import itertools
import math

import numpy as np
import pytest
import torch

import bwd_situ_glu_gb300 as sg
from bwd_situ_glu_gb300 import moe
import _moe_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = {torch.bfloat16: 1.01 * ref.BF16_HALF, torch.float32: 2 * ref.U24}
P_TOL = 8e-6


def gen(seed):
    return torch.Generator().manual_seed(seed)


def np64(t):
    return t.detach().cpu().double().numpy()


def make_ids(T, K, E, g, drop=0.0):
    """Distinct experts per token (all of them when K = E), some tokens without any."""
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]) if T else torch.zeros(0, K)
    ids = ids.to(torch.int32).reshape(T, K)
    if drop:
        ids[torch.rand(T, generator=g) < drop] = -1
        ids[torch.rand(T, K, generator=g) < drop / 4] = -1
    return ids


# ---------------------------------------------------------------- routing

def check_route(logits, K, dp=None):
    p, ids = sg.situ_route_topk(logits.to(DEV), K)
    assert p.dtype == torch.float32 and ids.dtype == torch.int32
    want_p, want_ids = ref.route(logits, K)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    ref.near(p, want_p, P_TOL * np.abs(np.nan_to_num(want_p)) + 2.0 ** -126, "p")
    return p, ids


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 896, 16), (3, 7, 7), (17, 32, 32), (9, 33, 32), (5, 100, 6), (64, 896, 16),
                                   (7, 897, 16), (5, 1024, 32), (2, 1023, 1), (33, 112, 8), (4, 256, 2), (3, 512, 9)])
def test_route_matches(T, E, K, dtype):
    check_route((torch.randn(T, E, generator=gen(T * E + K)) * 2).to(dtype), K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K", [(896, 16), (1024, 32), (100, 32), (33, 5)])
def test_route_ties_and_order(E, K, dtype):
    """Ties go to the lower index and rows whose bound leaves many scores still give the same choice."""
    g = gen(E)
    rows = [torch.zeros(E), torch.arange(E).float(), -torch.arange(E).float(),
            torch.randint(0, 3, (E,), generator=g).float(), torch.where(torch.rand(E, generator=g) < 0.5, 0.0, -0.0),
            torch.randint(-2, 2, (E,), generator=g).float() * 1e-30, (torch.arange(E) % 32).float(),
            (torch.arange(E) // 32).float(), torch.full((E,), -3.0e38), torch.full((E,), 3.0e38)]
    check_route(torch.stack(rows).to(dtype), K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K", [(896, 16), (40, 8), (5, 5)])
def test_route_masks(E, K, dtype):
    """-inf is never chosen: rows with all, all but one, or K - 1 scores masked; the lowest finite value is a score."""
    g = gen(K)
    x = torch.randn(8, E, generator=g).to(dtype)
    x[0] = -math.inf
    x[1] = -math.inf
    x[1, E - 1] = 0.5
    x[2, K - 1:] = -math.inf
    x[3] = torch.finfo(dtype).min
    x[4, 1:] = torch.finfo(dtype).min
    x[5, torch.rand(E, generator=g) < 0.9] = -math.inf
    p, ids = check_route(x, K)
    assert (ids[0] == -1).all() and (p[0] == 0).all()
    assert ids[1, 0] == E - 1 and p[1, 0] == 1.0 and (ids[1, 1:] == -1).all()


def test_route_nonfinite():
    """NaN ranks first and makes the token's p NaN; so does a chosen +inf. Other tokens are untouched."""
    x = torch.randn(4, 70, generator=gen(0))
    x[1, 40] = math.nan
    x[2, 3] = math.inf
    x[3, 5], x[3, 6] = -math.nan, -math.inf
    p, ids = sg.situ_route_topk(x.to(DEV), 4)
    assert ids[1, 0] == 40 and ids[2, 0] == 3 and ids[3, 0] == 5
    assert torch.isfinite(p[0]).all() and all(torch.isnan(p[r]).all() for r in (1, 2, 3))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (13, 896, 16), (5, 101, 7), (6, 1024, 32), (4, 32, 32), (9, 12, 3)])
def test_route_bwd(T, E, K, dtype):
    g = gen(T + E)
    x = torch.randn(T, E, generator=g)
    x[0, K // 2 + 1:] = -math.inf if E > 1 else x[0, K // 2 + 1:]
    p, ids = sg.situ_route_topk(x.to(DEV), K)
    dp = torch.randn(T, K, generator=g)
    dp[ids.cpu() < 0] = math.nan                       # places without an expert take no part
    d = sg.situ_route_topk_bwd(ids, p, dp.to(DEV), E, dtype=dtype)
    assert d.dtype == dtype and d.shape == (T, E)
    pn, idn, dpn = np64(p), ids.cpu().numpy(), np64(dp)
    want = ref.route_bwd(pn, idn, dpn, E)
    mag = np.zeros((T, E))                             # p_k(|dp_k| + Σ p|dp|): what the rounding scales with
    for t, k in itertools.product(range(T), range(K)):
        if idn[t, k] >= 0:
            mag[t, idn[t, k]] = pn[t, k] * (abs(dpn[t, k]) + np.nansum(pn[t] * np.abs(dpn[t])))
    ref.near(d, want, 40 * ref.U24 * mag + (HALF[dtype] * np.abs(want) if dtype == torch.bfloat16 else 0), "dlogits")
    # the same dp in row order
    offsets, row_of, src, _ = sg.situ_dispatch_plan(ids, E)
    rows = torch.full((T * K,), math.nan, device=DEV)
    used = src >= 0
    rows[used] = dp.to(DEV).reshape(-1)[src[used].long()]
    assert torch.equal(sg.situ_route_topk_bwd(ids, p, rows, E, dtype=dtype, row_of=row_of), d)


def test_route_gradient_by_differences():
    """Central differences of <dp, p(s)> along random directions, at well separated scores."""
    g = gen(3)
    T, E, K = 6, 50, 5
    s = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float() * 0.125
    dp, v = torch.randn(T, K, generator=g), torch.randn(T, E, generator=g)
    eps = 2.0 ** -6
    plus, _ = sg.situ_route_topk((s + eps * v).to(DEV), K)
    minus, _ = sg.situ_route_topk((s - eps * v).to(DEV), K)
    p, ids = sg.situ_route_topk(s.to(DEV), K)
    d = np64(sg.situ_route_topk_bwd(ids, p, dp.to(DEV), E))
    num = ((np64(plus) - np64(minus)) * np64(dp)).sum(1) / (2 * eps)
    # third derivative of a softmax along v: below 6·|v|³·Σ|dp|, times eps²/6; and the rounding of p over 2·eps
    vmax = float(v.abs().max())
    tol = eps ** 2 * vmax ** 3 * np64(dp).__abs__().sum(1) + P_TOL / eps * np64(dp).__abs__().max()
    ref.near((d * np64(v)).sum(1), num, tol, "directional derivative")


# ---------------------------------------------------------------- the row plan

@pytest.mark.parametrize("T,K,E,drop", [(1, 1, 1, 0), (5, 3, 3, 0.4), (8, 16, 896, 0), (33, 7, 100, 0.2), (1000, 2, 1024, 0.1),
                                        (513, 16, 16, 0), (600, 16, 896, 0.05), (3001, 5, 7, 0.3), (20000, 2, 3, 0.2),
                                        (7000, 16, 64, 0.1)])
def test_plan_matches(T, K, E, drop):
    g = gen(T + E)
    ids = make_ids(min(T, 64), K, E, g, drop).repeat(-(-T // min(T, 64)), 1)[:T].contiguous()
    p = torch.rand(T, K, generator=g)
    offsets, row_of, src, p_rows = sg.situ_dispatch_plan(ids.to(DEV), E, p=p.to(DEV))
    want = ref.plan(ids.numpy(), E)
    for got, w in zip((offsets, row_of, src), want):
        assert np.array_equal(got.cpu().numpy(), w)
    assert offsets.dtype == torch.int64 and row_of.dtype == src.dtype == torch.int32
    want_p = np.where(want[2] >= 0, p.numpy().reshape(-1)[np.maximum(want[2], 0)], np.float32(0))
    assert np.array_equal(p_rows.cpu().numpy(), want_p)


@pytest.mark.parametrize("n", [300, 30000])
def test_plan_odd_ids(n):
    """One expert for all; ids outside the range; an expert repeated within a token; nothing routed at all."""
    for ids in (torch.full((n, 1), 2), torch.full((n, 2), 5), torch.tensor([[0, -7, 2, 1 << 30]] * n),
                torch.full((n, 2), -1), torch.tensor([[3, 3, 0]] * n)):
        ids = ids.to(torch.int32)
        offsets, row_of, src, p_rows = sg.situ_dispatch_plan(ids.to(DEV), 4)
        want = ref.plan(ids.numpy(), 4)
        assert p_rows is None
        for got, w in zip((offsets, row_of, src), want):
            assert np.array_equal(got.cpu().numpy(), w)


def test_plan_no_tokens():
    offsets, row_of, src, p_rows = sg.situ_dispatch_plan(torch.empty(0, 4, dtype=torch.int32, device=DEV), 9,
                                                         p=torch.empty(0, 4, device=DEV))
    assert (offsets == 0).all() and offsets.numel() == 10 and row_of.shape == (0, 4) and src.numel() == 0
    assert p_rows.numel() == 0


# ---------------------------------------------------------------- dispatch and combine

SHAPES = [(1, 1, 1, 1), (5, 3, 4, 7), (4, 2, 9, 8), (3, 16, 20, 1000), (70, 4, 6, 130), (9, 40, 64, 24), (2, 2, 2, 3584),
          (130, 5, 8, 72), (3, 9, 9, 2056)]


def rows_of(T, K, E, g, drop):
    ids = make_ids(T, K, E, g, drop)
    offsets, row_of, _ = ref.plan(ids.numpy(), E)
    return torch.from_numpy(offsets).to(DEV), torch.from_numpy(row_of).to(torch.int32).to(DEV), row_of


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E,D", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.5])
def test_dispatch(T, K, E, D, drop, dtype):
    g = gen(T * D + K)
    offsets, row_dev, row_of = rows_of(T, K, E, g, drop)
    x, w = torch.randn(T, D, generator=g).to(dtype), torch.rand(T, K, generator=g)
    h = sg.situ_dispatch(x.to(DEV), row_dev, offsets)
    assert np.array_equal(np64(h), ref.dispatch(np64(x), row_of, T * K))
    h = sg.situ_dispatch(x.to(DEV), row_dev, offsets, weights=w.to(DEV))
    want = ref.dispatch(np64(x), row_of, T * K, np64(w))
    ref.near(h, want, HALF[dtype] * np.abs(want), "weighted rows")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E,D", SHAPES)
@pytest.mark.parametrize("weighted,with_residual", [(True, False), (False, True)])
def test_combine(T, K, E, D, weighted, with_residual, dtype):
    g = gen(T + D + K)
    _, row_dev, row_of = rows_of(T, K, E, g, 0.3)
    o, w = torch.randn(T * K, D, generator=g).to(dtype), torch.rand(T, K, generator=g)
    r = torch.randn(T, D, generator=g).to(dtype)
    kw = dict(weights=w.to(DEV) if weighted else None, residual=r.to(DEV) if with_residual else None)
    y = sg.situ_combine(o.to(DEV), row_dev, **kw)
    want, mag = ref.combine(np64(o), row_of, np64(w) if weighted else None, np64(r) if with_residual else None)
    tol = (K + 2) * ref.U24 * mag + HALF[dtype] * np.abs(want)
    ref.near(y, want, tol, "y")
    if with_residual:                                  # in place: the residual stream itself
        res = r.to(DEV)
        assert sg.situ_combine(o.to(DEV), row_dev, residual=res, y=res) is res and torch.equal(res, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E,D", SHAPES)
def test_combine_bwd(T, K, E, D, dtype):
    g = gen(3 * T + D + K)
    offsets, row_dev, row_of = rows_of(T, K, E, g, 0.3)
    o, dy, w = torch.randn(T * K, D, generator=g).to(dtype), torch.randn(T, D, generator=g).to(dtype), torch.rand(T, K, generator=g)
    do, dw = sg.situ_combine_bwd(dy.to(DEV), o.to(DEV), row_dev, w.to(DEV), offsets)
    want_do, want_dw, mag = ref.combine_bwd(np64(dy), np64(o), row_of, np64(w))
    ref.near(do, want_do, HALF[dtype] * np.abs(want_do), "do")
    ref.near(dw, want_dw, (D / 256 + 8 + 5 + 8 + 2) * ref.U24 * mag, "dweights")


def test_combine_gradient_by_differences():
    """fp32, weights and rows: central differences of <y, dy> (bilinear, so they are exact but for rounding)."""
    g = gen(8)
    T, K, E, D = 6, 3, 5, 40
    offsets, row_dev, row_of = rows_of(T, K, E, g, 0.3)
    o, w, dy = torch.randn(T * K, D, generator=g), torch.rand(T, K, generator=g), torch.randn(T, D, generator=g)
    do, dw = sg.situ_combine_bwd(dy.to(DEV), o.to(DEV), row_dev, w.to(DEV), offsets)
    loss = lambda o, w: (np64(sg.situ_combine(o.to(DEV), row_dev, weights=w.to(DEV))) * np64(dy)).sum()  # noqa: E731
    mag = float((ref.combine(np.abs(np64(o)), row_of, np64(w))[0] * np.abs(np64(dy))).sum())
    eps = 2.0 ** -3
    for v, grad, args in ((torch.randn(T * K, D, generator=g), do, lambda s, v: (o + s * v, w)),
                          (torch.randn(T, K, generator=g), dw, lambda s, v: (o, w + s * v))):
        num = (loss(*args(eps, v)) - loss(*args(-eps, v))) / (2 * eps)
        assert abs(num - (np64(grad) * np64(v)).sum()) <= 20 * 8 * ref.U24 * mag / eps


def test_offsets_past_32_bits():
    """More than 2^31 elements of rows: tokens at both ends are right."""
    T, K, E, D = 38000, 16, 896, 3584                   # 2.18e9 elements
    g = torch.Generator(device=DEV).manual_seed(1)
    ids = torch.topk(torch.rand(T, E, generator=g, device=DEV), K, dim=1).indices.to(torch.int32)
    offsets, row_of, src, _ = sg.situ_dispatch_plan(ids, E)
    assert torch.equal(src.sort().values, torch.arange(T * K, dtype=torch.int32, device=DEV))
    x = torch.randn(T, D, generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.rand(T, K, generator=g, device=DEV)
    h = sg.situ_dispatch(x, row_of, offsets)
    for r in (slice(0, 40), slice(2 ** 31 // D - 20, 2 ** 31 // D + 20), slice(T * K - 40, T * K)):
        assert torch.equal(h[r], x[(src[r] // K).long()])
    y = sg.situ_combine(h, row_of, weights=w)
    do, dw = sg.situ_combine_bwd(x, h, row_of, w, offsets)
    for t in (0, 1, T // 2, T - 1):
        rows, xt, wt = row_of[t].long(), x[t].double(), w[t].double()
        near = lambda got, want, tol: ((got.double() - want).abs() <= tol).all()  # noqa: E731
        assert near(y[t], xt * wt.sum(), (K + 2) * ref.U24 * (xt.abs() * wt.sum()) + HALF[torch.bfloat16] * (xt * wt.sum()).abs())
        assert near(do[rows], wt[:, None] * xt, HALF[torch.bfloat16] * (wt[:, None] * xt).abs())
        assert near(dw[t], (xt * xt).sum().expand(K), (D / 128 + 8 + 5 + 8 + 2) * ref.U24 * (xt * xt).sum())


def test_rows_out_of_range_are_skipped():
    """row_of entries at or past R, and negative ones, are neither read nor written."""
    o = torch.ones(4, 8, device=DEV)
    row_of = torch.tensor([[0, 4], [3, -5], [1 << 30, 2]], dtype=torch.int32, device=DEV)
    y = sg.situ_combine(o, row_of)
    assert torch.equal(y[:, 0].cpu(), torch.tensor([1.0, 1.0, 1.0]))
    offsets = torch.tensor([0, 4], device=DEV)
    do, dw = sg.situ_combine_bwd(torch.ones(3, 8, device=DEV), o, row_of, torch.ones(3, 2, device=DEV), offsets)
    assert torch.equal(dw.cpu(), torch.tensor([[8.0, 0], [8, 0], [0, 8]]))


def test_masked_values_do_not_leak():
    """NaN and inf in rows that no token has, and in the weights of dropped places, stay out of the results."""
    g = gen(1)
    T, K, E, D = 9, 4, 6, 64
    ids = make_ids(T, K, E, g)
    ids[2] = -1
    ids[5, 1:] = -1
    offsets, row_of, _ = ref.plan(ids.numpy(), E)
    o, w = torch.randn(T * K, D, generator=g), torch.rand(T, K, generator=g)
    o[int(offsets[-1]):] = math.nan
    w[ids < 0] = math.inf
    dev = torch.from_numpy(row_of).to(torch.int32).to(DEV)
    y = sg.situ_combine(o.to(DEV), dev, weights=w.to(DEV))
    assert torch.isfinite(y).all() and (y[2] == 0).all()
    do, dw = sg.situ_combine_bwd(torch.ones(T, D, device=DEV), o.to(DEV), dev, w.to(DEV), torch.from_numpy(offsets).to(DEV))
    assert torch.isfinite(do).all() and torch.isfinite(dw).all() and (dw[2] == 0).all()


def test_unaligned_bases():
    """Views that start off a 16-byte boundary take the element path."""
    T, K, E, D = 7, 3, 5, 64
    g = gen(2)
    offsets, row_dev, row_of = rows_of(T, K, E, g, 0.2)
    buf = torch.randn(T * K * D + 1, generator=g).to(torch.bfloat16).to(DEV)
    o = buf[1:].view(T * K, D)
    w = torch.rand(T, K, generator=g)
    want, mag = ref.combine(np64(o), row_of, np64(w))
    ref.near(sg.situ_combine(o, row_dev, weights=w.to(DEV)), want, 5 * ref.U24 * mag + HALF[torch.bfloat16] * np.abs(want), "y")
    x = buf[1:1 + T * D].view(T, D)
    assert np.array_equal(np64(sg.situ_dispatch(x, row_dev, offsets)), ref.dispatch(np64(x), row_of, T * K))
    logits = torch.randn(5 * 64 + 1, generator=g)
    p, ids = sg.situ_route_topk(logits.to(DEV)[1:].view(5, 64), 6)
    want_p, want_ids = ref.route(logits[1:].view(5, 64), 6)
    assert np.array_equal(ids.cpu().numpy(), want_ids)


def test_no_tokens():
    e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    p, ids = sg.situ_route_topk(e(0, 8), 2)
    assert p.shape == (0, 2) and sg.situ_route_topk_bwd(ids, p, e(0, 2), 8).shape == (0, 8)
    off = torch.zeros(4, dtype=torch.int64, device=DEV)
    row = e(0, 2, dtype=torch.int32)
    assert sg.situ_dispatch(e(0, 8), row, off).shape == (0, 8)
    assert sg.situ_combine(e(0, 8), row).shape == (0, 8)
    do, dw = sg.situ_combine_bwd(e(0, 8), e(0, 8), row, e(0, 2), off)
    assert do.shape == (0, 8) and dw.shape == (0, 2)


def test_results_repeat():
    """No result depends on timing: three runs are bit-identical."""
    g = gen(5)
    T, K, E, D = 900, 16, 64, 264
    ids = make_ids(60, K, E, g, 0.1).repeat(15, 1)
    o, dy, w = torch.randn(T * K, D, generator=g), torch.randn(T, D, generator=g), torch.rand(T, K, generator=g)
    outs = []
    for _ in range(3):
        offsets, row_of, src, p_rows = sg.situ_dispatch_plan(ids.to(DEV), E, p=w.to(DEV))
        outs.append([offsets, row_of, src, p_rows, sg.situ_combine(o.to(DEV), row_of, weights=w.to(DEV)),
                     *sg.situ_combine_bwd(dy.to(DEV), o.to(DEV), row_of, w.to(DEV), offsets)])
    assert all(torch.equal(a, b) for other in outs[1:] for a, b in zip(outs[0], other))


@pytest.mark.parametrize("raw", [False, True])
def test_another_stream(raw):
    """Everything on a side stream (as an object or a raw handle), behind a kernel that is still running there."""
    s = torch.cuda.Stream()
    g = gen(6)
    T, K, E, D = 40, 4, 12, 512
    x, logits = torch.randn(T, D, generator=g).to(DEV), torch.randn(T, E, generator=g).to(DEV)
    p0, ids0 = sg.situ_route_topk(logits, K)
    off0, row0, _, _ = sg.situ_dispatch_plan(ids0, E)
    y0 = sg.situ_combine(sg.situ_dispatch(x, row0, off0), row0, weights=p0)
    torch.cuda.synchronize()
    late = torch.zeros_like(logits)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device=DEV)
        for _ in range(5):
            big = big @ big * 1e-2
        late.copy_(logits)
    h = s.cuda_stream if raw else s
    p, ids = sg.situ_route_topk(late, K, stream=h)
    off, row, _, _ = sg.situ_dispatch_plan(ids, E, stream=h)
    y = sg.situ_combine(sg.situ_dispatch(x, row, off, stream=h), row, weights=p, stream=h)
    s.synchronize()
    assert torch.equal(ids, ids0) and torch.equal(p, p0) and torch.equal(y, y0)


def test_default_stream_handle():
    """Handle 0 is the legacy default stream, as everywhere in the library."""
    x = torch.randn(5, 40, device=DEV)
    for a, b in zip(sg.situ_route_topk(x, 3, stream=0), sg.situ_route_topk(x, 3)):
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_autograd_matches_the_calls():
    """moe.route_topk / moe_dispatch / moe_combine: gradients flow through a routed identity layer like the
    float64 chain of the same choices."""
    g = gen(9)
    T, K, E, D = 20, 3, 7, 48
    x, logits, dy = torch.randn(T, D, generator=g), torch.randn(T, E, generator=g), torch.randn(T, D, generator=g)
    xg, lg = x.to(DEV).requires_grad_(), logits.to(DEV).requires_grad_()
    p, ids = moe.route_topk(lg, K)
    offsets, row_of, _, _ = sg.situ_dispatch_plan(ids, E)
    y = moe.moe_combine(moe.moe_dispatch(xg, row_of, offsets), p, row_of, offsets, residual=xg)
    y.backward(dy.to(DEV))
    xd, ld = x.double().requires_grad_(), logits.double().requires_grad_()
    v, _ = ld.topk(K)
    pd = torch.softmax(v, 1)
    yd = xd + (pd[:, :, None] * xd[:, None, :]).sum(1)
    yd.backward(dy.double())
    ref.near(y, yd.detach().numpy(), 1e-5 * (1 + np.abs(yd.detach().numpy())), "y")
    ref.near(xg.grad, xd.grad.numpy(), 1e-5 * (1 + np.abs(xd.grad.numpy())), "dx")
    # dp is a sum of D products of N(0,1) values: its rounding is below 60·2^-24·Σ|.| with Σ|.| < 2·D
    ref.near(lg.grad, ld.grad.numpy(), 60 * ref.U24 * 2 * D + 1e-5, "dlogits")


def test_autograd_combine_without_weights():
    """The plain sum's gradient is dy at every row of a token, zero at the rows of none."""
    ids = torch.tensor([[0, 2], [1, -1], [2, 0]], dtype=torch.int32, device=DEV)
    offsets, row_of, src, _ = sg.situ_dispatch_plan(ids, 3)
    o = torch.randn(6, 24, generator=gen(10)).to(DEV).requires_grad_()
    dy = torch.randn(3, 24, generator=gen(11)).to(DEV)
    y = moe.moe_combine(o, None, row_of, offsets)
    assert torch.equal(y, sg.situ_combine(o.detach(), row_of))
    y.backward(dy)
    want = torch.zeros_like(dy[:1]).repeat(6, 1)
    for r, s in enumerate(src.tolist()):
        if s >= 0:
            want[r] = dy[s // 2]
    assert torch.equal(o.grad, want)


@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("op", ["route", "dispatch", "combine", "linear"])
def test_second_derivatives_are_refused(op, constant):
    """The gradients are kernels without a derivative of their own: differentiating them raises, it does not
    give zeros."""
    g = gen(12)
    x = torch.randn(4, 16, generator=g).to(DEV)
    offsets, row_of, _, _ = sg.situ_dispatch_plan(torch.tensor([[0], [2], [1], [2]], dtype=torch.int32, device=DEV), 3)
    p = torch.rand(4, 1, generator=g).to(DEV)
    if op == "linear":
        x = x.to(torch.bfloat16)
    x.requires_grad_()
    out = {"route": lambda: moe.route_topk(x, 2)[0], "dispatch": lambda: moe.moe_dispatch(x, row_of, offsets),
           "combine": lambda: moe.moe_combine(x, p.requires_grad_(), row_of, offsets),
           "linear": lambda: moe.linear(x, torch.ones(8, 16, dtype=torch.bfloat16, device=DEV), act="silu")}[op]()
    scale = torch.rand(out.shape, generator=g).to(DEV, out.dtype).requires_grad_(not constant)
    (dx,) = torch.autograd.grad(out, x, scale, create_graph=True)
    if op == "dispatch" and constant:      # linear: the gradient does not depend on x
        (dx * x).sum().backward()
        assert torch.equal(x.grad, dx)
        return
    with pytest.raises(RuntimeError):
        (dx * x).sum().backward()


def test_refusals():
    f = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    off = torch.zeros(5, dtype=torch.int64, device=DEV)
    for bad in (lambda: sg.situ_route_topk(f(2, 8, dtype=torch.float16), 2), lambda: sg.situ_combine(f(4, 8), i(2, 2).long()),
                lambda: sg.situ_route_topk(f(2, 8).cpu().numpy(), 2), lambda: sg.situ_dispatch_plan(i(2, 2).long(), 4)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: sg.situ_route_topk(f(8), 2), lambda: sg.situ_route_topk(f(8, 2).t(), 2),
                lambda: sg.situ_route_topk(f(2, 8).cpu(), 2), lambda: sg.situ_combine(f(4, 8), i(2, 2), weights=f(2, 3)),
                lambda: sg.situ_combine(f(4, 8), i(2, 2), residual=f(2, 9)), lambda: sg.situ_dispatch(f(3, 8), i(2, 2), off),
                lambda: sg.situ_dispatch(f(2, 16)[:, ::2], i(2, 2), off),
                lambda: sg.situ_combine_bwd(f(3, 8), f(4, 8), i(2, 2), f(2, 2), off)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sg.situ_route_topk(f(2, 8), 9), lambda: sg.situ_route_topk(f(2, 8), 0),
                lambda: sg.situ_route_topk(f(2, 1025), 2), lambda: sg.situ_route_topk(f(2, 64), 33),
                lambda: sg.situ_dispatch_plan(i(2, 2), 0), lambda: sg.situ_dispatch_plan(i(2, 2), 1025)):
        with pytest.raises(sg.SituGluError) as err:
            bad()
        assert err.value.status == 1
    o = f(4, 8)
    with pytest.raises(sg.SituGluError) as err:        # an output over an input
        sg.situ_combine(o, i(2, 2), y=o[:2])
    assert err.value.status == 2
