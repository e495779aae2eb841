"""Plain definitions, in float64 on the CPU, of the operators around the expert activation: routing, the
row plan, dispatch, combine and the per-expert linear, with their gradients. Written out one row at a
time where that is the definition; they share nothing with the library."""
import math

import numpy as np
import torch

U24 = 2.0 ** -24            # half an ulp of fp32, relative
BF16_HALF = 2.0 ** -8       # half an ulp of bf16 (7 stored bits), relative to the value: 1 + 2^-8 rounds to 1


def route(logits, K):
    """(p [T,K], ids [T,K]) with ids by descending score, ties to the lower index, -inf never chosen."""
    x = logits.double().numpy()
    T, E = x.shape
    p, ids = np.zeros((T, K)), np.full((T, K), -1, np.int64)
    for t in range(T):
        live = [e for e in range(E) if not x[t, e] == -math.inf]
        live.sort(key=lambda e: (0 if math.isnan(x[t, e]) else 1, 0.0 if math.isnan(x[t, e]) else -x[t, e], e))
        live = live[:K]
        ids[t, :len(live)] = live
        if live:
            s = x[t, live]
            with np.errstate(invalid="ignore"):
                ex = np.exp(s - s[0])
                p[t, :len(live)] = ex / ex.sum() if not np.isnan(s[0]) else np.nan
    return p, ids


def route_bwd(p, ids, dp, E):
    T, K = ids.shape
    d = np.zeros((T, E))
    for t in range(T):
        live = [k for k in range(K) if 0 <= ids[t, k] < E]
        dot = sum(p[t, k] * dp[t, k] for k in live)
        for k in live:
            d[t, ids[t, k]] = p[t, k] * (dp[t, k] - dot)
    return d


def plan(ids, E):
    """(offsets [E+1], row_of [T,K], src [T*K]) by walking the experts and, in each, the pairs in order."""
    T, K = ids.shape
    flat = ids.reshape(-1)
    row_of, src, offsets = np.full(T * K, -1, np.int64), np.full(T * K, -1, np.int64), [0]
    by = {}
    for i, e in enumerate(flat):
        by.setdefault(int(e), []).append(i)
    n = 0
    for e in range(E):
        for i in by.get(e, ()):
            row_of[i], src[n] = n, i
            n += 1
        offsets.append(n)
    return np.array(offsets), row_of.reshape(T, K), src


def dispatch(x, row_of, R, weights=None):
    T, K = row_of.shape
    h = np.zeros((R, x.shape[1]))
    for t in range(T):
        for k in range(K):
            if 0 <= row_of[t, k] < R:
                h[row_of[t, k]] = x[t] * (1.0 if weights is None else weights[t, k])
    return h


def combine(o, row_of, weights=None, residual=None):
    """(y, the sum of absolute values that bounds its rounding)"""
    T, K = row_of.shape
    y = np.zeros((T, o.shape[1])) if residual is None else residual.copy()
    mag = np.abs(y)
    for t in range(T):
        for k in range(K):
            r = row_of[t, k]
            if 0 <= r < o.shape[0]:
                v = o[r] * (1.0 if weights is None else weights[t, k])
                y[t] += v
                mag[t] += np.abs(v)
    return y, mag


def combine_bwd(dy, o, row_of, weights):
    T, K = row_of.shape
    do, dw, mag = np.zeros(o.shape), np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            r = row_of[t, k]
            if 0 <= r < o.shape[0]:
                do[r] = weights[t, k] * dy[t]
                dw[t, k] = float(dy[t] @ o[r])
                mag[t, k] = float(np.abs(dy[t]) @ np.abs(o[r]))
    return do, dw, mag


def act(z, name):
    """(value, derivative) by the definitions."""
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.maximum(z, 0), (z > 0).astype(np.float64)
    if name == "silu":
        s = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        return z * s, s + z * s * (1 - s)
    cdf = 0.5 * torch.special.erfc(torch.from_numpy(-z / math.sqrt(2))).numpy()
    return z * cdf, cdf + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def linear(a, w, offsets, bias, residual, name):
    """(out, z, Σ|a·w|) of a [R,K], w [E,N,K]; NaN in rows of no expert."""
    R, N = a.shape[0], w.shape[1]
    z, mag = np.full((R, N), np.nan), np.zeros((R, N))
    for e in range(w.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        z[r] = a[r] @ w[e].T + (0 if bias is None else bias[e])
        mag[r] = np.abs(a[r]) @ np.abs(w[e]).T + (0 if bias is None else np.abs(bias[e]))
    out = act(z, name)[0]
    return out + (0 if residual is None else residual), z, mag


def linear_bwd(dout, a, w, offsets, pre, name):
    """dict of da, dw, db and the sums of absolute values behind each."""
    dz = dout * (1 if name == "none" else act(pre, name)[1])
    E, N, K = w.shape
    da, dam = np.full(a.shape, np.nan), np.zeros(a.shape)
    dw, dwm, db, dbm = np.zeros(w.shape), np.zeros(w.shape), np.zeros((E, N)), np.zeros((E, N))
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        da[r], dam[r] = dz[r] @ w[e], np.abs(dz[r]) @ np.abs(w[e])
        dw[e], dwm[e] = dz[r].T @ a[r], np.abs(dz[r]).T @ np.abs(a[r])
        db[e], dbm[e] = dz[r].sum(0), np.abs(dout[r]).sum(0)
    return dict(da=da, dam=dam, dw=dw, dwm=dwm, db=db, dbm=dbm, dz=dz)


def near(got, want, tol, what):
    """Every element within its own tolerance; NaN exactly where the reference has NaN."""
    got = got.detach().cpu().double().numpy() if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    want = np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    nan = np.isnan(want)
    assert np.array_equal(nan, np.isnan(got)), f"{what}: NaN in other places"
    off = np.abs(got - want)[~nan] - np.broadcast_to(tol, want.shape)[~nan]
    assert off.size == 0 or off.max() <= 0, f"{what}: {off.max()} past its tolerance, {(off > 0).sum()} of {off.size}"
