"""Cases of the expert layer's operators around the SiTU-GLU kernels: routing, tokens sorted by expert
and back, and the per-expert matrix product with bias, activation and residual.

A case's ``op`` says which operator it takes:

* ``route``    top-k softmax of the router scores (``train``: and the scores' gradient);
* ``sort``     the row plan of the chosen experts and the tokens copied to their rows;
* ``combine``  the weighted rows of a token summed back (``dir`` bwd: the rows' and weights' gradient);
* ``linear``   out = act(a W_eT + b_e) + residual of every row's expert (``dir`` bwd: gradients).

``E = 0`` in a linear case is one weight for all rows. ``drop`` is the share of tokens without a routed
row (padding). Rows of experts are ragged: an expert may have none.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step: the scores of eight sequences' next tokens over all experts
        dict(name="route decode", op="route", T=8, E=896, K=16, dtype="fp32", train=False, drop=0.0),
        # one training micro-batch's router, forward and backward; an odd token count
        dict(name="route train", op="route", T=65537, E=896, K=16, dtype="fp32", train=True, drop=0.0),
        # a padded batch on one expert shard, scores in bf16 (so with ties), some tokens masked out whole
        dict(name="route padded bf16", op="route", T=4099, E=112, K=8, dtype="bf16", train=True, drop=0.25),
        # a decoding step's tokens copied to their experts' rows
        dict(name="sort decode", op="sort", T=8, K=16, E=896, D=3584, dtype="bf16", drop=0.0),
        # a training micro-batch: 262144 rows over 896 experts
        dict(name="sort train", op="sort", T=16384, K=16, E=896, D=3584, dtype="bf16", drop=0.0),
        # a decoding step's expert outputs back into the residual stream
        dict(name="combine decode", op="combine", dir="fwd", T=8, K=16, E=896, D=3584, dtype="bf16", residual=True,
             drop=0.0),
        # a training micro-batch's expert outputs back into token order
        dict(name="combine train", op="combine", dir="fwd", T=16384, K=16, E=896, D=3584, dtype="bf16",
             residual=False, drop=0.0),
        # its gradient: expert output rows and router weights; a padded, odd batch
        dict(name="combine bwd", op="combine", dir="bwd", T=12289, K=16, E=896, D=3584, dtype="bf16",
             residual=False, drop=0.05),
        # a decoding step's down projection on an eighth of the experts: hardly a row each, weights streamed once
        dict(name="linear decode", op="linear", dir="fwd", R=128, E=112, N=3584, K=3072, act="none", bias=True,
             residual=False),
        # a prompt's down projection on the same shard, ragged rows
        dict(name="linear prompt", op="linear", dir="fwd", R=32768, E=112, N=3584, K=3072, act="none", bias=True,
             residual=False),
        # a dense layer for every token: activation and residual in the epilogue, odd rows, sizes off the tiles
        dict(name="linear dense gelu", op="linear", dir="fwd", R=4099, E=0, N=3584, K=1000, act="gelu", bias=True,
             residual=True),
        # training: input, weight (fp32, for the optimizer) and bias gradients of a shard's down projection
        dict(name="linear bwd", op="linear", dir="bwd", R=16384, E=16, N=3584, K=3072, act="none", bias=True,
             residual=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "sort", "combine", "linear"])
    if op == "route":
        E = _log_int(rng, 8, 896)
        return dict(op=op, T=_log_int(rng, 1, 60000), E=E, K=rng.randint(1, min(16, E)),
                    dtype=rng.choice(["fp32", "bf16"]), train=rng.random() < 0.6, drop=rng.choice([0.0, 0.1, 0.5]))
    if op in ("sort", "combine"):
        E, D = _log_int(rng, 8, 896), _log_int(rng, 64, 3584)
        if rng.random() < 0.7:
            D = -(-D // 8) * 8
        K = rng.randint(1, min(16, E))
        c = dict(op=op, T=_log_int(rng, 1, 12000), K=K, E=E, D=D, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                 drop=rng.choice([0.0, 0.1, 0.5]))
        if op == "combine":
            c["dir"] = rng.choice(["fwd", "bwd"])
            c["residual"] = c["dir"] == "fwd" and rng.random() < 0.5
        return c
    E = rng.choice([0, 0, _log_int(rng, 1, 112), _log_int(rng, 1, 112)])
    N, K = (8 * _log_int(rng, 8, 448) for _ in range(2))
    d = rng.choice(["fwd", "fwd", "bwd"])
    return dict(op=op, dir=d, R=_log_int(rng, 1, 16000), E=E, N=N, K=K,
                act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.7,
                residual=d == "fwd" and rng.random() < 0.5)


def _active(c):
    """Experts expected to own a row when R rows fall on E experts."""
    E = max(1, c["E"])
    return E * (1.0 - (1.0 - 1.0 / E) ** c["R"])


def work(c):
    if c["op"] == "route":
        te, tk = c["T"] * c["E"], c["T"] * c["K"]
        b = te * SIZES[c["dtype"]] + 8 * tk
        if c["train"]:
            b += te * SIZES[c["dtype"]] + 4 * tk
        return {"bytes": b, "flops": te + 4 * tk}
    if c["op"] in ("sort", "combine"):
        tk = c["T"] * c["K"]
        rows = tk * (1.0 - c["drop"])
        td, rd = c["T"] * c["D"] * SIZES[c["dtype"]], rows * c["D"] * SIZES[c["dtype"]]
        if c["op"] == "sort":
            return {"bytes": int(8 * tk + td + rd + 12 * tk + 8 * c["E"]), "flops": tk}
        if c["dir"] == "fwd":
            return {"bytes": int(8 * tk + rd + td * (2 if c["residual"] else 1)), "flops": int(2 * rows * c["D"])}
        return {"bytes": int(12 * tk + 2 * rd + td), "flops": int(3 * rows * c["D"])}
    R, N, K = c["R"], c["N"], c["K"]
    E, w = max(1, c["E"]), _active(c) * N * K
    if c["dir"] == "fwd":
        return {"bytes": int(2 * R * (K + N * (2 if c["residual"] else 1)) + 2 * w + (4 * E * N if c["bias"] else 0)),
                "flops": 2 * R * N * K}
    # dout, a and the weights (and the saved pre-activation) in; da, dw of every expert and dbias out
    pre = 2 * R * N if c["act"] != "none" else 0
    return {"bytes": int(2 * R * (N + K) + pre + 2 * w + 2 * R * K
                         + (2 if c["act"] != "none" else 4) * E * N * K + (4 * E * N if c["bias"] else 0)),
            "flops": 4 * R * N * K}


# ---------------------------------------------------------------- inputs

def _experts(g, T, K, E, drop, dev):
    """Distinct experts of each token, some experts liked more than others; -1 throughout for padding."""
    liked = torch.randn(E, generator=g, device=dev) * 0.3
    ids = torch.topk(torch.randn(T, E, generator=g, device=dev) + liked, K, dim=1).indices.to(torch.int32)
    if drop:
        ids[torch.rand(T, generator=g, device=dev) < drop] = -1
    return ids


def _rows(ids, E):
    """(first row of each expert [E + 1], row of each token's k-th expert [T, K] or -1)."""
    T, K = ids.shape
    key = torch.where(ids < 0, E, ids.long()).reshape(-1)
    order = torch.sort(key, stable=True).indices
    row = torch.empty(T * K, dtype=torch.int32, device=ids.device)
    row[order] = torch.arange(T * K, dtype=torch.int32, device=ids.device)
    row[key == E] = -1
    counts = torch.bincount(key, minlength=E + 1)[:E]
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]), row.reshape(T, K)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape, dtype=torch.bfloat16, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(scale)

    s = dict(case=dict(case))
    op = case["op"]
    if op == "route":
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"] = randn(T, E, dtype=torch.float32).to(DTYPES[case["dtype"]])
        if case["drop"]:  # padding tokens have no expert; of the others, some experts are switched off
            s["logits"][torch.rand(T, generator=g, device=dev) < case["drop"]] = -math.inf
            off = torch.rand(T, E, generator=g, device=dev) < 0.1
            s["logits"].masked_fill_(off, -math.inf)
        if case["train"]:
            s["dp"] = randn(T, K, dtype=torch.float32)
    elif op in ("sort", "combine"):
        T, K, E, D, dt = case["T"], case["K"], case["E"], case["D"], DTYPES[case["dtype"]]
        ids = _experts(g, T, K, E, case["drop"], dev)
        s["p"] = torch.softmax(randn(T, K, dtype=torch.float32), dim=1)
        if op == "sort":
            s["ids"], s["x"] = ids, randn(T, D, dtype=dt)
        else:
            s["offsets"], s["row_of"] = _rows(ids, E)
            s["o"] = randn(T * K, D, dtype=dt)
            if case["residual"]:
                s["residual"] = randn(T, D, dtype=dt)
            if case["dir"] == "bwd":
                s["dy"] = randn(T, D, dtype=dt)
    else:
        R, E, N, K = case["R"], case["E"], case["N"], case["K"]
        s["a"] = randn(R, K)
        s["w"] = randn(max(1, E), N, K, scale=1.0 / math.sqrt(K))
        s["offsets"], s["most"] = None, R
        if E:
            liked = torch.softmax(torch.randn(E, generator=g, device=dev) * 0.3, dim=0)
            e = torch.multinomial(liked, R, replacement=True, generator=g)
            counts = torch.bincount(e, minlength=E)
            s["offsets"], s["most"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]), int(counts.max())
        else:
            s["w"] = s["w"][0]
        if case["bias"]:
            s["bias"] = randn(*s["w"].shape[:-1], dtype=torch.float32, scale=0.5)
        if case["residual"]:
            s["residual"] = randn(R, N)
        if case["dir"] == "bwd":
            s["dout"] = randn(R, N)
            if case["act"] != "none":
                s["pre"] = randn(R, N)
    return s


# ---------------------------------------------------------------- the plain forms

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return sig * (1.0 + z * (1.0 - sig))
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    return torch.ones_like(z)


def _plain_route(s, c):
    T, E, K = c["T"], c["E"], c["K"]
    v, ids = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    v, ids = v[:, :K], ids[:, :K]
    live = v > -math.inf
    top = torch.where(live[:, :1], v[:, :1], torch.zeros_like(v[:, :1]))
    ex = torch.exp(v - top)
    p = ex / torch.where(live[:, :1], ex.sum(1, keepdim=True), torch.ones_like(top))
    out = dict(p=p, ids=torch.where(live, ids, -1).to(torch.int32))
    if c["train"]:
        dp = torch.where(live, s["dp"], torch.zeros_like(p))
        d = p * (dp - (p * dp).sum(1, keepdim=True))
        out["dlogits"] = torch.zeros(T, E, device=d.device).scatter_(1, ids, d).to(s["logits"].dtype)
    return out


def _plain_sort(s, c):
    T, K, E = c["T"], c["K"], c["E"]
    offsets, row_of = _rows(s["ids"], E)
    flat = row_of.reshape(-1)
    live = flat >= 0
    src = torch.full((T * K,), -1, dtype=torch.int32, device=flat.device)
    at = flat[live].long()
    src[at] = torch.arange(T * K, dtype=torch.int32, device=flat.device)[live]
    used = src >= 0
    p_rows = torch.where(used, s["p"].reshape(-1)[src.clamp(min=0).long()], 0.0)
    h = s["x"][torch.div(src.clamp(min=0), K, rounding_mode="floor").long()] * used[:, None].to(s["x"].dtype)
    return dict(offsets=offsets, row_of=row_of, src=src, p_rows=p_rows, h=h)


def _plain_combine(s, c):
    row = s["row_of"].long()
    live = row >= 0
    w = s["p"] * live
    o = s["o"].float()[row.clamp(min=0).reshape(-1)].reshape(*row.shape, -1)
    if c["dir"] == "fwd":
        y = (o * w[:, :, None]).sum(1)
        if "residual" in s:
            y = y + s["residual"].float()
        return dict(y=y.to(s["o"].dtype))
    dy = s["dy"].float()
    dp = (o * dy[:, None, :]).sum(2) * live
    do = torch.zeros(s["o"].shape, device=o.device)
    do[row[live]] = (dy[:, None, :] * w[:, :, None])[live]
    return dict(do=do.to(s["o"].dtype), dp=dp)


def _padded(x, offsets, most):
    """[rows, C] of ragged experts -> [E, most, C], zeros past an expert's rows."""
    at = offsets[:-1, None] + torch.arange(most, device=x.device)
    live = at < offsets[1:, None]
    return x[at.clamp(max=max(0, x.shape[0] - 1))] * live[:, :, None]


def _rows_back(x, offsets, R):
    """[E, most, C] -> [R, C]."""
    r = torch.arange(R, device=x.device)
    e = torch.searchsorted(offsets, r, right=True) - 1
    return x[e, r - offsets[e]]


def _plain_linear(s, c):
    R, off, a, w = c["R"], s["offsets"], s["a"].float(), s["w"].float()
    if c["dir"] == "fwd":
        if off is None:
            z = a @ w.t()
            z = z + s["bias"] if c["bias"] else z
        else:
            z = torch.bmm(_padded(a, off, s["most"]), w.transpose(1, 2))
            z = _rows_back(z + s["bias"][:, None, :] if c["bias"] else z, off, R)
        y = _act(z, c["act"])
        return dict(out=(y + s["residual"].float() if c["residual"] else y).to(torch.bfloat16))
    dz = s["dout"].float()
    dw_type = torch.float32
    if c["act"] != "none":
        dz, dw_type = dz * _act_grad(s["pre"].float(), c["act"]), torch.bfloat16
    if off is None:
        da, dw, db = dz @ w, dz.t() @ a, dz.sum(0)
    else:
        dz = _padded(dz, off, s["most"])
        da = _rows_back(torch.bmm(dz, w), off, R)
        dw, db = torch.bmm(dz.transpose(1, 2), _padded(a, off, s["most"])), dz.sum(1)
    out = dict(da=da.to(torch.bfloat16), dw=dw.to(dw_type))
    if c["bias"]:
        out["dbias"] = db
    return out


# ---------------------------------------------------------------- the framework's operators

def _own(s, c):
    import bwd_situ_glu_gb300 as sg
    op = c["op"]
    if op == "route":
        p, ids = sg.situ_route_topk(s["logits"], c["K"])
        out = dict(p=p, ids=ids)
        if c["train"]:
            out["dlogits"] = sg.situ_route_topk_bwd(ids, p, s["dp"], c["E"], dtype=s["logits"].dtype)
        return out
    if op == "sort":
        offsets, row_of, src, p_rows = sg.situ_dispatch_plan(s["ids"], c["E"], p=s["p"])
        h = sg.situ_dispatch(s["x"], row_of, offsets)
        return dict(offsets=offsets, row_of=row_of, src=src, p_rows=p_rows, h=h)
    if op == "combine":
        if c["dir"] == "fwd":
            return dict(y=sg.situ_combine(s["o"], s["row_of"], weights=s["p"], residual=s.get("residual")))
        do, dp = sg.situ_combine_bwd(s["dy"], s["o"], s["row_of"], s["p"], s["offsets"])
        return dict(do=do, dp=dp)
    if c["dir"] == "fwd":
        return dict(out=sg.situ_linear(s["a"], s["w"], expert_offsets=s["offsets"], bias=s.get("bias"),
                                       residual=s.get("residual"), act=c["act"]))
    # fp32 weight gradients where the rounding of dz does not come first, bf16 ones behind an activation
    dw_dtype = torch.float32 if c["act"] == "none" else torch.bfloat16
    da, dw, dbias = sg.situ_linear_bwd(s["dout"], s["a"], s["w"], expert_offsets=s["offsets"], act=c["act"],
                                       pre=s.get("pre"), dw_dtype=dw_dtype, bias=c["bias"])
    out = dict(da=da, dw=dw)
    if c["bias"]:
        out["dbias"] = dbias
    return out


_PLAIN = {"route": _plain_route, "sort": _plain_sort, "combine": _plain_combine, "linear": _plain_linear}


def run(state):
    c = state["case"]
    return _own(state, c) if own else _PLAIN[c["op"]](state, c)


# ---------------------------------------------------------------- 64 bits

def _exact_act(z, act):
    """(activation, its derivative) in float64."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "route":
        x = s["logits"].cpu().double().numpy()
        # the k-th place goes to the largest score left, of equal ones to the first
        order = np.argsort(-x, axis=1, kind="stable")[:, :c["K"]]
        v = np.take_along_axis(x, order, 1)
        live = np.isfinite(v)
        ex = np.where(live, np.exp(np.where(live, v - np.where(live[:, :1], v[:, :1], 0.0), 0.0)), 0.0)
        p = ex / np.maximum(ex.sum(1, keepdims=True), 1e-300)
        out = dict(p=p, ids=None)
        if c["train"]:
            dp = s["dp"].cpu().double().numpy() * live
            d = np.zeros_like(x)
            np.put_along_axis(d, order, p * (dp - (p * dp).sum(1, keepdims=True)), 1)
            out["dlogits"] = d
        return out
    if op == "sort":
        flat = s["ids"].reshape(-1).cpu().numpy()
        live = np.flatnonzero((flat >= 0) & (flat < c["E"]))
        src = live[np.lexsort((live, flat[live]))]
        p, h = np.zeros(flat.size), torch.zeros(flat.size, c["D"], dtype=torch.float64, device="cuda")
        p[:src.size] = s["p"].reshape(-1).cpu().double().numpy()[src]
        h[:src.size] = s["x"].double()[torch.from_numpy(src // c["K"]).cuda()]
        return dict(offsets=None, row_of=None, src=None, p_rows=p, h=h)
    if op == "combine":
        w, row = s["p"].double(), s["row_of"].long()
        if c["dir"] == "fwd":
            y = torch.zeros(c["T"], c["D"], dtype=torch.float64, device="cuda")
            for k in range(c["K"]):
                t = torch.nonzero(row[:, k] >= 0)[:, 0]
                y[t] += w[t, k, None] * s["o"][row[t, k]].double()
            return dict(y=y + s["residual"].double() if c["residual"] else y)
        do = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
        dp = torch.zeros(c["T"], c["K"], dtype=torch.float64, device="cuda")
        for k in range(c["K"]):
            t = torch.nonzero(row[:, k] >= 0)[:, 0]
            dy = s["dy"][t].double()
            do[row[t, k]] = w[t, k, None] * dy
            dp[t, k] = torch.einsum("td,td->t", dy, s["o"][row[t, k]].double())
        return dict(do=do, dp=dp)
    off = s["offsets"].tolist() if c["E"] else [0, c["R"]]
    W = s["w"] if c["E"] else s["w"][None]
    b = s["bias"].reshape(len(W), -1).double() if c["bias"] else None
    if c["dir"] == "fwd":
        out = torch.empty(c["R"], c["N"], dtype=torch.float64, device="cuda")
        for e in range(len(W)):
            r = slice(off[e], off[e + 1])
            z = s["a"][r].double() @ W[e].double().t()
            out[r] = _exact_act(z + b[e] if c["bias"] else z, c["act"])[0]
        return dict(out=out + s["residual"].double() if c["residual"] else out)
    da = torch.empty(c["R"], c["K"], dtype=torch.float64, device="cuda")
    dw = torch.empty(W.shape, dtype=torch.float64, device="cuda")
    db = torch.empty(W.shape[:2], dtype=torch.float64, device="cuda")
    for e in range(len(W)):
        r = slice(off[e], off[e + 1])
        dz = s["dout"][r].double()
        if c["act"] != "none":
            dz = dz * _exact_act(s["pre"][r].double(), c["act"])[1]
        da[r], dw[e], db[e] = dz @ W[e].double(), dz.t() @ s["a"][r].double(), dz.sum(0)
    out = dict(da=da, dw=dw if c["E"] else dw[0])
    if c["bias"]:
        out["dbias"] = db if c["E"] else db[0]
    return out
