"""Cases of the expert layer's training in 8 bits: block-scaled quantisation, the per-expert (or dense)
product of quantised rows and weights with its gradients, and the AdamW step over many tensors.

A case's ``op`` says which operator it takes:

* ``quant``   E4M3 codes and power-of-two scales of blocks of 128 (``block`` 1: of a row, 128: 128 x 128 of a weight);
* ``linear``  out = act(Q(a) W_eT + b_e) + residual of every row's expert, W in 8 bits, a quantised within the pass
  (``dir`` bwd: the gradients from dout and the saved 8-bit rows);
* ``adamw``   one AdamW step over many tensors, states in fp32 or in 8 bits (E4M3 with a scale for each 128).

``E = 0`` in a linear case is one weight for all rows. Rows of experts are ragged: an expert may have none.

The scale of a block is 2^(b - 127) with the least byte b >= 1 for which every finite value is at most 448 times it; a
value's code is the nearest E4M3 number to value / scale (ties to even), NaN for one that is not finite. A state in 8
bits is rounded up or down at random, with the mean kept: the 16 random bits come from the seed and the element's place.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp32": 4}
BLOCK = 128
HYPER = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step: the rows of eight sequences before a product in 8 bits
        dict(name="quant decode", op="quant", E=1, R=8, D=3584, dtype="bf16", block=1),
        # a training micro-batch's rows; an odd count
        dict(name="quant rows", op="quant", E=1, R=65537, D=3584, dtype="bf16", block=1),
        # after an optimizer step: a shard's weights from their fp32 masters
        dict(name="quant weights", op="quant", E=56, R=3584, D=2048, dtype="fp32", block=128),
        # one token through one dense weight: latency
        dict(name="linear token", op="linear", dir="fwd", R=1, E=0, N=3584, K=3584, act="none", bias=False,
             residual=False),
        # a decoding step's down projection on an eighth of the experts: hardly a row each, weights streamed once
        dict(name="linear decode", op="linear", dir="fwd", R=128, E=112, N=3584, K=2048, act="none", bias=True,
             residual=False),
        # a prompt's down projection on the same shard, ragged rows
        dict(name="linear prompt", op="linear", dir="fwd", R=32768, E=112, N=3584, K=2048, act="none", bias=True,
             residual=False),
        # a dense layer for every token of a training micro-batch; an odd count
        dict(name="linear dense", op="linear", dir="fwd", R=16385, E=0, N=3584, K=3584, act="none", bias=False,
             residual=False),
        # activation and residual in the epilogue, odd rows, a contraction that ends inside a block
        dict(name="linear dense gelu", op="linear", dir="fwd", R=4099, E=0, N=3584, K=1008, act="gelu", bias=True,
             residual=True),
        # training: input, weight (fp32, for the optimizer) and bias gradients of a shard's down projection
        dict(name="linear bwd", op="linear", dir="bwd", R=16384, E=16, N=3584, K=2048, act="none", bias=True,
             residual=False),
        # the small tensors of a few layers (norms, biases, router rows): many, odd, fp32 states
        dict(name="adamw small", op="adamw", tensors=64, least=100, most=20000, sizes=1, state="fp32", grad="fp32",
             work=False, clip=False),
        # a shard's parameters with fp32 states, fp32 gradients scaled by a clip factor, bf16 working copies
        dict(name="adamw fp32", op="adamw", tensors=16, least=4000000, most=32000000, sizes=2, state="fp32",
             grad="fp32", work=True, clip=True),
        # the same with states in 8 bits and bf16 gradients
        dict(name="adamw fp8", op="adamw", tensors=16, least=4000000, most=32000000, sizes=2, state="fp8",
             grad="bf16", work=True, clip=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "adamw"])
    if op == "quant":
        block = rng.choice([1, 1, 128])
        D = _log_int(rng, 16, 7168)
        if rng.random() < 0.7:
            D = -(-D // 16) * 16
        if block == 1:
            return dict(op=op, E=1, R=_log_int(rng, 1, 30000), D=D, dtype=rng.choice(["bf16", "bf16", "fp32"]), block=1)
        return dict(op=op, E=_log_int(rng, 1, 16), R=_log_int(rng, 16, 3584), D=D, dtype=rng.choice(["bf16", "fp32"]),
                    block=128)
    if op == "adamw":
        most = _log_int(rng, 200, 8000000)
        return dict(op=op, tensors=_log_int(rng, 1, 60), least=max(1, most // _log_int(rng, 1, 200)), most=most,
                    sizes=rng.randint(0, 1000000), state=rng.choice(["fp32", "fp8", "fp8"]),
                    grad=rng.choice(["fp32", "bf16"]), work=rng.random() < 0.6, clip=rng.random() < 0.5)
    E = rng.choice([0, 0, _log_int(rng, 1, 112), _log_int(rng, 1, 112)])
    N, K = (16 * _log_int(rng, 2, 224) for _ in range(2))
    d = rng.choice(["fwd", "fwd", "bwd"])
    return dict(op=op, dir=d, R=_log_int(rng, 1, 16000), E=E, N=N, K=K,
                act=rng.choice(["none", "none", "relu", "silu", "gelu"]), bias=rng.random() < 0.7,
                residual=d == "fwd" and rng.random() < 0.5)


def _blocks(n):
    return -(-n // BLOCK)


def _sizes(c):
    r = random.Random(c["sizes"])
    return [_log_int(r, c["least"], c["most"]) for _ in range(c["tensors"])]


def work(c):
    if c["op"] == "quant":
        n = c["E"] * c["R"] * c["D"]
        scales = c["E"] * (c["R"] if c["block"] == 1 else _blocks(c["R"])) * _blocks(c["D"])
        return {"bytes": n * (SIZES[c["dtype"]] + 1) + scales, "flops": 2 * n}
    if c["op"] == "adamw":
        n = sum(_sizes(c))
        state = 16 if c["state"] == "fp32" else 4 + 4 / BLOCK
        return {"bytes": int(n * (8 + SIZES[c["grad"]] + state + (2 if c["work"] else 0))), "flops": 14 * n}
    R, N, K = c["R"], c["N"], c["K"]
    E = max(1, c["E"])
    w = E * (1.0 - (1.0 - 1.0 / E) ** R) * N * K         # weights of the experts expected to own a row
    if c["dir"] == "fwd":
        return {"bytes": int(2 * R * (K + N * (2 if c["residual"] else 1)) + w + (4 * E * N if c["bias"] else 0)),
                "flops": 2 * R * N * K}
    # dout (and the value before the activation), the rows and weights in 8 bits in; da, dw of every expert and dbias out
    pre = 2 * R * N if c["act"] != "none" else 0
    return {"bytes": int(2 * R * N + pre + R * K + w + 2 * R * K + (2 if c["act"] != "none" else 4) * E * N * K
                         + (4 * E * N if c["bias"] else 0)),
            "flops": 4 * R * N * K}


# ---------------------------------------------------------------- the 8-bit format, plain

def _scale_bytes(amax):
    """Least byte b in 1 .. 254 with amax <= 448 * 2^(b - 127): 448 is 1.75 * 2^8, and the byte follows from the bits."""
    bits = amax.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=1)


def _two_to(bytes_):
    """2^(b - 127) in fp32, b in 1 .. 254."""
    return (bytes_.int() << 23).view(torch.float32)


def _finite_max(x, dims):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(dims, keepdim=True)


def _in_blocks(x, rows):
    """[E, R, D] -> [E, R / rows, rows, D / 128, 128], padded with zeros."""
    E, R, D = x.shape
    x = torch.nn.functional.pad(x, (0, _blocks(D) * BLOCK - D, 0, -(-R // rows) * rows - R))
    return x.reshape(E, -(-R // rows), rows, _blocks(D), BLOCK)


def _quantise(x, rows):
    """Codes (float8_e4m3fn [E, R, D]) and scale bytes (uint8 [E, R / rows, D / 128]) of x [E, R, D]."""
    E, R, D = x.shape
    x = _in_blocks(x.float(), rows)
    b = _scale_bytes(_finite_max(x, (2, 4)))
    y = (x * _two_to(254 - b)).to(torch.float8_e4m3fn)
    codes = y.reshape(E, x.shape[1] * rows, -1)[:, :R, :D].contiguous()
    return codes, b.to(torch.uint8).reshape(E, x.shape[1], x.shape[3])


def _values(codes, scales, rows):
    """What codes and scale bytes stand for, in fp32 [E, R, D]."""
    E, R, D = codes.shape
    x = _in_blocks(codes.float(), rows) * _two_to(scales)[:, :, None, :, None]
    return x.reshape(E, x.shape[1] * rows, -1)[:, :R, :D]


# ---------------------------------------------------------------- inputs

def _padded_sizes(c):
    """(sizes, first element of each in one flat buffer, its length): every tensor begins at a multiple of 128."""
    sizes, at, first = _sizes(c), 0, []
    for n in sizes:
        first.append(at)
        at += _blocks(n) * BLOCK
    return sizes, first, at


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape, dtype=torch.bfloat16, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(scale)

    c, s = case, dict(case=dict(case))
    if c["op"] == "quant":
        x = randn(c["E"], c["R"], c["D"], dtype=DTYPES[c["dtype"]])
        if c["block"] == 1:        # rows of different sizes, a few rows of zeros (padding) and large values in a channel
            x *= torch.exp(torch.randn(1, c["R"], 1, generator=g, device=dev)).to(x.dtype)
            x *= (torch.rand(1, c["R"], 1, generator=g, device=dev) > 0.02).to(x.dtype)
            x[:, :, c["D"] // 3] *= 30.0
        else:
            x *= 0.02
        s["x"] = x[0] if c["block"] == 1 else x
        return s
    if c["op"] == "adamw":
        sizes, first, total = _padded_sizes(c)
        live = torch.zeros(total, dtype=torch.bool, device=dev)
        for n, at in zip(sizes, first):
            live[at:at + n] = True
        rows = torch.rand(_blocks(total), generator=g, device=dev) > 0.05     # rows that no token reached: no gradient
        grad = randn(total, dtype=DTYPES[c["grad"]], scale=1e-3) * live
        grad.view(-1, BLOCK).mul_(rows[:, None])
        s["w"] = randn(total, dtype=torch.float32, scale=0.02) * live
        m, sv = randn(total, dtype=torch.float32, scale=3e-4), randn(total, dtype=torch.float32, scale=5e-4).abs_() + 5e-4
        m, sv = m * live, sv * live
        if c["state"] == "fp8":
            m, ms = _quantise(m.view(1, -1, BLOCK), 1)
            sv, vs = _quantise(sv.view(1, -1, BLOCK), 1)
            s["m"], s["v"] = m.view(torch.uint8).reshape(-1), sv.view(torch.uint8).reshape(-1)
            s["ms"], s["vs"] = ms.reshape(-1), vs.reshape(-1)
        else:
            s["m"], s["v"] = m, sv * sv
        s["g"] = grad
        if c["work"]:
            s["work"] = s["w"].to(torch.bfloat16)
        if c["clip"]:
            s["clip"] = torch.rand(1, generator=g, device=dev) * 0.5 + 0.5
        s["step"] = 1000 + int(seed) % 1000

        def views(t, per=1):
            return [t[at // per:(at + n + per - 1) // per] for n, at in zip(sizes, first)]
        s["grads"] = views(grad)
        if own:            # the optimizer object that a program keeps
            import bwd_situ_glu_gb300 as sg
            eight = c["state"] == "fp8"
            s["plan"] = sg.AdamWPlan(views(s["w"]), views(s["m"]), views(s["v"]),
                                     m_scales=views(s["ms"], BLOCK) if eight else None,
                                     v_scales=views(s["vs"], BLOCK) if eight else None,
                                     work=views(s["work"]) if c["work"] else None)
        return s
    R, E, N, K = c["R"], c["E"], c["N"], c["K"]
    w = randn(max(1, E), N, K, scale=1.0 / math.sqrt(K))
    codes, scales = zip(*(_quantise(w[i:i + 8], BLOCK) for i in range(0, max(1, E), 8)))
    s["wq"], s["ws"] = torch.cat(codes).view(torch.uint8), torch.cat(scales)
    a = randn(R, K)
    s["offsets"], s["most"] = None, R
    if E:
        liked = torch.softmax(torch.randn(E, generator=g, device=dev) * 0.3, dim=0)
        e = torch.multinomial(liked, R, replacement=True, generator=g)
        counts = torch.bincount(e, minlength=E)
        s["offsets"], s["most"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]), int(counts.max())
    else:
        s["wq"], s["ws"] = s["wq"][0], s["ws"][0]
    if c["bias"]:
        s["bias"] = randn(*s["wq"].shape[:-1], dtype=torch.float32, scale=0.5)
    if c["residual"]:
        s["residual"] = randn(R, N)
    if c["dir"] == "fwd":
        s["a"] = a
    else:                  # what the forward kept: the rows in 8 bits and, behind an activation, the value before it
        codes, scales = _quantise(a[None], 1)
        s["aq"], s["as"] = codes[0].view(torch.uint8), scales[0]
        s["dout"] = randn(R, N)
        if c["act"] != "none":
            s["pre"] = randn(R, N)
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_quant(s, c):
    codes, scales = _quantise(s["x"][None] if c["block"] == 1 else s["x"], c["block"])
    return dict(codes=codes[0], scales=scales[0]) if c["block"] == 1 else dict(codes=codes, scales=scales)


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


def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn)


def _plain_linear(s, c):
    R, off = c["R"], s["offsets"]
    w = _values(_e4m3(s["wq"]).reshape(-1, c["N"], c["K"]), s["ws"].reshape(-1, _blocks(c["N"]), _blocks(c["K"])), BLOCK)
    if c["dir"] == "fwd":
        a = _values(*_quantise(s["a"][None], 1), 1)[0]
        if off is None:
            z = a @ w[0].t()
            z = z + s["bias"] if c["bias"] else z
        else:
            z = torch.bmm(_padded(a, off, s["most"]), w.transpose(1, 2))
            z = _rows_back(z + s["bias"][:, None, :] if c["bias"] else z, off, R)
        y = _act(z, c["act"])
        return dict(out=(y + s["residual"].float() if c["residual"] else y).to(torch.bfloat16))
    # the gradient behind an activation is a bf16 tensor; da takes it in 8 bits, dw the rows that the forward used
    dz, dw_type = s["dout"], torch.float32
    if c["act"] != "none":
        dz, dw_type = dz.float() * _act_grad(s["pre"].float(), c["act"]), torch.bfloat16
    db = dz.float()
    dz = dz.to(torch.bfloat16)
    dq = _values(*_quantise(dz[None], 1), 1)[0]
    a, dz = _values(_e4m3(s["aq"])[None], s["as"][None], 1)[0], dz.float()
    if off is None:
        da, dw, db = dq @ w[0], dz.t() @ a, db.sum(0)
    else:
        da = _rows_back(torch.bmm(_padded(dq, off, s["most"]), w), off, R)
        dw = torch.bmm(_padded(dz, off, s["most"]).transpose(1, 2), _padded(a, off, s["most"]))
        db = _padded(db, off, s["most"]).sum(1)
    out = dict(da=da.to(torch.bfloat16), dw=dw.to(dw_type))
    if c["bias"]:
        out["dbias"] = db
    return out


def _f32(x):
    """x rounded to fp32, as a number."""
    return torch.tensor(x, dtype=torch.float64).to(torch.float32).item()


def _coefficients(step):
    h = HYPER
    return dict(b1=_f32(h["beta1"]), b2=_f32(h["beta2"]), c1=_f32(1.0 - h["beta1"]), c2=_f32(1.0 - h["beta2"]),
                s=_f32(h["lr"] / (1.0 - h["beta1"] ** step)), r=_f32(1.0 / math.sqrt(1.0 - h["beta2"] ** step)),
                eps=_f32(h["eps"]), d=_f32(1.0 - h["lr"] * h["weight_decay"]))


def _mix(x):
    """A mixing of 32 bits, held in int64: shifts and multiplications by the fractions of the golden ratio and of sqrt 2."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _places(c, dev):
    """Each element's index within its tensor, over the flat buffer."""
    sizes, first, total = _padded_sizes(c)
    first = torch.tensor(first, device=dev)
    at = torch.arange(total, device=dev)
    return at - first[torch.searchsorted(first, at, right=True) - 1]


def _random_bits(at, seed):
    """32 random bits of each place (below 2^32) for one seed."""
    key = _mix(torch.tensor((seed * 0x9E3779B1) & 0xFFFFFFFF, device=at.device))
    return _mix((at + key) & 0xFFFFFFFF)


def _round_at_random(x, bits16):
    """Codes (uint8) and scale bytes of x in blocks of 128: as fp32 with its exponent moved to E4M3's, a code is the bits
    above the lowest 20, after the addition of 20 random ones (16, and four zeros)."""
    blocks = x.view(-1, BLOCK)
    b = _scale_bytes(_finite_max(blocks, 1))
    y = (blocks * _two_to(254 - b)).reshape(-1)
    code = ((y.abs() * 2.0 ** -120).view(torch.int32) + (bits16.int() << 4)) >> 20
    code = torch.where(torch.isfinite(y), code.clamp(max=0x7E), 0x7F)
    return code, y, b.to(torch.uint8).reshape(-1)


def _plain_adamw(s, c):
    k = _coefficients(s["step"])
    w, g = s["w"], s["g"].float()
    if c["clip"]:
        g = g * s["clip"]
    eight = c["state"] == "fp8"
    if eight:
        m = (_e4m3(s["m"]).float().view(-1, BLOCK) * _two_to(s["ms"])[:, None]).reshape(-1)
        v = (_e4m3(s["v"]).float().view(-1, BLOCK) * _two_to(s["vs"])[:, None]).reshape(-1)
        v = v * v
    else:
        m, v = s["m"], s["v"]
    m1 = k["b1"] * m + k["c1"] * g
    v1 = k["b2"] * v + k["c2"] * (g * g)
    root = torch.sqrt(v1)
    q = root * k["r"] + k["eps"]
    w.copy_(w * k["d"] - k["s"] * (m1 / q))
    out = dict(w=w)
    if eight:
        bits = _random_bits(_places(c, w.device), s["step"])
        code, y, scale = _round_at_random(m1, bits & 0xFFFF)
        s["m"].copy_((code + 128 * (y < 0).int()).to(torch.uint8))
        s["ms"].copy_(scale)
        code, y, scale = _round_at_random(root, bits >> 16)
        s["v"].copy_(torch.where(y > 0, code.clamp(min=1), code).to(torch.uint8))
        s["vs"].copy_(scale)
        out.update(m=_e4m3(s["m"]), v=_e4m3(s["v"]), ms=s["ms"], vs=s["vs"])
    else:
        s["m"].copy_(m1)
        s["v"].copy_(v1)
        out.update(m=s["m"], v=s["v"])
    if c["work"]:
        s["work"].copy_(w)
        out["work"] = s["work"]
    return out


# ---------------------------------------------------------------- the framework's operators

def _own(s, c):
    import bwd_situ_glu_gb300 as sg
    if c["op"] == "quant":
        codes, scales = sg.situ_quant_fp8(s["x"], block_rows=c["block"])
        return dict(codes=_e4m3(codes), scales=scales)
    if c["op"] == "adamw":
        s["plan"].step(s["grads"], sg.adam_params(step=s["step"], **HYPER), seed=s["step"], grad_scale=s.get("clip"))
        out = dict(w=s["w"])
        if c["state"] == "fp8":
            out.update(m=_e4m3(s["m"]), v=_e4m3(s["v"]), ms=s["ms"], vs=s["vs"])
        else:
            out.update(m=s["m"], v=s["v"])
        if c["work"]:
            out["work"] = s["work"]
        return out
    w = (s["wq"], s["ws"])
    if c["dir"] == "fwd":
        a = sg.situ_quant_fp8(s["a"])
        return dict(out=sg.situ_linear_fp8(a, w, expert_offsets=s["offsets"], bias=s.get("bias"),
                                           residual=s.get("residual"), act=c["act"]))
    # fp32 weight gradients where the rounding of dz does not come first, bf16 ones behind an activation
    dw_dtype = torch.float32 if c["act"] == "none" else torch.bfloat16
    da, dw, dbias = sg.situ_linear_fp8_bwd(s["dout"], (s["aq"], s["as"]), w, expert_offsets=s["offsets"], act=c["act"],
                                           pre=s.get("pre"), dw_dtype=dw_dtype, bias=c["bias"])
    out = dict(da=da, dw=dw)
    if c["bias"]:
        out["dbias"] = dbias
    return out


_PLAIN = {"quant": _plain_quant, "linear": _plain_linear, "adamw": _plain_adamw}


def run(state):
    c = state["case"]
    return _own(state, c) if own else _PLAIN[c["op"]](state, c)


# ---------------------------------------------------------------- 64 bits

def _exact_scale(x, dims):
    """log2 of the scales of blocks of finite x (float64): the least e >= -126 with max |x| <= 448 * 2^e."""
    frac, e = torch.frexp(x.abs().amax(dims, keepdim=True) / 448.0)       # in [0.5, 1) * 2^e
    e = torch.where(frac == 0.5, e - 1, e)
    return torch.where(frac == 0, -126, e.clamp(min=-126)).double()


def _exact_step(y):
    """Distance of neighbouring E4M3 numbers at |y|: 3 bits below the leading one, 2^-9 at least."""
    _, e = torch.frexp(y.abs())
    return torch.exp2((e - 1).clamp(min=-6).double() - 3.0)


def _exact_quant(x, rows):
    """(codes' values, log2 of the scales, values) of float64 x [E, R, D]."""
    E, R, D = x.shape
    p = torch.zeros(E, -(-R // rows) * rows, _blocks(D) * BLOCK, dtype=torch.float64, device=x.device)
    p[:, :R, :D] = x
    p = p.view(E, -1, rows, _blocks(D), BLOCK)
    e = _exact_scale(p, (2, 4))
    y = p * torch.exp2(-e)
    step = _exact_step(y)
    y = torch.round(y / step) * step
    flat = lambda t: t.reshape(E, -1, p.shape[3] * BLOCK)[:, :R, :D]  # noqa: E731
    return flat(y), e[:, :, 0, :, 0], flat(y * torch.exp2(e))


def _exact_code_values(codes, log_scales, rows):
    """The float64 numbers of E4M3 codes (uint8 [E, R, D]) with these log2 scales."""
    c = codes.long()
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (8.0 + f) * torch.exp2(e.double() - 10.0))
    v = torch.where(c >= 128, -v, v)
    s = torch.exp2(log_scales).repeat_interleave(rows, 1).repeat_interleave(BLOCK, 2)
    return v * s[:, :c.shape[1], :c.shape[2]]


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


def _exact_adamw(s, c):
    h, t, n = HYPER, s["step"], s["w"].numel()
    w, g = s["w"].double(), s["g"].double()
    if c["clip"]:
        g = g * s["clip"].double()
    if c["state"] == "fp8":
        m, root = (_exact_code_values(s[k].view(1, -1, BLOCK), s[k + "s"].view(1, -1, 1).double() - 127.0, 1).view(-1)
                   for k in ("m", "v"))
        v = root.square()
    else:
        m, v = s["m"].double(), s["v"].double()
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g.square()
    bc1, bc2 = 1 - h["beta1"] ** t, 1 - h["beta2"] ** t
    w = w * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * (m / bc1) / ((v / bc2).sqrt() + h["eps"])
    out = dict(w=w, m=m, v=v)
    if c["state"] == "fp8":
        place = torch.cat([torch.arange(_blocks(k) * BLOCK, device=w.device) for k in _sizes(c)])

        def scatter(x):      # the stated permutation of 32 bits
            for shift, factor in ((16, 2654435761), (15, 1779033703), (16, 1)):
                x = ((x ^ (x >> shift)) * factor) % 2 ** 32
            return x
        r = scatter((place + scatter(torch.tensor(t * 2654435761 % 2 ** 32, device=w.device))) % 2 ** 32)
        for name, x, u in (("m", m, r % 65536), ("v", v.sqrt(), r // 65536)):
            p = x.view(-1, BLOCK)
            y = (p * torch.exp2(-_exact_scale(p, 1))).view(-1)
            step = _exact_step(y)
            code = torch.floor(y.abs() / step + u.double() / 65536.0) * step
            if name == "v":
                code = torch.where((y > 0) & (code == 0), 2.0 ** -9, code)
            out[name] = torch.sign(y) * code
        out.update(ms=None, vs=None)
    if c["work"]:
        out["work"] = w
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quant":
        x = s["x"].double()
        codes, _, _ = _exact_quant(x[None] if c["block"] == 1 else x, c["block"])
        return dict(codes=codes[0] if c["block"] == 1 else codes, scales=None)
    if c["op"] == "adamw":
        return _exact_adamw(s, c)
    R, N, K = c["R"], c["N"], c["K"]
    off = s["offsets"].tolist() if c["E"] else [0, R]
    E = len(off) - 1
    wq, ws = s["wq"].view(E, N, K), s["ws"].view(E, _blocks(N), _blocks(K))
    bias = s["bias"].reshape(E, N).double() if c["bias"] else None

    def weight(e):
        return _exact_code_values(wq[e:e + 1], ws[e:e + 1].double() - 127.0, BLOCK)[0]
    if c["dir"] == "fwd":
        a = _exact_quant(s["a"].double()[None], 1)[2][0]
        out = torch.empty(R, N, dtype=torch.float64, device="cuda")
        for e in range(E):
            r = slice(off[e], off[e + 1])
            z = a[r] @ weight(e).t()
            out[r] = _exact_act(z + bias[e] if c["bias"] else z, c["act"])[0]
        return dict(out=out + s["residual"].double() if c["residual"] else out)
    a = _exact_code_values(s["aq"][None], s["as"][None].double() - 127.0, 1)[0]
    dz = s["dout"].double()
    if c["act"] != "none":
        dz = dz * _exact_act(s["pre"].double(), c["act"])[1]
    db_from = dz
    dz = dz.to(torch.bfloat16).double()      # the gradient that the layer's products take
    dq = _exact_quant(dz[None], 1)[2][0]
    da = torch.empty(R, K, dtype=torch.float64, device="cuda")
    dw = torch.empty(E, N, K, dtype=torch.float64, device="cuda")
    db = torch.empty(E, N, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(off[e], off[e + 1])
        da[r], dw[e], db[e] = dq[r] @ weight(e), dz[r].t() @ a[r], db_from[r].sum(0)
    out = dict(da=da, dw=dw if c["E"] else dw[0])
    if c["bias"]:
        out["dbias"] = db if c["E"] else db[0]
    return out
