"""Products in 8 bits for the expert layer (C ABI: ``include/situ_fp8.h``).

* ``situ_quant_fp8`` / ``situ_dequant_fp8``: E4M3 codes with a power-of-two scale for each 128 elements of a row, or
  128 x 128 of a weight
* ``situ_linear_fp8`` / ``situ_linear_fp8_bwd``: the product of quantised rows and weights, per expert or dense, with bias,
  activation and residual, and its gradients
* ``linear_fp8``: the same as an autograd operator of bf16 rows and a bf16 or fp32 weight

A quantised tensor is a pair (codes uint8, scale bytes uint8): a byte b stands for 2^(b-127). ``codes.view(torch.float8_e4m3fn)``
are the codes' values. The conventions are those of the module ``moe``. Outputs that are given (``out``, ``codes``, ``scales``) count as
written in place: a backward that has saved them raises.
"""
from __future__ import annotations

import torch

from bwd_situ_glu_gb300 import _check, load as _lib, moe
from bwd_situ_glu_gb300.moe import (_act, _device_now, _elsewhere, _empty, _need, _out, _ptr, _increment_version, _raw_stream, _two,
                                    _type, _BF16, _CODE, _F32, _I32, _I64)

_U8 = torch.uint8
BLOCK = 128   # elements of a row (or rows and columns of a weight) that share a scale


def _blocks(n):
    return -(-n // BLOCK)


def _up(n):
    """Bytes up to a multiple of 256."""
    return (n + 255) & -256


def _shape3(x, name):
    """(E, R, D) of a tensor [R, D] or [E, R, D] on a CUDA device."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = x.shape
    n = len(shape)
    if not (n == 2 or n == 3) or not x.is_cuda:
        raise ValueError(f"{name} must be a two- or three-dimensional CUDA tensor, got {tuple(shape)} on {x.device}")
    return shape if n == 3 else (1, *shape)


def _scale_shape(shape, block_rows):
    if block_rows != 1 and block_rows != BLOCK:
        raise ValueError(f"block_rows must be 1 or {BLOCK}, got {block_rows!r}")
    *lead, R, D = shape
    return (*lead, R if block_rows == 1 else (R + 127) // 128, (D + 127) // 128)


def situ_quant_fp8(x, block_rows=1, codes=None, scales=None, stream=None):
    """(codes uint8 of x's shape, scales uint8 [.., R/block_rows, D/128], rounded up): x bf16 or fp32 [R, D] or [E, R, D]
    in blocks of 128 elements of a row (block_rows 1, the rows of a product) or 128 x 128 (128, a weight). A block's
    scale is the least power of two (2^-126 at least) with every finite value at most 448 times it; the code is
    x / scale rounded to nearest, ties to even, and 0x7F (NaN) for a value that is not finite."""
    ty, dev = _type(x, "x"), x.device
    shape = x.shape
    E, R, D = _shape3(x, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, x, lambda: situ_quant_fp8(x, block_rows, codes, scales))
    given = None if codes is None and scales is None else [t for t in (codes, scales) if t is not None]
    if codes is None:
        codes = _empty(shape, dtype=_U8, device=dev)
    else:
        _need(codes, _U8, shape, dev, "codes")
    s_shape = _scale_shape(shape, block_rows)
    if scales is None:
        scales = _empty(s_shape, dtype=_U8, device=dev)
    else:
        _need(scales, _U8, s_shape, dev, "scales")
    _check(_lib().situ_quant_fp8(x.data_ptr(), ty, codes.data_ptr(), scales.data_ptr(), E, R, D, block_rows,
                                 _raw_stream(dev.index)))
    if given:
        _increment_version(given)
    return codes, scales


def situ_dequant_fp8(codes, scales, block_rows=1, dtype=None, out=None, stream=None):
    """What (codes, scales) of situ_quant_fp8 stand for, in ``dtype`` (bf16, the default, or fp32): code * 2^(scale - 127).
    bf16 holds it exactly down to 2^-126."""
    E, R, D = _shape3(codes, "codes")
    dev, shape = codes.device, tuple(codes.shape)
    _need(codes, _U8, codes.shape, dev, "codes")
    _need(scales, _U8, _scale_shape(shape, block_rows), dev, "scales")
    if out is not None:
        dtype = out.dtype
    dtype = dtype or _BF16
    if dtype not in _CODE:
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, codes, lambda: situ_dequant_fp8(codes, scales, block_rows, dtype, out))
    given, out = out, _out(out, shape, dtype, dev, "out")
    _check(_lib().situ_dequant_fp8(codes.data_ptr(), scales.data_ptr(), out.data_ptr(), _CODE[dtype], E, R, D, block_rows,
                                   _raw_stream(dev.index)))
    if given is not None:
        _increment_version(given)
    return out


# ---------------------------------------------------------------- linear

def _pair(t, name):
    """(codes, scales) of a quantised tensor."""
    if not isinstance(t, (tuple, list)) or len(t) != 2 or not (isinstance(t[0], torch.Tensor) and isinstance(t[1], torch.Tensor)):
        raise TypeError(f"{name} must be a pair (codes, scales) of situ_quant_fp8")
    return t


def _weight(w, expert_offsets, dev):
    """(codes, scales, E, N, K, lead) of a quantised weight, [N,K] without expert_offsets, [E,N,K] with them."""
    wq, ws = _pair(w, "w")
    shape = wq.shape
    if expert_offsets is None:
        if len(shape) != 2:
            raise ValueError("w must be [N, K] without expert_offsets, [E, N, K] with them")
        E, lead = 1, ()
        N, K = shape
        s_shape = ((N + 127) // 128, (K + 127) // 128)
    else:
        if len(shape) != 3:
            raise ValueError("w must be [N, K] without expert_offsets, [E, N, K] with them")
        E, N, K = shape
        lead = (E,)
        s_shape = (E, (N + 127) // 128, (K + 127) // 128)
        _need(expert_offsets, _I64, (E + 1,), dev, "expert_offsets")
    _need(wq, _U8, shape, dev, "w codes")
    _need(ws, _U8, s_shape, dev, "w scales")
    return wq, ws, E, N, K, lead


def situ_linear_fp8(a, w, expert_offsets=None, bias=None, residual=None, act="none", save_pre=False, out=None, out_dtype=None,
                    status=None, stream=None):
    """situ_linear with rows and weights in 8 bits: out [R,N] = act(a W_eT + b_e) + residual. a: (codes [R,K], scales) of
    situ_quant_fp8, or a bf16 or fp32 tensor [R,K], which is quantised first; w: (codes [E,N,K] or [N,K], scales) of
    situ_quant_fp8 with block_rows 128. The other arguments are those of situ_linear. N and K multiples of 16."""
    plain = isinstance(a, torch.Tensor)
    aq, as_ = (a, None) if plain else _pair(a, "a")
    R, dev = _two(aq, "a")[0], aq.device
    wq, ws, E, N, K, lead = _weight(w, expert_offsets, dev)
    if plain:
        _type(a, "a")
        _need(a, a.dtype, (R, K), dev, "a")
    else:
        _need(aq, _U8, (R, K), dev, "a codes")
        _need(as_, _U8, (R, _blocks(K)), dev, "a scales")
    if bias is not None:
        _need(bias, _F32, (*lead, N), dev, "bias")
    if residual is not None:
        _need(residual, _BF16, (R, N), dev, "residual")
    if status is not None:
        _need(status, _I32, (1,), dev, "status")
    code = _act(act)
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, aq, lambda: situ_linear_fp8(a, w, expert_offsets, bias, residual, act, save_pre, out,
                                                              out_dtype, status))
    if out is not None:
        out_dtype = out.dtype
    given, out = out, _out(out, (R, N), out_dtype or _BF16, dev, "out")
    if plain:
        aq, as_ = situ_quant_fp8(a)
    pre = _empty((R, N), dtype=_BF16, device=dev) if save_pre else None
    _check(_lib().situ_linear_fp8_fwd(aq.data_ptr(), as_.data_ptr(), wq.data_ptr(), ws.data_ptr(), _ptr(expert_offsets), E,
                                      _ptr(bias), _ptr(residual), code, out.data_ptr(), _type(out, "out"), _ptr(pre),
                                      _ptr(status), R, N, K, _raw_stream(dev.index)))
    if given is not None:
        _increment_version(given)
    return (out, pre) if save_pre else out


def situ_linear_fp8_bwd(dout, a, w, expert_offsets=None, act="none", pre=None, dw_dtype=None, bias=True, need_da=True,
                        need_dw=True, status=None, stream=None):
    """(da bf16 [R,K], dw [E,N,K] (or [N,K]) of dw_dtype (default fp32), dbias fp32 [E,N] (or [N])) of situ_linear_fp8 for
    dout bf16 [R,N], a and w quantised as in the forward (a is not used without need_dw). dz = dout*act'(pre), rounded to
    bf16, as in situ_linear_bwd; da is the product of dz in 8 bits and the weights as they are; dw is the product of dz
    and the decoded rows, which bf16 holds exactly, on bf16 operands: it feeds an optimizer. What is not asked for is
    None. An expert without rows gets zeros in dw and dbias; da of rows of no expert is not written."""
    R, N_ = _two(dout, "dout")
    dev = dout.device
    wq, ws, E, N, K, lead = _weight(w, expert_offsets, dev)
    _need(dout, _BF16, (R, N), dev, "dout")
    if need_dw:
        aq, as_ = _pair(a, "a")
        _need(aq, _U8, (R, K), dev, "a codes")
        _need(as_, _U8, (R, _blocks(K)), dev, "a scales")
        if dw_dtype is not None and dw_dtype not in _CODE:       # w's own, from linear_fp8
            raise TypeError(f"dw_dtype must be torch.bfloat16 or torch.float32, got {dw_dtype}")
    code = _act(act)
    if code:
        if pre is None:
            raise ValueError(f"act {act!r} needs the saved pre (situ_linear_fp8 with save_pre=True)")
        _need(pre, _BF16, (R, N), dev, "pre")
    else:
        pre = None
    if status is not None:
        _need(status, _I32, (1,), dev, "status")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, dout, lambda: situ_linear_fp8_bwd(dout, a, w, expert_offsets, act, pre, dw_dtype, bias,
                                                                    need_da, need_dw, status))
    lib, s = _lib(), _raw_stream(dev.index)
    off, codes, kept = _ptr(expert_offsets), R * N, R * N * 2 if code else 0
    n_bias = lib.situ_linear_act_bwd_workspace(R, N, E) if bias else 0
    n_dw = lib.situ_linear_wgrad_workspace(R, N, K, E) if need_dw else 0
    # One buffer for what does not leave: dz behind an activation, and then in turn, in the stream's order, the bias sums'
    # workspace, dz in 8 bits, and the decoded rows with the weight gradient's workspace. (A small step is all host time.)
    first, rows_bytes = _up(kept), _up(R * K * 2)
    buf = _empty(first + max(n_bias, _up(codes) + R * _blocks(N) if need_da else 0, rows_bytes + n_dw if need_dw else 0), dtype=_U8,
                 device=dev)
    base = buf.data_ptr()
    at = base + first
    dz = base if code else dout.data_ptr()
    da = dw = dbias = None
    if code or bias:
        if bias:
            dbias = _empty((*lead, N), dtype=_F32, device=dev)
        _check(lib.situ_linear_act_bwd(dout.data_ptr(), _ptr(pre), code, off, E, base if code else 0, _ptr(dbias), at if n_bias else 0,
                                       n_bias, R, N, s))
    if need_da:
        da = _empty((R, K), dtype=_BF16, device=dev)
        ds = at + _up(codes)
        _check(lib.situ_quant_fp8(dz, 0, at, ds, 1, R, N, 1, s))
        _check(lib.situ_linear_fp8_dgrad(at, ds, wq.data_ptr(), ws.data_ptr(), off, E, da.data_ptr(), _ptr(status), R, N, K, s))
    if need_dw:
        dw = _empty((*lead, N, K), dtype=dw_dtype or _F32, device=dev)
        _check(lib.situ_dequant_fp8(aq.data_ptr(), as_.data_ptr(), at, 0, 1, R, K, 1, s))
        _check(lib.situ_linear_wgrad(dz, at, off, E, dw.data_ptr(), _type(dw, "dw"), at + rows_bytes if n_dw else 0, n_dw, _ptr(status), R,
                                     N, K, s))
    return da, dw, dbias


# ---------------------------------------------------------------- autograd operator

_function = None


def _autograd():
    """The autograd Function, created on first use."""
    global _function
    if _function is not None:
        return _function
    moe._autograd()

    class LinearFp8(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, w, bias, residual, expert_offsets, act, wq, status, grad):
            # needs_input_grad goes by the inputs alone; without grad mode there is no backward to keep anything for
            needs = grad and any(ctx.needs_input_grad[:3])
            keep = act != "none" and needs
            aq = situ_quant_fp8(a)
            wq = situ_quant_fp8(w, block_rows=BLOCK) if wq is None else wq
            out = situ_linear_fp8(aq, wq, expert_offsets, bias, residual, act, save_pre=keep, status=status)
            out, pre = out if keep else (out, None)
            if needs:
                # a, w and bias only mark what the gradients depend on (a second derivative raises there). w does for a as well, where it
                # has a gradient, and the rows need not be kept. Masters are not saved as tensors: the backward does not read them,
                # and an optimizer may have written them before it.
                with_w = ctx.needs_input_grad[1]
                ctx.save_for_backward(*(aq if with_w else (None, None)), *wq, expert_offsets, pre, a if keep and not with_w else None)
                ctx.masters = w if with_w else None, bias if keep else None
            ctx.act, ctx.status, ctx.dw_dtype = act, status, w.dtype   # status is not saved as a tensor: the kernels write it
            return out

        @staticmethod
        def backward(ctx, dout):
            need = ctx.needs_input_grad
            none = (None,) * 5
            if not any(need[:3]):      # the residual's alone
                return None, None, None, dout, *none
            aq, as_, wq, ws, expert_offsets, pre, a = ctx.saved_tensors
            dout = dout.contiguous()
            da, dw, db = situ_linear_fp8_bwd(dout, (aq, as_) if need[1] else None, (wq, ws), expert_offsets, ctx.act, pre,
                                             dw_dtype=ctx.dw_dtype, bias=need[2], need_da=need[0], need_dw=need[1], status=ctx.status)
            da, dw, db = moe._once((da, dw, db), dout, a, *ctx.masters)
            return da, dw, db, dout if need[3] else None, *none

    _function = LinearFp8
    return _function


def linear_fp8(a, w, bias=None, residual=None, expert_offsets=None, act="none", wq=None, status=None):
    """situ_linear_fp8 of bf16 rows a and a bf16 or fp32 weight w (both quantised here; ``wq``: w's codes and scales where
    the program has them, as after an optimizer step), bf16 out, differentiable in a, w (gradient in w's type), bias and
    residual. The gradients are those of the product of the quantised operands, taken for the operands' own (the codes'
    rounding has no derivative). The backward keeps the rows' codes, not the rows (those only where w has no gradient and an
    activation follows), and ``wq`` itself: it has to stay as it is until then, or the backward raises (w and bias may be stepped before it). Before a backward is captured in a graph, every eager
    graph of the same leaves has to be gone, as for any autograd operator: PyTorch ties a leaf's gradient to the stream that it was
    first used on."""
    if wq is not None:
        if tuple(_pair(wq, "wq")[0].shape) != tuple(w.shape):
            raise ValueError("wq must be w's codes and scales")
    if isinstance(a, torch.Tensor) and a.dtype != _BF16:
        raise TypeError(f"a must be torch.bfloat16, got {a.dtype}")
    return _autograd().apply(a, w, bias, residual, expert_offsets, act, wq, status, torch.is_grad_enabled())
