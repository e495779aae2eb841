"""The operators around the expert activation in one MoE layer (C ABI: ``include/situ_moe.h``).

* ``situ_route_topk`` / ``situ_route_topk_bwd``: top-k softmax of the router scores
* ``situ_dispatch_plan``: the token-expert pairs in expert order (offsets, rows and back)
* ``situ_dispatch``: tokens copied to their rows (its gradient is ``situ_combine`` without weights)
* ``situ_combine`` / ``situ_combine_bwd``: the weighted rows of a token summed back
* ``situ_linear`` / ``situ_linear_bwd``: per-expert or dense product with bias, activation, residual
* ``route_topk``, ``moe_dispatch``, ``moe_combine``, ``linear``: the same as autograd operators

Like the rest of the package these check tensor metadata, marshal pointers and raise ``SituGluError``
on a non-zero status; every tensor is contiguous and on one CUDA device. ``stream`` (a torch stream or
a raw handle; default: the current stream) is where the work runs; outputs that are not given and
workspaces are allocated on that stream.
"""
from __future__ import annotations

import torch

import bwd_situ_glu_gb300 as _sg
from bwd_situ_glu_gb300 import _check, load as _lib

# A decoding step's kernels take 3 to 5 us, an allocation and a launch through ctypes 5 us of host time; hence the
# names bound here, the one expression per tensor in _need, and the raw stream handle: a third less host time a call (with
# its allocations a one-kernel call takes 10.5 to 15 us, depending on the host).
_T, _BF16, _F32, _I32, _I64 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32, torch.int64
_CODE = {_BF16: 0, _F32: 1}  # SITU_BF16, SITU_FP32
_empty = torch.empty
_device_now, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
# Tells autograd that a kernel wrote a given tensor: a backward that still needs what it held raises then, as behind PyTorch's own
# operators in place.
_increment_version = torch.autograd.graph.increment_version

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
MAX_EXPERTS, MAX_TOPK = 1024, 32  # SITU_MAX_EXPERTS, SITU_MAX_TOPK


def _type(t, name):
    """SITU_BF16 or SITU_FP32 of a tensor."""
    if not isinstance(t, _T):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return code


def _two(t, name):
    """The shape of a two-dimensional CUDA tensor."""
    if not isinstance(t, _T):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a two-dimensional CUDA tensor, got {tuple(t.shape)} on {t.device}")
    return t.shape


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _elsewhere(stream, t, call):
    """call() with t's device and ``stream`` current, so that what it allocates belongs to that stream."""
    with torch.cuda.device(t.device):
        if stream is None:
            return call()
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=t.device)
        with torch.cuda.stream(stream):
            return call()


def _need(t, dtype, shape, dev, name):
    """A contiguous tensor of this type and shape on this device."""
    if t.__class__ is not _T or t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
        _sg._need(t, dtype, shape, name)   # says what is wrong (a subclass of Tensor is fine)
        if t.device != dev:
            raise ValueError("all tensors must be on the same device")


def _out(t, shape, dtype, dev, name):
    if t is None:
        return _empty(shape, dtype=dtype, device=dev)
    _need(t, dtype, shape, dev, name)
    return t


def _scratch(nbytes, like):
    return torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes else None


# ---------------------------------------------------------------- routing

def situ_route_topk(logits, k, p=None, ids=None, stream=None):
    """(p fp32 [T,k], ids int32 [T,k]): softmax over the k largest scores of each token, in descending
    order, ties to the lower index. A score of -inf is never chosen (id -1, p 0). logits [T,E] bf16 or
    fp32, E <= 1024, k <= min(E, 32)."""
    ty = _type(logits, "logits")
    T, E = _two(logits, "logits")
    dev = logits.device
    _need(logits, logits.dtype, (T, E), dev, "logits")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, logits, lambda: situ_route_topk(logits, k, p, ids))
    p = _out(p, (T, k), _F32, dev, "p")
    ids = _out(ids, (T, k), _I32, dev, "ids")
    _check(_lib().situ_route_topk(logits.data_ptr(), ty, p.data_ptr(), ids.data_ptr(), T, E, k, _raw_stream(dev.index)))
    return p, ids


def situ_route_topk_bwd(ids, p, dp, num_experts, dtype=None, row_of=None, dlogits=None, stream=None):
    """dlogits [T,num_experts] of ``dtype`` (default fp32): p_k(dp_k - sum_j p_j dp_j) at ids, 0 elsewhere.
    dp fp32 [T,k], or with ``row_of`` (int32 [T,k]) fp32 [R] in row order."""
    T, k = _two(ids, "ids")
    dev = ids.device
    _need(ids, _I32, (T, k), dev, "ids")
    _need(p, _F32, (T, k), dev, "p")
    R = 0
    if row_of is None:
        _need(dp, _F32, (T, k), dev, "dp")
    else:
        _need(row_of, _I32, (T, k), dev, "row_of")
        R = dp.numel()
        _need(dp, _F32, (R,), dev, "dp")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, ids, lambda: situ_route_topk_bwd(ids, p, dp, num_experts, dtype, row_of, dlogits))
    if dlogits is not None:
        dtype = dlogits.dtype
    dlogits = _out(dlogits, (T, num_experts), dtype or _F32, dev, "dlogits")
    _check(_lib().situ_route_topk_bwd(ids.data_ptr(), p.data_ptr(), dp.data_ptr(), _ptr(row_of), R, dlogits.data_ptr(),
                                      _type(dlogits, "dlogits"), T, num_experts, k, _raw_stream(dev.index)))
    return dlogits


# ---------------------------------------------------------------- tokens sorted by expert and back

def situ_dispatch_plan(ids, num_experts, p=None, stream=None):
    """(expert_offsets int64 [E+1], row_of int32 [T,k], src int32 [T*k], p_rows fp32 [T*k] or None): the rows
    of the token-expert pairs, sorted by expert and, within one, by token and choice. An id outside
    [0, num_experts) has no row (row_of -1); src past the last row is -1, p_rows 0."""
    T, k = _two(ids, "ids")
    dev = ids.device
    _need(ids, _I32, (T, k), dev, "ids")
    if p is not None:
        _need(p, _F32, (T, k), dev, "p")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, ids, lambda: situ_dispatch_plan(ids, num_experts, p))
    lib, n = _lib(), T * k
    offsets = _empty(max(0, num_experts + 1), dtype=_I64, device=dev)
    row_of = _empty((T, k), dtype=_I32, device=dev)
    src = _empty(n, dtype=_I32, device=dev)
    p_rows = None if p is None else _empty(n, dtype=_F32, device=dev)
    nb = lib.situ_dispatch_plan_workspace(T, k, num_experts)
    ws = _scratch(nb, ids)
    # without tokens there is nothing to weigh: the pointers of empty tensors are null
    _check(lib.situ_dispatch_plan(ids.data_ptr(), _ptr(p), offsets.data_ptr(), row_of.data_ptr(), src.data_ptr(),
                                  _ptr(p_rows), _ptr(ws), nb, T, k, num_experts, _raw_stream(dev.index)))
    return offsets, row_of, src, p_rows


def situ_dispatch(x, row_of, expert_offsets, weights=None, h=None, stream=None):
    """h [T*k, D]: h[row_of[t,j]] = x[t], or weights[t,j]*x[t] with weights fp32 [T,k]; rows from
    expert_offsets[-1] on are zero. x [T,D] bf16 or fp32. row_of and expert_offsets are one plan's: a row before
    expert_offsets[-1] that row_of does not name is not written, so a token-expert pair is dropped by its id
    (-1) before the plan, not by its row_of after it."""
    ty = _type(x, "x")
    (T, D), k = _two(x, "x"), _two(row_of, "row_of")[1]
    dev = x.device
    _need(x, x.dtype, (T, D), dev, "x")
    _need(row_of, _I32, (T, k), dev, "row_of")
    E = expert_offsets.numel() - 1
    _need(expert_offsets, _I64, (E + 1,), dev, "expert_offsets")
    if weights is not None:
        _need(weights, _F32, (T, k), dev, "weights")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, x, lambda: situ_dispatch(x, row_of, expert_offsets, weights, h))
    h = _out(h, (T * k, D), x.dtype, dev, "h")
    _check(_lib().situ_dispatch(x.data_ptr(), ty, row_of.data_ptr(), expert_offsets.data_ptr(), E, _ptr(weights),
                                h.data_ptr(), T, k, T * k, D, _raw_stream(dev.index)))
    return h


def situ_combine(o, row_of, weights=None, residual=None, y=None, stream=None):
    """y [T,D] = residual + sum_j weights[t,j]*o[row_of[t,j]] (weights default to 1, residual to 0; fp32,
    rounded once). o [R,D] bf16 or fp32; ``y`` may be ``residual`` itself."""
    ty = _type(o, "o")
    (R, D), (T, k) = _two(o, "o"), _two(row_of, "row_of")
    dev = o.device
    _need(o, o.dtype, (R, D), dev, "o")
    _need(row_of, _I32, (T, k), dev, "row_of")
    if weights is not None:
        _need(weights, _F32, (T, k), dev, "weights")
    if residual is not None:
        _need(residual, o.dtype, (T, D), dev, "residual")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, o, lambda: situ_combine(o, row_of, weights, residual, y))
    y = _out(y, (T, D), o.dtype, dev, "y")
    _check(_lib().situ_combine(o.data_ptr(), ty, row_of.data_ptr(), _ptr(weights), _ptr(residual), y.data_ptr(), T, k,
                               R, D, _raw_stream(dev.index)))
    return y


def situ_combine_bwd(dy, o, row_of, weights, expert_offsets, do=None, dweights=None, stream=None):
    """(do [R,D] of o's type, dweights fp32 [T,k]): do[row_of[t,j]] = weights[t,j]*dy[t] (rows from
    expert_offsets[-1] on are zero; one before it that row_of does not name is not written, as in
    situ_dispatch), dweights[t,j] = <dy[t], o[row_of[t,j]]> (0 without a row)."""
    ty = _type(o, "o")
    (R, D), (T, k) = _two(o, "o"), _two(row_of, "row_of")
    dev = o.device
    _need(o, o.dtype, (R, D), dev, "o")
    _need(dy, o.dtype, (T, D), dev, "dy")
    _need(row_of, _I32, (T, k), dev, "row_of")
    _need(weights, _F32, (T, k), dev, "weights")
    E = expert_offsets.numel() - 1
    _need(expert_offsets, _I64, (E + 1,), dev, "expert_offsets")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, o, lambda: situ_combine_bwd(dy, o, row_of, weights, expert_offsets, do, dweights))
    do = _out(do, (R, D), o.dtype, dev, "do")
    dweights = _out(dweights, (T, k), _F32, dev, "dweights")
    _check(_lib().situ_combine_bwd(dy.data_ptr(), o.data_ptr(), ty, row_of.data_ptr(), weights.data_ptr(),
                                   expert_offsets.data_ptr(), E, do.data_ptr(), dweights.data_ptr(), T, k, R, D,
                                   _raw_stream(dev.index)))
    return do, dweights


# ---------------------------------------------------------------- linear

def _linear_shape(a, w, expert_offsets, a_name="a"):
    """(R, N, K, E, lead): w is [N,K] without expert_offsets, [E,N,K] with them; lead is () or (E,)."""
    R, dev = _two(a, a_name)[0], a.device
    if expert_offsets is None:
        if w.dim() != 2:
            raise ValueError("w must be [N, K] without expert_offsets")
        E, lead = 1, ()
        N, K = w.shape
    else:
        if w.dim() != 3:
            raise ValueError("w must be [E, N, K] with expert_offsets")
        E, N, K = w.shape
        lead = (E,)
        _need(expert_offsets, _I64, (E + 1,), dev, "expert_offsets")
    _need(w, _BF16, (*lead, N, K), dev, "w")
    return R, N, K, E, lead


def _act(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def situ_linear(a, w, expert_offsets=None, bias=None, residual=None, act="none", save_pre=False, out=None,
                out_dtype=None, status=None, stream=None):
    """out [R,N] = act(a W_eT + b_e) + residual for the rows of every expert e (rows
    expert_offsets[e] .. expert_offsets[e+1]-1; rows of no expert are not written), or with one weight
    for all rows without expert_offsets. a bf16 [R,K]; w bf16 [E,N,K] (or [N,K]); bias fp32 [E,N] (or
    [N]); residual bf16 [R,N]; act none | relu | silu | gelu; out bf16 (default) or fp32. With
    ``save_pre`` returns (out, pre): pre bf16 [R,N] is the value before the activation, for
    situ_linear_bwd. N and K multiples of 8. ``status`` (int32 [1] on the device, zeroed by the caller)
    turns 1 if a pipeline wait timed out."""
    R, N, K, E, lead = _linear_shape(a, w, expert_offsets)
    dev = a.device
    _need(a, _BF16, (R, K), dev, "a")
    if bias is not None:
        _need(bias, _F32, (*lead, N), dev, "bias")
    if residual is not None:
        _need(residual, _BF16, (R, N), dev, "residual")
    if status is not None:
        _need(status, _I32, (1,), dev, "status")
    code = _act(act)
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, a, lambda: situ_linear(a, w, expert_offsets, bias, residual, act, save_pre, out,
                                                         out_dtype, status))
    if out is not None:
        out_dtype = out.dtype
    out = _out(out, (R, N), out_dtype or _BF16, dev, "out")
    pre = _empty((R, N), dtype=_BF16, device=a.device) if save_pre else None
    _check(_lib().situ_linear_fwd(a.data_ptr(), w.data_ptr(), _ptr(expert_offsets), E, _ptr(bias), _ptr(residual), code,
                                  out.data_ptr(), _type(out, "out"), _ptr(pre), _ptr(status), R, N, K, _raw_stream(dev.index)))
    return (out, pre) if save_pre else out


def situ_linear_bwd(dout, a, w, expert_offsets=None, act="none", pre=None, dw_dtype=None, bias=True, need_da=True,
                    need_dw=True, status=None, stream=None):
    """(da bf16 [R,K], dw [E,N,K] (or [N,K]) of dw_dtype (default fp32), dbias fp32 [E,N] (or [N])) of
    situ_linear for dout bf16 [R,N]; the residual's gradient is dout itself. An activation needs ``pre`` of
    the forward; dz = dout*act'(pre) is then rounded to bf16 before the two products (dbias is the sum
    of the unrounded dz). What is not asked for (bias, need_da, need_dw) is None. An expert without rows
    gets zeros in dw and dbias; da of rows of no expert is not written."""
    R, N, K, E, lead = _linear_shape(dout, w, expert_offsets, "dout")
    dev = dout.device
    _need(dout, _BF16, (R, N), dev, "dout")
    if need_dw:
        _need(a, _BF16, (R, K), dev, "a")
    code = _act(act)
    if code:
        if pre is None:
            raise ValueError(f"act {act!r} needs the saved pre (situ_linear with save_pre=True)")
        _need(pre, _BF16, (R, N), dev, "pre")
    else:
        pre = None
    if status is not None:
        _need(status, _I32, (1,), dev, "status")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, dout, lambda: situ_linear_bwd(dout, a, w, expert_offsets, act, pre, dw_dtype, bias,
                                                                need_da, need_dw, status))
    lib, s = _lib(), _raw_stream(dev.index)
    da = dw = dbias = None
    dz, off = dout, _ptr(expert_offsets)
    if code or bias:
        if code:
            dz = _empty((R, N), dtype=_BF16, device=dev)
        nb, ws = 0, None
        if bias:
            dbias = _empty((*lead, N), dtype=_F32, device=dev)
            nb = lib.situ_linear_act_bwd_workspace(R, N, E)
            ws = _scratch(nb, dout)
        _check(lib.situ_linear_act_bwd(dout.data_ptr(), _ptr(pre), code, off, E, dz.data_ptr() if code else 0,
                                       _ptr(dbias), _ptr(ws), nb, R, N, s))
    if need_da:
        da = _empty((R, K), dtype=_BF16, device=dev)
        _check(lib.situ_linear_dgrad(dz.data_ptr(), w.data_ptr(), off, E, da.data_ptr(), _ptr(status), R, N, K, s))
    if need_dw:
        dw = _empty((*lead, N, K), dtype=dw_dtype or _F32, device=dev)
        nb = lib.situ_linear_wgrad_workspace(R, N, K, E)
        ws = _scratch(nb, dout)
        _check(lib.situ_linear_wgrad(dz.data_ptr(), a.data_ptr(), off, E, dw.data_ptr(), _type(dw, "dw"), _ptr(ws), nb,
                                     _ptr(status), R, N, K, s))
    return da, dw, dbias


def selftest_wait_timeout(status, elapsed_ns=None, stream=None):
    """Launch the self-test of the linear operator's bounded waits: after ~2 s it writes 1 to ``status`` (int32 [1]
    on the device, zeroed by the caller); ``elapsed_ns`` (int64 [1]) receives the wait's duration."""
    _sg._need(status, _I32, (1,), "status")
    dev = status.device
    if elapsed_ns is not None:
        _need(elapsed_ns, _I64, (1,), dev, "elapsed_ns")
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, status, lambda: selftest_wait_timeout(status, elapsed_ns))
    _check(_lib().situ_linear_selftest_wait_timeout(status.data_ptr(), _ptr(elapsed_ns), _raw_stream(dev.index)))


# ---------------------------------------------------------------- autograd operators

_functions = None
_once = None      # set by _autograd: gradients whose second derivative raises


def _autograd():
    """The autograd Functions, created on first use."""
    global _functions, _once
    if _functions is not None:
        return _functions

    class Once(torch.autograd.Function):
        """The first n of its arguments; what depends on the arguments through them has no derivative here."""
        @staticmethod
        def forward(ctx, n, *args):
            return tuple(None if t is None else t.view_as(t) for t in args[:n])

        @staticmethod
        def backward(ctx, *grads):
            raise RuntimeError("the gradients of the routing, dispatch, combine and linear operators are not "
                               "differentiable themselves")

    def once(grads, *inputs):
        """The gradients, which depend on inputs: where a graph of them is made, a second derivative raises."""
        return Once.apply(len(grads), *grads, *inputs) if torch.is_grad_enabled() else grads

    class RouteTopk(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, k):
            p, ids = situ_route_topk(logits, k)
            ctx.save_for_backward(p, ids)
            ctx.experts, ctx.dtype = logits.shape[1], logits.dtype
            ctx.mark_non_differentiable(ids)
            return p, ids

        @staticmethod
        def backward(ctx, dp, _):
            p, ids = ctx.saved_tensors
            return *once((situ_route_topk_bwd(ids, p, dp.contiguous(), ctx.experts, dtype=ctx.dtype),), p, dp), None

    class Dispatch(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, row_of, expert_offsets):
            ctx.save_for_backward(row_of)
            return situ_dispatch(x, row_of, expert_offsets)

        @staticmethod
        def backward(ctx, dh):
            (row_of,) = ctx.saved_tensors
            return *once((situ_combine(dh.contiguous(), row_of),), dh), None, None

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, o, weights, residual, row_of, expert_offsets):
            ctx.save_for_backward(o, weights, row_of, expert_offsets)
            return situ_combine(o, row_of, weights=weights, residual=residual)

        @staticmethod
        def backward(ctx, dy):
            o, weights, row_of, expert_offsets = ctx.saved_tensors
            if not any(ctx.needs_input_grad[:2]):      # the residual's alone
                return None, None, dy, None, None
            plain = weights is None    # a sum: the weights are ones without a gradient
            if plain:
                weights = torch.ones(row_of.shape, dtype=_F32, device=o.device)
            do, dw = situ_combine_bwd(dy.contiguous(), o, row_of, weights, expert_offsets)
            do, dw = once((do, None if plain else dw), dy, o, weights)
            return do, dw, dy if ctx.needs_input_grad[2] else None, None, None

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, w, bias, residual, expert_offsets, act, status, grad):
            # needs_input_grad goes by the inputs alone; without grad mode there is no backward to keep anything for
            keep = act != "none" and grad and any(ctx.needs_input_grad[:3])
            out = situ_linear(a, w, expert_offsets, bias, residual, act, save_pre=keep, status=status)
            out, pre = out if keep else (out, None)
            ctx.save_for_backward(a, w, expert_offsets, pre)
            # not saved as tensors: the kernels write the status, and bias only marks what dz depends on (an optimizer may have written it
            # before the backward, which does not read it)
            ctx.act, ctx.status, ctx.bias = act, status, bias if keep else None
            return out

        @staticmethod
        def backward(ctx, dout):
            a, w, expert_offsets, pre = ctx.saved_tensors
            need = ctx.needs_input_grad
            if not any(need[:3]):      # the residual's alone: no pre was kept
                return None, None, None, dout, None, None, None, None
            dout = dout.contiguous()
            da, dw, db = situ_linear_bwd(dout, a, w, expert_offsets, ctx.act, pre, dw_dtype=_BF16,
                                         bias=need[2], need_da=need[0], need_dw=need[1], status=ctx.status)
            da, dw, db = once((da, dw, db), dout, a, w, ctx.bias)
            return da, dw, db, dout if need[3] else None, None, None, None, None

    _once = once
    _functions = (RouteTopk, Dispatch, Combine, Linear)
    return _functions


def route_topk(logits, k):
    """situ_route_topk, differentiable in the scores: (p, ids)."""
    return _autograd()[0].apply(logits, int(k))


def moe_dispatch(x, row_of, expert_offsets):
    """situ_dispatch, differentiable in x (row_of and expert_offsets of one plan, as there)."""
    return _autograd()[1].apply(x, row_of, expert_offsets)


def moe_combine(o, weights, row_of, expert_offsets, residual=None):
    """situ_combine, differentiable in o, weights (None: all 1) and residual; row_of and expert_offsets are one
    plan's (the gradient of o at a row before expert_offsets[-1] that row_of does not name is undefined)."""
    return _autograd()[2].apply(o, weights, residual, row_of, expert_offsets)


def linear(a, w, bias=None, residual=None, expert_offsets=None, act="none", status=None):
    """situ_linear (bf16 out), differentiable in a, w (gradient in bf16, as PyTorch's autograd wants),
    bias and residual. Gradients of rows that belong to no expert are undefined. ``status`` as in
    situ_linear, for the backward's kernels too."""
    return _autograd()[3].apply(a, w, bias, residual, expert_offsets, act, status, torch.is_grad_enabled())
