"""One AdamW step over many tensors on the device, states in fp32 or in 8 bits (C ABI: ``include/situ_adamw.h``).

* ``adamw_state``: the states of a list of parameters, zero
* ``AdamWPlan``: parameters, states and working copies that belong together; ``plan.step(grads, adam_params(...))``
* ``situ_adamw_step``: the same as one call
* ``adamw_coefficients``: what a step computes with, as a tensor, for steps captured in a graph

Parameters (the masters) are fp32, gradients fp32 or bf16 (all of one type), working copies bf16. States in 8 bits are E4M3
codes and a scale byte for each 128 elements (module ``fp8``), of m and of the ROOT of v, rounded up or down at random with the
mean kept (of the root: v itself comes out 2 to 7 % high for gradients that vary, and roots below 2^-17 of their block's largest are lifted
to about that). The conventions are those of the module ``moe``.
"""
from __future__ import annotations

import ctypes
import operator
import threading

import numpy as np
import torch

import bwd_situ_glu_gb300 as _sg
from bwd_situ_glu_gb300 import AdamParams, _check, load as _lib
from bwd_situ_glu_gb300.moe import _device_now, _elsewhere, _increment_version, _ptr, _raw_stream, _CODE, _F32, _BF16

_T, _U8 = torch.Tensor, torch.uint8
_TYPES = {torch.Tensor, torch.nn.Parameter}
_dtype, _shape, _nbytes = operator.attrgetter("dtype"), operator.attrgetter("shape"), operator.attrgetter("nbytes")
_E4M3 = 2         # SITU_E4M3
_MOVABLE = {"params": (_F32, 0), "work": (_BF16, 6)}   # type and column of what may move between steps
_COEFFICIENTS = 9  # words of situ_adamw_coefficients


def adamw_state(params, state="fp8"):
    """dict of m, v and, with state "fp8", m_scales and v_scales: zero states of ``params`` (fp32 CUDA tensors), as AdamWPlan
    takes them. "fp32": 8 bytes a parameter, "fp8": 2 and 1/64."""
    if state not in ("fp8", "fp32"):
        raise ValueError(f'state must be "fp8" or "fp32", got {state!r}')
    if state == "fp32":
        return dict(m=[torch.zeros_like(p, dtype=_F32, memory_format=torch.contiguous_format) for p in params],
                    v=[torch.zeros_like(p, dtype=_F32, memory_format=torch.contiguous_format) for p in params])
    new = lambda p, n: torch.ones(n, dtype=_U8, device=p.device)  # noqa: E731
    codes = lambda: [torch.zeros(p.shape, dtype=_U8, device=p.device) for p in params]  # noqa: E731
    scales = lambda: [new(p, -(-p.numel() // 128)) for p in params]  # noqa: E731
    return dict(m=codes(), v=codes(), m_scales=scales(), v_scales=scales())


def adamw_coefficients(params: AdamParams, seed=None, out=None):
    """What a step with these hyper-parameters and this seed (default: the step count) computes with: an int32 tensor [9] on the
    host (the words of situ_adamw_coefficients), or ``out``, filled. Copied to a CUDA tensor before each replay, it lets a captured
    AdamWPlan.step(grads, that tensor) go on counting."""
    if out is None:
        out = torch.empty(_COEFFICIENTS, dtype=torch.int32)
    if out.device.type != "cpu" or out.dtype != torch.int32 or tuple(out.shape) != (_COEFFICIENTS,) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous int32 [{_COEFFICIENTS}] tensor on the host")
    seed = params.step if seed is None else seed
    _check(_lib().situ_adamw_coefficients_of(ctypes.byref(params), int(seed) & 0xFFFFFFFF, out.data_ptr()))
    return out


class AdamWPlan:
    """Parameters with their states and, if any, working copies: what AdamW keeps.

    ``params``: fp32 tensors of any shape; ``m``, ``v``: fp32 of the same shapes, or uint8 codes with ``m_scales`` and
    ``v_scales`` (uint8, ceil(n / 128) each); ``work``: bf16 of the same shapes, or None. All contiguous, on one CUDA device, and
    no two sharing memory. The plan holds them; ``step`` updates them in place. A parameter's or working copy's ``.data`` may be
    replaced between steps by one of the same kind; states are refilled with copy_ (a plan whose states were moved raises, and their
    memory stays with the plan).
    Steps from several threads are each taken whole. To autograd a step is an operation in place on ``params`` and ``work``, as
    PyTorch's optimizers are: a backward that has saved what one of them held before raises. (That goes by the tensors given here: pass
    parameters, not their ``.data``. Replays of a captured step are not counted.)"""

    def __init__(self, params, m, v, m_scales=None, v_scales=None, work=None):
        params, m, v = list(params), list(m), list(v)
        if (m_scales is None) != (v_scales is None):
            raise ValueError("m_scales and v_scales go together")
        self._eight = m_scales is not None
        lists = dict(params=params, m=m, v=v)
        if self._eight:
            lists.update(m_scales=list(m_scales), v_scales=list(v_scales))
        if work is not None:
            lists["work"] = list(work)
        for name, ts in lists.items():
            if len(ts) != len(params):
                raise ValueError(f"{name} must have {len(params)} tensors, got {len(ts)}")
        self._params, self._lists, self._updated = params, lists, params + lists.get("work", [])
        self._shapes = [p.shape for p in params if isinstance(p, torch.Tensor)]
        self._device = params[0].device if params and isinstance(params[0], torch.Tensor) else None
        state = _U8 if self._eight else _F32
        kinds = dict(params=_F32, m=state, v=state, m_scales=_U8, v_scales=_U8, work=_BF16)
        for name, ts in lists.items():
            for i, t in enumerate(ts):
                n = -(-params[i].numel() // 128) if name.endswith("scales") else None
                _sg._need(t, kinds[name], params[i].shape if n is None else (n,), f"{name}[{i}]")
                if t.device != self._device:
                    raise ValueError("all tensors must be on the same device")
        # rows of situ_adamw_tensor: w, grad, m, v, m_scales, v_scales, work, n
        self._table = np.zeros((len(params), 8), dtype=np.int64)
        for column, name in ((0, "params"), (2, "m"), (3, "v"), (4, "m_scales"), (5, "v_scales"), (6, "work")):
            if name in lists:
                self._table[:, column] = [t.data_ptr() for t in lists[name]]
        self._table[:, 7] = [p.numel() for p in params]
        self._table_ptr = self._table.ctypes.data
        self._lock = threading.Lock()
        self._at = {name: [t.data_ptr() for t in ts] for name, ts in lists.items()}
        # The place says that nothing moved only with what is there: of parameters and working copies the bytes are looked at again every
        # step, and that they are contiguous; the states' memory cannot become another tensor's, for it is held here.
        self._bytes = {name: [t.nbytes for t in lists[name]] for name in _MOVABLE if name in lists}
        self._kept = [t.detach() for name, ts in lists.items() if name not in _MOVABLE for t in ts]

    def _alike(self, tensors, dtype):
        """Whether every one is contiguous, of this type, of its parameter's shape and on the plan's device: one pass of map for each
        property, which takes half the time of one loop with all of them."""
        return ((set(map(type, tensors)) <= _TYPES or all([isinstance(t, _T) for t in tensors]))
                and set(map(_dtype, tensors)) == {dtype} and set(map(_T.get_device, tensors)) == {self._device.index}
                and all(map(_T.is_contiguous, tensors)) and list(map(_shape, tensors)) == self._shapes)

    def step(self, grads, params, seed=None, grad_scale=None, stream=None):
        """One step with ``grads`` (a tensor for each parameter, all fp32 or all bf16) and ``params``: adam_params(...), or an int32
        CUDA tensor [9] that holds adamw_coefficients(...) when the step runs. ``grad_scale`` (fp32 [1] on the device)
        multiplies the gradients. ``seed`` (default: the step count) is that of the states' rounding in 8 bits: another for every step.
        A step captured in a graph repeats what it was captured with, but for what it reads from tensors."""
        dev = self._device
        if len(grads) != len(self._params):
            raise ValueError(f"grads must have {len(self._params)} tensors, got {len(grads)}")
        if dev is None:
            return
        on_device = isinstance(params, torch.Tensor)
        if on_device:
            _sg._need(params, torch.int32, (_COEFFICIENTS,), "params")
            if seed is not None:
                raise ValueError("the seed is among the coefficients")
        elif not isinstance(params, AdamParams):
            raise TypeError("params must be adam_params(...) or a tensor of adamw_coefficients")
        if grad_scale is not None:
            _sg._need(grad_scale, _F32, (1,), "grad_scale")
        for t in (params if on_device else None, grad_scale):
            if t is not None and t.device != dev:
                raise ValueError("all tensors must be on the same device")
        kind = grads[0].dtype if isinstance(grads[0], torch.Tensor) else None
        if kind not in _CODE:
            raise TypeError(f"grads must be torch.float32 or torch.bfloat16 tensors, got {kind}")
        if not self._alike(grads, kind):
            for i, (g, shape) in enumerate(zip(grads, self._shapes)):
                _sg._need(g, kind, shape, f"grads[{i}]")
            raise ValueError("all tensors must be on the same device")
        if stream is not None or dev.index != _device_now():
            return _elsewhere(stream, self._params[0], lambda: self.step(grads, params, seed, grad_scale))
        if not on_device and seed is None:
            seed = params.step
        with self._lock:                     # the table is read before the call returns, without Python's lock
            table = self._table
            # A parameter's or working copy's .data may have been replaced since the last step, and is then checked again.
            for name, at in self._at.items():
                tensors = self._lists[name]
                now = list(map(_T.data_ptr, tensors))
                want, column = _MOVABLE.get(name, (None, None))
                if now != at and want is None:
                    raise ValueError(f"{name} is no longer where it was when the plan was made: make another plan")
                if want and (now != at or list(map(_nbytes, tensors)) != self._bytes[name] or not all(map(_T.is_contiguous, tensors))):
                    for i, (p, shape) in enumerate(zip(tensors, self._shapes)):
                        _sg._need(p, want, shape, f"{name}[{i}]")
                        if p.device != dev:
                            raise ValueError("all tensors must be on the same device")
                    table[:, column] = self._at[name] = now
            table[:, 1] = list(map(_T.data_ptr, grads))
            _check(_lib().situ_adamw_step(self._table_ptr, len(table), _CODE[kind], _E4M3 if self._eight else _CODE[_F32],
                                          None if on_device else ctypes.byref(params), 0 if on_device else int(seed) & 0xFFFFFFFF,
                                          params.data_ptr() if on_device else None, _ptr(grad_scale), _raw_stream(dev.index)))
            _increment_version(self._updated)


def situ_adamw_step(params, grads, m, v, hp, m_scales=None, v_scales=None, work=None, seed=None, grad_scale=None, stream=None):
    """AdamWPlan(params, m, v, m_scales, v_scales, work).step(grads, hp, seed, grad_scale, stream), for a single step. Making the plan is most
    of its host time: 64 tensors 0.34 ms with states in fp32 and 0.48 ms in 8 bits, against 0.08 and 0.09 of a kept plan's step."""
    AdamWPlan(params, m, v, m_scales, v_scales, work).step(grads, hp, seed, grad_scale, stream)
