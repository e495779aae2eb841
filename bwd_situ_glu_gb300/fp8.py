"""Products in 8 bits for the expert layer (C ABI: ``include/situ_fp8.h``).

* ``situ_quant_fp8`` / ``situ_dequant_fp8``: E4M3 codes with a power-of-two scale for each 128 elements of a row, or
  128 x 128 of a weight

A quantised tensor is a pair (codes uint8, scale bytes uint8): a byte b stands for 2^(b-127). ``codes.view(torch.float8_e4m3fn)``
are the codes' values. The conventions are those of the module ``moe``.
"""
from __future__ import annotations

import torch

from bwd_situ_glu_gb300 import _check, load as _lib
from bwd_situ_glu_gb300.moe import _device_now, _elsewhere, _empty, _need, _out, _raw_stream, _type, _CODE, _BF16

_U8 = torch.uint8
BLOCK = 128   # elements of a row (or rows and columns of a weight) that share a scale


def _blocks(n):
    return -(-n // BLOCK)


def _shape3(x, name):
    """(E, R, D) of a tensor [R, D] or [E, R, D] on a CUDA device."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() not in (2, 3) or not x.is_cuda:
        raise ValueError(f"{name} must be a two- or three-dimensional CUDA tensor, got {tuple(x.shape)} on {x.device}")
    return x.shape if x.dim() == 3 else (1, *x.shape)


def _scale_shape(shape, block_rows):
    if block_rows not in (1, BLOCK):
        raise ValueError(f"block_rows must be 1 or {BLOCK}, got {block_rows!r}")
    return (*shape[:-2], shape[-2] if block_rows == 1 else _blocks(shape[-2]), _blocks(shape[-1]))


def situ_quant_fp8(x, block_rows=1, codes=None, scales=None, stream=None):
    """(codes uint8 of x's shape, scales uint8 [.., R/block_rows, D/128], rounded up): x bf16 or fp32 [R, D] or [E, R, D]
    in blocks of 128 elements of a row (block_rows 1, the rows of a product) or 128 x 128 (128, a weight). A block's
    scale is the least power of two (2^-126 at least) with every finite value at most 448 times it; the code is
    x / scale rounded to nearest, ties to even, and 0x7F (NaN) for a value that is not finite."""
    ty = _type(x, "x")
    E, R, D = _shape3(x, "x")
    dev, shape = x.device, tuple(x.shape)
    _need(x, x.dtype, x.shape, dev, "x")
    s_shape = _scale_shape(shape, block_rows)
    if stream is not None or dev.index != _device_now():
        return _elsewhere(stream, x, lambda: situ_quant_fp8(x, block_rows, codes, scales))
    codes = _out(codes, shape, _U8, dev, "codes")
    scales = _out(scales, s_shape, _U8, dev, "scales")
    _check(_lib().situ_quant_fp8(x.data_ptr(), ty, codes.data_ptr(), scales.data_ptr(), E, R, D, block_rows,
                                 _raw_stream(dev.index)))
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
    out = _out(out, shape, dtype, dev, "out")
    _check(_lib().situ_dequant_fp8(codes.data_ptr(), scales.data_ptr(), out.data_ptr(), _CODE[dtype], E, R, D, block_rows,
                                   _raw_stream(dev.index)))
    return out
