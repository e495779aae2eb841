"""include/situ_fp8.h and include/situ_adamw.h: every declared function is exported, and bad arguments are refused on the host
before any CUDA call. No call here passes validation, so the pointers are plain integers that are never dereferenced (the
AdamW step's array of tensors is real host memory)."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

import bwd_situ_glu_gb300 as sg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, OVERLAP = 0, 1, 2
A, B, C, D, E, F, G, H, I = (k << 40 for k in range(1, 10))   # far apart, 256-byte aligned
BF16, FP32, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    sg.build()
    return sg.load()


@pytest.mark.parametrize("header,count", [("situ_fp8.h", 4), ("situ_adamw.h", 2)])
def test_every_declared_symbol_is_exported(lib, header, count):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(situ_\w+)\s*\(", text, flags=re.M)
    assert len(names) == count
    assert not [n for n in names if not hasattr(lib, n)]


GOOD = {
    "situ_quant_fp8": dict(x=A, type=BF16, codes=B, scales=C, E=2, R=9, D=300, block=1, stream=0),
    "situ_dequant_fp8": dict(codes=A, scales=B, x=C, type=BF16, E=2, R=9, D=300, block=128, stream=0),
    "situ_linear_fp8_fwd": dict(a=A, as_=B, w=C, ws=D, offsets=E, E=3, bias=F, residual=G, act=1, out=H, out_type=BF16, pre=I, status=0,
                                R=9, N=16, K=32, stream=0),
    "situ_linear_fp8_dgrad": dict(dz=A, dzs=B, w=C, ws=D, offsets=E, E=3, da=F, status=0, R=9, N=16, K=32, stream=0),
}

BAD = {
    "situ_quant_fp8": [dict(x=0), dict(codes=0), dict(scales=0), dict(type=2), dict(type=-1), dict(E=-1), dict(R=-1), dict(D=0), dict(block=64),
                       dict(block=0), dict(x=A + 1), dict(type=FP32, x=A + 2), dict(R=1 << 40, D=1 << 30), dict(E=1 << 40, D=1 << 30)],
    "situ_dequant_fp8": [dict(x=0), dict(codes=0), dict(scales=0), dict(type=2), dict(E=-1), dict(R=-1), dict(D=-4), dict(block=2),
                         dict(x=C + 1), dict(type=FP32, x=C + 2), dict(R=1 << 61)],
    "situ_linear_fp8_fwd": [dict(a=0), dict(as_=0), dict(w=0), dict(ws=0), dict(out=0), dict(offsets=0), dict(E=0), dict(E=1025), dict(N=24),
                            dict(N=8), dict(K=24), dict(N=0), dict(K=-16), dict(R=-1), dict(R=(1 << 31) - 1024), dict(act=4), dict(act=-1),
                            dict(out_type=2), dict(a=A + 8), dict(w=C + 4), dict(out=H + 8), dict(residual=G + 4), dict(pre=I + 2), dict(bias=F + 2),
                            dict(status=2), dict(offsets=E + 4), dict(N=1 << 30, E=1024)],
    "situ_linear_fp8_dgrad": [dict(dz=0), dict(dzs=0), dict(w=0), dict(ws=0), dict(da=0), dict(offsets=0), dict(N=24), dict(K=8), dict(R=-1),
                              dict(da=F + 2), dict(dz=A + 4), dict(w=C + 8), dict(status=1)],
}

# an output over an input, over another output, or a part of one
OVER = {
    "situ_quant_fp8": [dict(codes=A), dict(codes=A + 8), dict(scales=A + 64), dict(scales=B), dict(scales=B + 5399)],
    "situ_dequant_fp8": [dict(x=A), dict(x=B), dict(x=A + 5398)],
    "situ_linear_fp8_fwd": [dict(out=A), dict(out=B), dict(out=C), dict(out=D), dict(out=F), dict(out=G), dict(out=E), dict(pre=H), dict(pre=A),
                            dict(status=H + 4), dict(status=E), dict(status=D)],
    "situ_linear_fp8_dgrad": [dict(da=A), dict(da=B), dict(da=C + 16), dict(da=D), dict(da=E), dict(status=F), dict(status=A)],
}


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in BAD.items() for c in cs], ids=str)
def test_bad_arguments(lib, name, change):
    assert getattr(lib, name)(*{**GOOD[name], **change}.values()) == INVALID


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in OVER.items() for c in cs], ids=str)
def test_overlaps(lib, name, change):
    assert getattr(lib, name)(*{**GOOD[name], **change}.values()) == OVERLAP


@pytest.mark.parametrize("name,change", [("situ_quant_fp8", dict(R=0, x=0)), ("situ_quant_fp8", dict(E=0, codes=0)),
                                         ("situ_dequant_fp8", dict(R=0)), ("situ_linear_fp8_fwd", dict(R=0, out=0)),
                                         ("situ_linear_fp8_dgrad", dict(R=0, da=0))], ids=str)
def test_nothing_to_do(lib, name, change):
    assert getattr(lib, name)(*{**GOOD[name], **change}.values()) == OK


# ---------------------------------------------------------------- AdamW

COLUMNS = dict(w=0, grad=1, m=2, v=3, m_scales=4, v_scales=5, work=6, n=7)
TENSOR = dict(w=A, grad=B, m=C, v=D, m_scales=E, v_scales=F, work=G, n=300)


def step(lib, *tensors, grad_type=BF16, state_type=E4M3, count=None, coefficients=None, grad_scale=None, hp=None, null=False):
    table = np.array([[{**TENSOR, **t}[c] for c in COLUMNS] for t in tensors], dtype=np.int64).reshape(-1, 8)
    hp = sg.adam_params() if hp is None else hp
    return lib.situ_adamw_step(None if null else table.ctypes.data, len(tensors) if count is None else count, grad_type, state_type,
                               None if hp is False else ctypes.byref(hp), 0, coefficients, grad_scale, None)


def test_the_arrays_row_is_the_header_struct():
    text = open(os.path.join(ROOT, "include", "situ_adamw.h")).read()
    fields = re.search(r"typedef struct \{(.*?)\} situ_adamw_tensor;", text, flags=re.S).group(1)
    names = re.findall(r"(\w+);", re.sub(r"/\*.*?\*/", "", fields, flags=re.S))
    assert names == list(COLUMNS)            # seven pointers and an int64: rows of eight 64-bit words


@pytest.mark.parametrize("change", [dict(w=0), dict(grad=0), dict(m=0), dict(v=0), dict(m_scales=0), dict(v_scales=0), dict(n=-1), dict(n=1 << 42),
                                    dict(w=A + 2), dict(grad=B + 1), dict(work=G + 1)], ids=str)
def test_bad_tensors(lib, change):
    assert step(lib, change) == INVALID
    assert step(lib, dict(n=0), change) == INVALID


def test_bad_calls(lib):
    assert step(lib, {}, count=-1) == step(lib, {}, null=True) == step(lib, {}, grad_type=2) == step(lib, {}, state_type=BF16) == INVALID
    assert step(lib, {}, coefficients=H + 2) == step(lib, {}, grad_scale=H + 1) == step(lib, {}, hp=False) == INVALID
    assert step(lib, dict(m=C + 2), state_type=FP32) == step(lib, dict(grad=B + 2), grad_type=FP32) == INVALID
    for bad in (dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan),
                dict(eps=0.0), dict(eps=-1e-8), dict(weight_decay=-0.1), dict(weight_decay=math.inf), dict(step=0)):
        assert step(lib, {}, hp=sg.adam_params(**bad)) == INVALID, bad


@pytest.mark.parametrize("change", [dict(m=A), dict(v=C), dict(w=B), dict(grad=A + 4), dict(grad=C), dict(m_scales=F), dict(m_scales=C + 299),
                                    dict(v_scales=D), dict(work=A + 1198), dict(work=B)], ids=str)
def test_overlaps_within_a_tensor(lib, change):
    assert step(lib, change) == OVERLAP


def test_overlaps_between_tensors(lib):
    far = dict(w=A + (1 << 30), grad=B + (1 << 30), m=C + (1 << 30), v=D + (1 << 30), m_scales=E + (1 << 30), v_scales=F + (1 << 30),
               work=G + (1 << 30))
    for name in ("w", "m", "v", "m_scales", "v_scales", "work"):
        assert step(lib, {}, {**far, name: TENSOR[name]}) == OVERLAP, name
    assert step(lib, {}, {**far, "w": A + 1196}) == step(lib, {}, {**far, "grad": D}) == step(lib, {**far, "w": B}, {}) == OVERLAP
    assert step(lib, {}, grad_scale=A) == step(lib, {}, coefficients=D + 40) == OVERLAP


def test_nothing_to_update(lib):
    assert step(lib) == step(lib, dict(n=0, w=0, grad=0, m=0)) == OK


def test_coefficients(lib):
    """The constants of situ_adam_update_host, formed in double and rounded once, and the key of the seed."""
    hp = sg.adam_params(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=37)
    out = np.zeros(9, dtype=np.uint32)
    assert lib.situ_adamw_coefficients_of(ctypes.byref(hp), 5, out.ctypes.data) == OK
    f = out.view(np.float32)[:8]
    want = [0.9, 0.95, 1e-8, 1 - 0.9, 1 - 0.95, 3e-4 / (1 - 0.9 ** 37), 1 / math.sqrt(1 - 0.95 ** 37), 1 - 3e-4 * 0.1]
    assert f.tolist() == [float(np.float32(w)) for w in want]
    x = 5 * 0x9E3779B1 % 2 ** 32
    for shift, factor in ((16, 0x9E3779B1), (15, 0x6A09E667), (16, 1)):
        x = (x ^ x >> shift) * factor % 2 ** 32
    assert int(out[8]) == x
    assert lib.situ_adamw_coefficients_of(None, 5, out.ctypes.data) == lib.situ_adamw_coefficients_of(ctypes.byref(hp), 5, None) == INVALID
    assert lib.situ_adamw_coefficients_of(ctypes.byref(sg.adam_params(step=0)), 5, out.ctypes.data) == INVALID
