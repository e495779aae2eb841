"""include/situ_moe.h: every declared function is exported, and bad arguments are refused on the host before any
CUDA call. As in the checks of situ_glu.h, no call here passes validation, so the pointers are plain
integers that are never dereferenced."""
import os
import re

import pytest

import bwd_situ_glu_gb300 as sg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, OVERLAP = 1, 2
A, B, C, D, E, F, G = (k << 40 for k in range(1, 8))   # far apart, 256-byte aligned
BF16, FP32 = 0, 1


@pytest.fixture(scope="module")
def lib():
    sg.build()
    return sg.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "situ_moe.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(situ_\w+)\s*\(", text, flags=re.M)
    assert len(names) == 14
    assert not [n for n in names if not hasattr(lib, n)]


GOOD = {
    "situ_route_topk": dict(logits=A, type=FP32, p=B, ids=C, T=4, E=8, K=2, stream=0),
    "situ_route_topk_bwd": dict(ids=A, p=B, dp=C, row_of=D, R=8, dlogits=E, type=FP32, T=4, E=8, K=2, stream=0),
    "situ_dispatch_plan": dict(ids=A, p=B, offsets=C, row_of=D, src=E, p_rows=F, ws=G, ws_bytes=1 << 20, T=4, K=2, E=8, stream=0),
    "situ_dispatch": dict(x=A, type=BF16, row_of=B, offsets=C, E=8, weights=D, h=E, T=4, K=2, R=8, D=16, stream=0),
    "situ_combine": dict(o=A, type=BF16, row_of=B, weights=C, residual=D, y=E, T=4, K=2, R=8, D=16, stream=0),
    "situ_combine_bwd": dict(dy=A, o=B, type=BF16, row_of=C, weights=D, offsets=E, E=8, do=F, dw=G, T=4, K=2, R=8, D=16, stream=0),
    "situ_linear_fwd": dict(a=A, w=B, offsets=C, E=3, bias=D, residual=E, act=1, out=F, out_type=BF16, pre=G, status=0, R=9, N=16,
                            K=24, stream=0),
    "situ_linear_act_bwd": dict(dout=A, pre=B, act=1, offsets=C, E=3, dz=D, dbias=E, ws=F, ws_bytes=1 << 20, R=9, N=16, stream=0),
    "situ_linear_dgrad": dict(dz=A, w=B, offsets=C, E=3, da=D, status=0, R=9, N=16, K=24, stream=0),
    "situ_linear_wgrad": dict(dz=A, a=B, offsets=C, E=3, dw=D, dw_type=FP32, ws=E, ws_bytes=1 << 30, status=0, R=9, N=16, K=24,
                              stream=0),
}

BAD = {
    "situ_route_topk": [dict(logits=0), dict(p=0), dict(ids=0), dict(type=2), dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=1025),
                        dict(K=0), dict(K=9), dict(E=64, K=33), dict(logits=A + 2), dict(type=BF16, logits=A + 1), dict(p=B + 2),
                        dict(ids=C + 1)],
    "situ_route_topk_bwd": [dict(ids=0), dict(p=0), dict(dp=0), dict(dlogits=0), dict(R=-1), dict(K=9), dict(type=-1),
                            dict(dlogits=E + 2), dict(row_of=D + 1), dict(dp=C + 2), dict(T=-3), dict(E=2000)],
    "situ_dispatch_plan": [dict(ids=0), dict(offsets=0), dict(row_of=0), dict(src=0), dict(p=0), dict(p_rows=0), dict(K=0),
                           dict(K=1025), dict(E=0), dict(E=1025), dict(T=-1), dict(T=1 << 30, K=4), dict(offsets=C + 4), dict(ids=A + 2),
                           dict(T=100000, ws=0), dict(T=100000, ws_bytes=8), dict(T=100000, ws=G + 2)],
    "situ_dispatch": [dict(x=0), dict(row_of=0), dict(offsets=0), dict(h=0), dict(type=5), dict(T=-1), dict(K=0), dict(R=-1), dict(D=0),
                      dict(E=0), dict(E=1025), dict(x=A + 1), dict(type=FP32, h=E + 2), dict(weights=D + 2), dict(R=1 << 31),
                      dict(T=1 << 30, K=2)],
    "situ_combine": [dict(o=0), dict(row_of=0), dict(y=0), dict(type=2), dict(T=-1), dict(K=0), dict(D=0), dict(D=(1 << 30) + 1),
                     dict(y=E + 1), dict(type=FP32, residual=D + 2), dict(weights=C + 1), dict(row_of=B + 2)],
    "situ_combine_bwd": [dict(dy=0), dict(o=0), dict(row_of=0), dict(weights=0), dict(offsets=0), dict(do=0), dict(dw=0), dict(E=0),
                         dict(type=9), dict(R=-1), dict(dw=G + 1), dict(offsets=E + 4), dict(do=F + 1)],
    "situ_linear_fwd": [dict(a=0), dict(w=0), dict(out=0), dict(offsets=0), dict(E=0), dict(E=1025), dict(N=12), dict(K=20), dict(N=0),
                        dict(K=-8), dict(R=-1), dict(R=1 << 31), dict(act=4), dict(act=-1), dict(out_type=2), dict(a=A + 8), dict(w=B + 2),
                        dict(out=F + 8), dict(residual=E + 4), dict(pre=G + 2), dict(bias=D + 2), dict(status=2)],
    "situ_linear_act_bwd": [dict(dout=0), dict(pre=0), dict(dz=0), dict(offsets=0), dict(act=7), dict(ws=0), dict(ws_bytes=4),
                            dict(N=4), dict(R=-1), dict(E=0), dict(dz=D + 8), dict(dbias=E + 2)],
    "situ_linear_dgrad": [dict(dz=0), dict(w=0), dict(da=0), dict(offsets=0), dict(N=20), dict(K=4), dict(R=-1), dict(da=D + 2),
                          dict(status=1)],
    "situ_linear_wgrad": [dict(dz=0), dict(a=0), dict(dw=0), dict(offsets=0), dict(dw_type=2), dict(N=20), dict(K=4), dict(R=-1),
                          dict(dw=D + 8), dict(offsets=0, E=1, R=100000, ws_bytes=64), dict(offsets=0, E=1, R=100000, ws=0),
                          dict(offsets=0, E=1, R=100000, ws=E + 8)],
}

# an output over an input, over another output, or a part of one
OVER = {
    "situ_route_topk": [dict(p=A), dict(ids=A + 64), dict(ids=B + 8)],
    "situ_route_topk_bwd": [dict(dlogits=A), dict(dlogits=B), dict(dlogits=C - 16), dict(dlogits=D)],
    "situ_dispatch_plan": [dict(row_of=A), dict(src=D), dict(p_rows=B), dict(offsets=A - 8), dict(T=100000, ws=A)],
    "situ_dispatch": [dict(h=A), dict(h=B), dict(h=C), dict(h=D + 16)],
    "situ_combine": [dict(y=A), dict(y=B), dict(y=C), dict(y=D + 32)],
    "situ_combine_bwd": [dict(do=A), dict(do=B), dict(dw=D), dict(dw=F + 4), dict(dw=E)],
    "situ_linear_fwd": [dict(out=A), dict(out=B), dict(out=D), dict(out=E), dict(pre=F), dict(pre=A), dict(status=F + 4), dict(status=C)],
    "situ_linear_act_bwd": [dict(dz=A), dict(dz=B), dict(dbias=D), dict(ws=E), dict(ws=C)],
    "situ_linear_dgrad": [dict(da=A), dict(da=B + 16), dict(status=D), dict(status=A)],
    "situ_linear_wgrad": [dict(dw=A), dict(dw=B), dict(status=D + 4)],
}


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in BAD.items() for c in cs], ids=str)
def test_bad_arguments(lib, name, change):
    assert getattr(lib, name)(*{**GOOD[name], **change}.values()) == INVALID


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in OVER.items() for c in cs], ids=str)
def test_overlaps(lib, name, change):
    assert getattr(lib, name)(*{**GOOD[name], **change}.values()) == OVERLAP


def test_selftest_refusals(lib):
    assert [lib.situ_linear_selftest_wait_timeout(*a, 0) for a in ((0, 0), (A + 2, 0), (A, B + 4))] == [INVALID] * 3


def test_workspaces(lib):
    """Sizes are what the calls ask for; arguments that the calls refuse need none."""
    assert lib.situ_dispatch_plan_workspace(8, 16, 896) == 0
    n = lib.situ_dispatch_plan_workspace(16384, 16, 896)
    assert n > 0 and n % (896 * 4) == 0
    assert lib.situ_dispatch_plan_workspace(-1, 16, 896) == lib.situ_dispatch_plan_workspace(1 << 30, 16, 8) == 0
    assert lib.situ_linear_act_bwd_workspace(1000, 16, 3) >= (1000 // 256 + 3) * 16 * 4
    assert lib.situ_linear_wgrad_workspace(100, 16, 16, 1) == 0
    assert lib.situ_linear_wgrad_workspace(100000, 128, 256, 1) % (128 * 256 * 4) == 0
    assert lib.situ_linear_wgrad_workspace(100000, 128, 12, 1) == 0


def test_python_refuses_before_the_library():
    with pytest.raises(ValueError):
        sg.moe._act("swish")
    with pytest.raises(TypeError):
        sg.moe._type([1.0], "x")
