"""The per-expert / dense product and its gradients at the edges of their ranges on the GPU."""
import math

import numpy as np
import pytest
import torch

import bwd_situ_glu_gb300 as sg
from bwd_situ_glu_gb300 import moe
import _moe_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def test_most_rows():
    """The largest R, 2^31 - 1025 (34 GB a tensor): rows at both ends and in the middle, zeros elsewhere. Eighths up to 1
    make every product and sum exact in fp32, whatever its order; a bf16 result is that sum rounded once."""
    R, N, K = 2 ** 31 - 1025, 8, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    new = lambda *s: (torch.randint(-8, 9, s, generator=g, device=DEV) / 8).to(BF)  # noqa: E731
    places = [slice(0, 40), slice(2 ** 30 - 20, 2 ** 30 + 20), slice(R - 300, R)]
    w, a, dz = new(N, K), torch.zeros(R, K, dtype=BF, device=DEV), torch.zeros(R, N, dtype=BF, device=DEV)
    for r in places:
        a[r], dz[r] = new(r.stop - r.start, K), new(r.stop - r.start, N)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = sg.situ_linear(a, w, status=st)
    da, dw, db = sg.situ_linear_bwd(dz, a, w, status=st)
    assert st.item() == 0
    for r in places:
        assert torch.equal(out[r], (a[r].float() @ w.float().t()).to(BF)) and torch.equal(da[r], (dz[r].float() @ w.float()).to(BF))
    for r in (slice(40, 4000), slice(2 ** 30 + 20, 2 ** 30 + 4000), slice(R - 4000, R - 300)):
        assert not out[r].any() and not da[r].any()
    assert torch.equal(dw, sum(dz[r].float().t() @ a[r].float() for r in places))
    assert torch.equal(db, sum(dz[r].float().sum(0) for r in places))
