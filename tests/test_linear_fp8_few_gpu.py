"""The 8-bit product of few rows, whose weights stream past them: every way in which up to 16 rows, the most it takes, lie over
experts, and one row more. Small whole numbers, whose sums are exact in any order."""
import pytest
import torch

import bwd_situ_glu_gb300 as sg

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def whole(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device=DEV).to(BF)


@pytest.mark.parametrize("counts", [[16], [15], [16, 0, 0], [0, 0, 16], [8, 8], [9, 0, 7], [1] * 16, [0, 1] * 16, [3, 0, 12, 1], [17], [9, 8],
                                    [0] * 1008 + [1] * 16], ids=lambda c: f"{sum(c)}over{len(c)}at{c.index(max(c))}")
@pytest.mark.parametrize("N,K", [(16, 16), (272, 144), (80, 2064)])
@pytest.mark.parametrize("tail", [0, 3])
def test_rows_over_experts(counts, N, K, tail):
    """tail: rows of no expert behind the last, left as they were."""
    E, R = len(counts), sum(counts) + tail
    a, w, bias = whole(R, K, seed=1), whole(E, N, K, seed=2), whole(E, N, seed=3).float()
    off = torch.tensor([0] + counts, device=DEV).cumsum(0)
    out, st = torch.full((R, N), 7.0, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    sg.situ_linear_fp8(a, sg.situ_quant_fp8(w, block_rows=128), off, bias=bias, out=out, status=st)
    of = torch.arange(E, device=DEV).repeat_interleave(torch.tensor(counts, device=DEV))
    n = len(of)
    want = torch.einsum("rk,rnk->rn", a[:n].double(), w.double()[of]) + bias.double()[of]
    assert torch.equal(out[:n].double(), want) and (out[n:] == 7.0).all() and st.item() == 0
