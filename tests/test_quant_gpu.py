"""situ_quant_fp8 and situ_dequant_fp8 against the format in 64 bits. Nothing but the code rounds, and it rounds to nearest:
codes and scales have to be equal, and so have decoded values where their type holds them."""
import pytest
import torch

import _fp8_ref as ref

pytestmark = pytest.mark.gpu

ROWS = [(1, 1, 1), (1, 1, 128), (1, 3, 129), (1, 5, 1000), (1, 8, 3584), (1, 257, 7), (1, 4099, 136), (3, 5, 264), (1, 1, 70001),
        (1, 2051, 3584), (2, 33, 4096)]
TILES = [(1, 1, 1), (1, 128, 128), (1, 129, 127), (3, 130, 264), (2, 5, 1000), (5, 384, 256), (1, 1000, 3584), (4, 257, 33)]


def make(shape, dtype, seed=0, spread=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    if spread:      # rows over many binades, values far below their block's largest, zeros
        x *= torch.exp2(torch.randint(-40, 40, (*shape[:2], 1), generator=g, device="cuda").float())
        x *= torch.exp2(torch.randint(-22, 1, shape, generator=g, device="cuda").float())
        x *= torch.rand(shape, generator=g, device="cuda") > 0.05
    return x.to(dtype)


def check(sg, x, rows):
    codes, scales = sg.situ_quant_fp8(x, block_rows=rows)
    three = x if x.dim() == 3 else x[None]
    y, b, _ = ref.quantise(three, rows)
    assert codes.dtype == scales.dtype == torch.uint8 and codes.shape == x.shape
    assert torch.equal(scales.reshape(b.shape).long(), b)
    got = ref.code_values(codes).reshape(y.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(y))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(y))
    assert (codes[torch.isnan(x) | torch.isinf(x)] == 0x7F).all()
    return codes, scales


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", ROWS)
def test_rows(cuda_lib, shape, dtype):
    check(cuda_lib, make(shape, dtype), 1)
    check(cuda_lib, make(shape, dtype)[0].contiguous(), 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", TILES)
def test_weights(cuda_lib, shape, dtype):
    check(cuda_lib, make(shape, dtype, spread=False), 128)
    check(cuda_lib, make(shape, dtype), 128)


def _place(t, offset):
    """t's values in a contiguous tensor that begins `offset` elements into its storage."""
    flat = torch.empty(t.numel() + offset, dtype=t.dtype, device=t.device)
    flat[offset:] = t.reshape(-1)
    return flat[offset:].view(t.shape)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,shape", [(1, (1, 37, 256)), (128, (2, 130, 256))])
@pytest.mark.parametrize("offset", [1, 4, 8])
def test_bases_off_the_vectors(cuda_lib, dtype, rows, shape, offset):
    x = make(shape, dtype)
    codes, scales = check(cuda_lib, x, rows)
    out = _place(torch.zeros(shape, dtype=torch.uint8, device="cuda"), offset)
    s2 = _place(torch.zeros_like(scales), offset)
    cuda_lib.situ_quant_fp8(_place(x, offset), block_rows=rows, codes=out, scales=s2)
    assert torch.equal(out, codes) and torch.equal(s2, scales)
    v = cuda_lib.situ_dequant_fp8(out, s2, block_rows=rows, out=_place(torch.zeros_like(x), offset))
    assert torch.equal(v.double(), ref.values(codes, scales, rows).to(dtype).double())


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("D", [256, 131])
def test_values_that_are_not_finite_and_blocks_without_others(cuda_lib, rows, D):
    for dtype in (torch.bfloat16, torch.float32):
        x = make((2, 140, D), dtype)
        inf, nan = float("inf"), float("nan")
        x[0, 3, 5], x[0, 3, 6], x[0, 4, 7], x[1, 139, D - 1] = inf, -inf, nan, nan
        x[0, 9], x[1, 128:] = 0.0, nan
        x[0, 10], x[0, 11] = inf, -0.0
        check(cuda_lib, x, rows)


def test_scales_at_their_borders(cuda_lib):
    """The largest value of a block at, just below and just above 448 times a power of two, the largest and smallest numbers,
    subnormals, and ties of the code's rounding."""
    x = torch.zeros(1, 24, 128, device="cuda")
    tops = [448.0, 448.0 * (1 + 2.0 ** -23), 448.0 * (1 - 2.0 ** -24), 3.4028234e38, 2.0 ** -117 * 1.75, 2.0 ** -117 * 1.76,
            2.0 ** -118 * 1.75, 2.0 ** -126, 2.0 ** -140, 2.0 ** -149, 1.0, 449.0, 256.0, 447.9, 0.875, 0.8750001, 2.0 ** 120 * 1.75, 1e-30]
    for i, t in enumerate(tops):
        x[0, i, 17] = t
        x[0, i, 18] = -t / 3
        x[0, i, 19:] = torch.linspace(-1, 1, 109, device="cuda") * t
    ties = (torch.arange(128, device="cuda") + 0.5) * 2.0 ** -9     # halves of the smallest steps, and of larger ones
    x[0, 20], x[0, 21], x[0, 22] = ties, ties * 64, -ties * 512
    x[0, 20:23, 127] = 448.0
    check(cuda_lib, x, 1)
    check(cuda_lib, x, 128)


@pytest.mark.parametrize("rows", [1, 128])
def test_every_code_and_scale_decodes(cuda_lib, rows):
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256 * rows, 1)       # [256 * rows, 256]
    scales = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].repeat(1, 2).contiguous()
    want = ref.values(codes, scales, rows)
    for dtype in (torch.float32, torch.bfloat16):
        got = cuda_lib.situ_dequant_fp8(codes, scales, block_rows=rows, dtype=dtype)
        w = want.float().to(dtype)      # fp32 holds every product (2^-135 at least), so bf16 rounds once; 2^136 is inf
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(torch.nan_to_num(got, nan=0.0, posinf=9e37, neginf=-9e37), torch.nan_to_num(w, nan=0.0, posinf=9e37, neginf=-9e37))


@pytest.mark.parametrize("shape,rows", [((7, 1000), 1), ((3, 130, 264), 128), ((5, 33), 1), ((2, 9, 77), 128)])
def test_there_and_back(cuda_lib, shape, rows):
    """At most half a step of E4M3 away: 2^-4 of the value, or 2^-10 of the scale's unit below its smallest normal number."""
    x = make(shape if len(shape) == 3 else (1, *shape), torch.float32, 3, spread=False).reshape(shape)
    codes, scales = cuda_lib.situ_quant_fp8(x, block_rows=rows)
    back = cuda_lib.situ_dequant_fp8(codes, scales, block_rows=rows, dtype=torch.float32)
    three = x if x.dim() == 3 else x[None]
    s = torch.exp2(ref.expand(scales.reshape(-1, *scales.shape[-2:]).double() - 127, three.shape, rows)).reshape(x.shape)
    assert ((back.double() - x.double()).abs() <= torch.maximum(x.double().abs() * 2.0 ** -4, s * 2.0 ** -10)).all()


def test_offsets_past_32_bits(cuda_lib):
    """A tensor of more than 2^32 elements: the last rows and one in the middle."""
    R, D = (1 << 20) + 5, 4096
    x = torch.zeros(R, D, dtype=torch.bfloat16, device="cuda")
    at = [0, 1 << 19, (1 << 20) - 1, 1 << 20, R - 1]
    x[at] = make((1, len(at), D), torch.bfloat16)[0]
    codes, scales = cuda_lib.situ_quant_fp8(x)
    want, ws = cuda_lib.situ_quant_fp8(x[at].contiguous())
    assert torch.equal(codes[at], want) and torch.equal(scales[at], ws)
    back = cuda_lib.situ_dequant_fp8(codes, scales)
    assert torch.equal(back[at], cuda_lib.situ_dequant_fp8(want, ws))
    assert not back[1:1 << 19].any()
    del codes, scales, back
    codes, scales = cuda_lib.situ_quant_fp8(x[None], block_rows=128)
    assert torch.equal(scales[0, -1], cuda_lib.situ_quant_fp8(x[(1 << 20):][None].contiguous(), block_rows=128)[1][0, -1])


def test_on_another_stream_and_into_given_tensors(cuda_lib):
    x = make((1, 300, 1024), torch.bfloat16)[0]
    want, ws = cuda_lib.situ_quant_fp8(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    codes, scales = torch.empty_like(want), torch.empty_like(ws)
    got = cuda_lib.situ_quant_fp8(x, codes=codes, scales=scales, stream=s)
    v = cuda_lib.situ_dequant_fp8(codes, scales, stream=s.cuda_stream)
    s.synchronize()
    assert got[0] is codes and torch.equal(codes, want) and torch.equal(scales, ws)
    assert torch.equal(v, cuda_lib.situ_dequant_fp8(want, ws))


def test_captured_and_replayed(cuda_lib):
    x = make((1, 64, 512), torch.bfloat16)[0]
    codes, scales = cuda_lib.situ_quant_fp8(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.situ_quant_fp8(x, codes=codes, scales=scales)
    x.copy_(make((1, 64, 512), torch.bfloat16, 9)[0])
    graph.replay()
    want, ws = cuda_lib.situ_quant_fp8(x)
    assert torch.equal(codes, want) and torch.equal(scales, ws)


@pytest.mark.parametrize("shape", [(0, 128), (0, 7, 64), (3, 0, 64)])
def test_nothing_to_do(cuda_lib, shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    codes, scales = cuda_lib.situ_quant_fp8(x)
    assert codes.shape == shape and scales.numel() == 0
    assert cuda_lib.situ_dequant_fp8(codes, scales).shape == shape


def test_refusals(cuda_lib):
    sg, x = cuda_lib, make((1, 4, 128), torch.bfloat16)[0]
    codes, scales = sg.situ_quant_fp8(x)
    for call, error in (
            (lambda: sg.situ_quant_fp8(x.half()), TypeError), (lambda: sg.situ_quant_fp8(x[0]), ValueError),
            (lambda: sg.situ_quant_fp8(x.cpu()), ValueError), (lambda: sg.situ_quant_fp8(x.t()), ValueError),
            (lambda: sg.situ_quant_fp8(x, block_rows=64), ValueError), (lambda: sg.situ_quant_fp8(x, codes=codes[:2]), ValueError),
            (lambda: sg.situ_quant_fp8(x, scales=scales.int()), TypeError), (lambda: sg.situ_quant_fp8("x"), TypeError),
            (lambda: sg.situ_dequant_fp8(codes.float(), scales), TypeError), (lambda: sg.situ_dequant_fp8(codes, scales[:1]), ValueError),
            (lambda: sg.situ_dequant_fp8(codes, scales, dtype=torch.float16), TypeError),
            (lambda: sg.situ_quant_fp8(x, codes=x.view(torch.uint8)[:, :128].contiguous().copy_(codes), scales=codes[:, :1]), ValueError)):
        with pytest.raises(error):
            call()
    with pytest.raises(sg.SituGluError) as e:
        sg.situ_quant_fp8(x, codes=x.view(torch.uint8).view(-1)[:512].view(4, 128))
    assert e.value.status == 2
