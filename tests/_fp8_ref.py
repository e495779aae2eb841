"""The 8-bit block format in plain torch and 64 bits, for the tests of the operators that use it: scales by frexp, codes
by rounding to a multiple of E4M3's step."""
import torch

BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def log_scale(amax):
    """Least e >= -126 with amax <= 448 * 2^e, of float64 amax (finite)."""
    frac, e = torch.frexp(amax / 448.0)
    e = torch.where(frac == 0.5, e - 1, e)
    return torch.where(amax == 0, -126, e.clamp(min=-126))


def step(y):
    """Distance of E4M3 numbers at |y| <= 448."""
    _, e = torch.frexp(y.abs())
    return torch.exp2((e - 1).clamp(min=-6).double() - 3.0)


def expand(s, shape, rows):
    """Block values [E, R/rows, D/128] for every element of [E, R, D]."""
    return s.repeat_interleave(rows, 1).repeat_interleave(BLOCK, 2)[:, :shape[1], :shape[2]]


def quantise(x, rows):
    """(code values float64 with NaN where x is not finite, scale bytes int64, what they stand for) of x [E, R, D]."""
    E, R, D = x.shape
    x = x.double()
    fine = torch.isfinite(x)
    p = torch.zeros(E, -(-R // rows) * rows, blocks(D) * BLOCK, dtype=torch.float64, device=x.device)
    p[:, :R, :D] = torch.where(fine, x, 0.0)
    amax = p.view(E, -1, rows, blocks(D), BLOCK).abs().amax((2, 4))
    e = log_scale(amax)
    s = torch.exp2(expand(e.double(), x.shape, rows))
    y = torch.where(fine, x, 0.0) / s
    d = step(y)
    y = torch.where(fine, torch.round(y / d) * d, float("nan"))
    return y, e.long() + 127, y * s


def code_values(codes):
    """float64 numbers of E4M3 codes (uint8), from their bits."""
    c = codes.long()
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (8.0 + f) * torch.exp2(e.double() - 10.0))
    v = torch.where((c & 0x7F) == 0x7F, float("nan"), v)
    return torch.where(c >= 128, -v, v)


def values(codes, scales, rows):
    """float64 numbers that codes and scale bytes stand for; a byte of 255 is NaN."""
    three = codes if codes.dim() == 3 else codes[None]
    s = scales if scales.dim() == 3 else scales[None]
    s = torch.where(s == 255, float("nan"), torch.exp2(s.double() - 127.0))
    v = code_values(three) * expand(s, three.shape, rows)
    return v if codes.dim() == 3 else v[0]
