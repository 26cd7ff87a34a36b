"""The FP8 block operators in fp64, from their definitions (test infrastructure; nothing here is
shared with the library)."""
import torch

F64 = torch.float64


def pad(x, high):
    """x with zeros to whole blocks of high x 128, as [R, high, C, 128]."""
    rows, width = x.shape
    r, c = -(-rows // high), -(-width // 128)
    out = x.new_zeros((r * high, c * 128))
    out[:rows, :width] = x
    return out.reshape(r, high, c, 128)


def cut(x, rows, width):
    r, high, c, _ = x.shape
    return x.reshape(r * high, c * 128)[:rows, :width].contiguous()


def grid():
    """The 127 magnitudes of e4m3 (code 127 is NaN), in the order of their codes."""
    c = torch.arange(127)
    e, m = c // 8, (c % 8).double()
    return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))


GRID = grid()


def scale_of(top):
    """The least 2^e, e >= -126, with top <= 448 2^e; 1 for 0; NaN for infinities and NaN."""
    good = torch.isfinite(top)
    t = torch.where(good & (top > 0), top, torch.ones_like(top))
    m, e = torch.frexp(t)  # t = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)  # 448 = 0.875 * 2^9
    s = ((e.long() + 1023) << 52).view(F64)  # 2^e to the bit
    s = torch.where(top == 0, torch.ones_like(s), s)
    return torch.where(good, s, torch.full_like(s, float("nan")))


def nearest_code(y):
    """The code of the e4m3 nearest to y (|y| <= 448), ties to the even code."""
    g = GRID.to(y.device)
    m = y.abs()
    hi = torch.searchsorted(g, m.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = m - g[lo], g[hi] - m
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return pick + 128 * torch.signbit(y).long()


def quantize(x, high):
    """(codes uint8 [R, K], scales fp64 [K/128, R] (high 1) or [R/128, K/128])."""
    rows, width = x.shape
    v = pad(x.double(), high)
    top = torch.where(torch.isfinite(v), v.abs(), torch.full_like(v, float("inf"))).amax(dim=(1, 3))
    s = scale_of(top)
    bad = ~torch.isfinite(s)
    y = torch.where(bad[:, None, :, None], torch.zeros_like(v),
                    v / torch.where(bad, torch.ones_like(s), s)[:, None, :, None])
    codes = cut(nearest_code(y), rows, width).to(torch.uint8)
    return codes, s.t().contiguous() if high == 1 else s


def values(codes, scales, high):
    """What codes (uint8 or float8) and scales stand for, in fp64."""
    c = codes.view(torch.uint8).long()
    g = torch.cat([GRID, torch.tensor([float("nan")], dtype=F64)]).to(c.device)
    v = g[c & 127] * torch.where(c >= 128, -1.0, 1.0).double()
    s = scales.double().t() if high == 1 else scales.double()
    return cut(pad(v, high) * s[:, None, :, None], *codes.shape)


def q_values(x, high=1):
    return values(*quantize(x, high), high)
