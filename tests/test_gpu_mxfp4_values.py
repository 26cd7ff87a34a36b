"""MXFP4's special values wherever values are quantised: by mxfp4_quantize, by the launch ahead of the
tiled products, by the few-row kernels (x in bf16, h in fp32) and in the tiles' way out (h).

Operands are chosen so that every sum has one term or is exact in fp32, and the second operand is the
identity: results are the quantised values themselves, so everything is compared bit for bit."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe

from . import ffn_cuts
from .test_gpu_mxfp4 import quantize, values

pytestmark = pytest.mark.gpu

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def same(got, want):
    """Equal values, NaN where NaN is wanted."""
    got, want = got.double().cpu(), want.double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


def matrix(v, power=0):
    """An Mxfp4 of values of the grid times 2^power."""
    code = torch.zeros(v.shape, dtype=torch.uint8)
    for i, m in enumerate(GRID):
        code[v.abs() == m] = i
    assert torch.equal(torch.tensor(GRID)[code.long()], v.abs())
    code += 8 * (v < 0).to(torch.uint8)
    code = code.reshape(v.shape[0], -1, 2)
    scales = torch.full((v.shape[0], v.shape[1] // 32), 127 + power, dtype=torch.uint8)
    return moe.Mxfp4((code[..., 0] + 16 * code[..., 1]).cuda(), scales.cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_code_and_scale_in_16_bits(dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).repeat(16, 1).T.contiguous()
    got = moe.mxfp4_dequantize(moe.Mxfp4(codes.cuda(), scales.cuda()), dtype=dtype)
    # every value is exact in fp32 (6 * 2^127 and more: infinity), so this rounds once
    same(got, values(codes, scales).float().to(dtype))


@pytest.mark.parametrize("rows", [(0, 255), (0, 16), (100, 116), (239, 255), (0, 24), (60, 124)])
def test_every_pair_of_scales(rows):
    """2^(a - 127) * 2^(b - 127) for all bytes below 255: infinities and subnormals as fp32 has them."""
    one = torch.zeros(255, 32)
    one[:, 5] = 1.0
    ones = matrix(one)
    scales = torch.arange(255, dtype=torch.uint8).reshape(255, 1).cuda()
    a = moe.Mxfp4(ones.codes[rows[0]:rows[1]], scales[rows[0]:rows[1]])
    b = moe.Mxfp4(torch.cat([ones.codes, ones.codes[:1]]), torch.cat([scales, scales[:1]]))
    byte = torch.arange(255)
    power = byte[rows[0]:rows[1], None] + torch.cat([byte, byte[:1]])[None] - 254
    want = torch.ldexp(torch.ones(power.shape, dtype=torch.float64), power).float()
    same(moe.mxfp4_matmul(a, b, dtype=torch.float32), want)


def special_rows():
    """bf16 rows of 64: a block of special values, then an ordinary one."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9]).bfloat16()
    near = torch.cat([mids, (mids.view(torch.int16) + 1).view(torch.bfloat16),
                      (mids.view(torch.int16) - 1).view(torch.bfloat16)]).float()
    row = torch.cat([near, torch.tensor([0.0, -0.0])])
    blocks = [row, -row, row * 2.0 ** -100, row * 2.0 ** -124, row * 2.0 ** -127, row * 2.0 ** -130,
              row * 2.0 ** 125, torch.zeros(32), -torch.zeros(32), torch.full((32,), 2.0 ** -133),
              torch.full((32,), 3.38e38)]
    for special in (float("inf"), float("-inf"), float("nan")):
        b = torch.ones(32)
        b[17] = special
        blocks.append(b)
    plain = torch.linspace(-3.0, 5.0, 32)
    return torch.stack([torch.cat([b, plain]) for b in blocks]).bfloat16()


@pytest.mark.parametrize("M", [14, 40, 150])
@pytest.mark.parametrize("power", [0, -3])
def test_x_of_a_product(M, power):
    x = special_rows()
    assert x.shape[0] == 14
    want = values(*quantize(x))
    want[want.isnan().any(dim=1)] = float("nan")  # NaN times 0 is NaN in every column
    want = torch.ldexp(want, torch.tensor(power)).float()
    turn = torch.arange(M) % 14
    x, want = x[turn], want[turn]
    eye = matrix(torch.eye(64), power)
    same(moe.mxfp4_matmul(x.cuda(), eye, dtype=torch.float32), want)
    same(moe.mxfp4_matmul(x.cuda(), eye), want.bfloat16())
    same(moe.mxfp4_matmul(moe.mxfp4_quantize(x.cuda()), eye, dtype=torch.float32), want)


def pieces(total, count):
    """`count` values of the grid whose sum is `total`, a multiple of 0.5."""
    sign, rest, out = (-1.0 if total < 0 else 1.0), abs(total), []
    for m in reversed(GRID[1:]):
        while rest >= m and len(out) < count:
            out.append(sign * m)
            rest -= m
    assert rest == 0
    return out + [0.0] * (count - len(out))


@pytest.mark.parametrize("T,H,I", [(9, 544, 64), (16, 4128, 64), (40, 544, 64), (64, 4128, 96),
                                   *ffn_cuts.MX_VALUES])
def test_h_of_the_block(T, H, I):
    """g = 32 (silu(g) = g in fp32) or 2^-40 (g / 2), u = 2^p times sums of codes that lie on the borders
    between h's codes and next to them; h from subnormal to infinite, and NaN."""
    tops = [1024.0] + [m + d for m in (64.0, 192.0, 320.0, 448.0, 640.0, 896.0) for d in (0, 0.5, -0.5)]
    a = tops + [-v for v in tops[1:13]] + [0.0]
    b = [2040.0] + [m + d for m in (1280.0, 1536.0, 1792.0, 896.0, 128.0) for d in (0, 0.5, -0.5)]
    b = b + [-v for v in b]
    assert len(a) == 32 and len(b) == 32
    sums = torch.tensor((a + b) * ((I + 63) // 64))[:I]
    w1, w3 = torch.zeros(I, H), torch.zeros(I, H)
    w1[:, 3] = 4.0  # with its block's scale 8: g = 32 x[0]
    for i, s in enumerate(sums.tolist()):
        w3[i, 32:] = torch.tensor(pieces(s, H - 32))
    w13 = matrix(torch.cat([w1, w3]))
    w13.scales[:I, 0] = 127 + 3
    down = torch.zeros(H, I)
    n = min(H, I)
    down[torch.arange(n), torch.arange(n)] = 1.0
    rows = [(0, p) for p in (0, -60, -120, 90, 112, 113, 127)]
    rows += [(-45, p) for p in (-93, -95, -97, -100, -104, 60)]
    x = torch.zeros(len(rows) + 2, H)
    for i, (gate, p) in enumerate(rows):
        x[i, :32], x[i, 32:] = 2.0 ** gate, 2.0 ** p
    x[-2:, :32], x[-2:, 32:] = 1.0, 1.0
    x[-2, 40], x[-1, 50] = float("nan"), float("inf")
    gate, move = x[:, :1] * 32, x[:, 33:34]
    silu = torch.where(gate == 32, gate, gate / 2)
    h = silu * (move.double() * sums.double()).float()  # the fp32 u, then h as the kernels multiply
    h[-2:] = float("nan")
    want = values(*quantize(h))
    want[want.isnan().any(dim=1)] = float("nan")
    want = torch.cat([want[:, :n], torch.where(want[:, :1].isnan(), float("nan"), 0.0).expand(-1, H - n)], 1)
    turn = torch.arange(T) % x.shape[0]
    out = moe.mxfp4_ffn_forward(x[turn].bfloat16().cuda(), w13, matrix(down))
    same(out, want[turn].float().bfloat16())
