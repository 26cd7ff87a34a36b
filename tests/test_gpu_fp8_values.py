"""Special values through every kernel that multiplies FP8 codes: the kernels for a few rows, tiles on the FP8
matrix unit (bf16 results) and tiles that widen the codes (fp32 results), the gradients and the experts."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe
from tests import fp8_experts_oracle as x
from tests.test_gpu_fp8 import E4M3, published, rand

pytestmark = pytest.mark.gpu


def put(codes, at, code):
    """codes with `code` at `at`; the sign alternates, as 0x7f and 0xff are both NaN."""
    c = codes.view(torch.uint8).clone()
    for i, (r, k) in enumerate(at):
        c[r, k] = code | (0x80 * (i & 1))
    return c.view(E4M3)


def same_but(out, clean, rows, cols):
    """NaN in these rows and columns, and elsewhere the bits of the clean result."""
    bad = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    bad[list(rows)] = True
    bad[:, list(cols)] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])


# few rows, 64 x 64 and 128 x 128 tiles, 256 x 256 (bf16) and 128 x 256 (fp32) ones; a last stage of 16
SIZES = [(1, 264, 1040), (3, 264, 1040), (12, 264, 1040), (70, 264, 400), (70, 8504, 400), (6560, 1160, 144)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_codes_in_products(M, N, K, dtype):
    a, w = moe.fp8_quantize(rand(M, K, seed=M)), published(N, K, seed=N)
    last = M - 1
    a.codes.view(torch.uint8)[last, 40:60] = 0  # NaN times zero is NaN too
    clean = moe.fp8_matmul(a, w, dtype=dtype)
    at_b = [(0, 0), (131, K - 1), (N - 1, 50)]
    wn = moe.Fp8(put(w.codes, at_b, 0x7f), w.scales, 128)
    same_but(moe.fp8_matmul(a, wn, dtype=dtype), clean, [], [r for r, _ in at_b])
    at_a = [(0, K - 1), (last, 3)]
    an = moe.Fp8(put(a.codes, at_a, 0x7f), a.scales, 1)
    same_but(moe.fp8_matmul(an, w, dtype=dtype), clean, [0, last], [])
    rows = moe.Fp8(wn.codes, torch.ones(-(-K // 128), N, device="cuda"), 1)  # B in 1 x 128 blocks
    same_but(moe.fp8_matmul(an, rows, dtype=dtype),
             moe.fp8_matmul(a, moe.Fp8(w.codes, rows.scales, 1), dtype=dtype), [0, last], [r for r, _ in at_b])


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_largest_codes_and_subnormal_ones(M, N, K, dtype):
    """Codes of +-448 and of 2^-9, whose sums are known: exact in fp32 and in the FP8 matrix unit."""
    codes = torch.full((M, K), 0x7e, dtype=torch.uint8, device="cuda")
    codes[:, 1::2] = 0xfe
    ones = torch.ones(-(-K // 128), M, device="cuda")
    square = torch.ones(-(-N // 128), -(-K // 128), device="cuda")
    w = codes[:1].expand(N, K).contiguous()
    out = moe.fp8_matmul(moe.Fp8(codes.view(E4M3), ones, 1), moe.Fp8(w.view(E4M3), square, 128), dtype=dtype)
    assert (out.float() == torch.tensor(448.0 * 448 * K).to(dtype).float()).all()
    least = moe.Fp8(torch.full_like(codes, 1).view(E4M3), ones, 1)
    out = moe.fp8_matmul(least, moe.Fp8(torch.full_like(w, 0x81).view(E4M3), square, 128), dtype=dtype)
    assert (out.float() == torch.tensor(-(2.0 ** -18) * K).to(dtype).float()).all()


@pytest.mark.parametrize("M,N,K", [(1, 264, 400), (70, 264, 400), (1500, 264, 272)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_codes_in_gradients(M, N, K, dtype):
    a, w, d = rand(M, K, seed=M), published(N, K, seed=N), rand(M, N, seed=K)
    da, db = moe.fp8_matmul_backward(d, a, w, dtype=dtype)
    at = [(0, 0), (131, K - 1), (N - 1, 50)]
    wn = moe.Fp8(put(w.codes, at, 0x7f), w.scales, 128)
    na, nb = moe.fp8_matmul_backward(d, a, wn, dtype=dtype)
    same_but(na, da, [], [k for _, k in at])
    assert torch.equal(nb, db)


@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (90, 8, 2), (400, 2, 1)])  # few rows; tiles of up to 128 and of 256
def test_nan_codes_in_experts(T, E, k):
    args = [*x.inputs(T, 512, 256, E, E, k, 0, seed=T, device="cuda")]
    act, ids, weights, (c13, s13), (c2, s2) = args
    call = lambda p, q: moe.fp8_experts_forward(act, ids, weights, moe.Fp8(p, s13, 128), moe.Fp8(q, s2, 128))  # noqa: E731
    clean, e = call(c13, c2), int(ids[0, 0])
    mine = (ids == e).any(dim=1)
    # a row of W1: the block of h is NaN, and with it the expert's tokens
    bad = c13.clone()
    bad[e] = put(c13[e], [(7, 300)], 0x7f)
    out = call(bad, c2)
    assert out[mine].isnan().all() and torch.equal(out[~mine], clean[~mine])
    # a row of W2: that column of out
    bad = c2.clone()
    bad[e] = put(c2[e], [(260, 255)], 0x7f)
    out = call(c13, bad)
    assert out[mine, 260].isnan().all()
    out[mine, 260] = clean[mine, 260]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("M", [1, 3, 12, 70, 1500])
@pytest.mark.parametrize("powers", [(-126, 0), (-126, 126), (0, -126), (120, -100), (-100, 127), (60, 40), (-60, -66)])
def test_scales_to_the_ends_of_fp32(M, powers):
    """Scales of any power whose product is a normal number: the result is that of scales of 1, moved."""
    N, K, (pa, pb) = 264, 400, powers
    a, w = moe.fp8_quantize(rand(M, K, seed=M)), published(N, K, seed=N)
    ones = lambda s, p: torch.full_like(s, 2.0 ** p)  # noqa: E731
    for block, sb in ((128, w.scales), (1, torch.ones(-(-K // 128), N, device="cuda"))):
        for dtype in (torch.bfloat16, torch.float32):
            base = moe.fp8_matmul(moe.Fp8(a.codes, ones(a.scales, 0), 1), moe.Fp8(w.codes, ones(sb, 0), block), dtype=dtype)
            out = moe.fp8_matmul(moe.Fp8(a.codes, ones(a.scales, pa), 1), moe.Fp8(w.codes, ones(sb, pb), block), dtype=dtype)
            assert torch.equal(out.double(), base.double() * 2.0 ** (pa + pb)), (block, dtype)


def test_dequantised_values_are_fp32_products_rounded():
    """Scales that are no powers of two: the product of code and scale in fp32, then the type."""
    w = published(130, 144, seed=3)
    want = moe.fp8_dequantize(w, dtype=torch.float32)
    s = w.scales.repeat_interleave(128, 0)[:130].repeat_interleave(128, 1)[:, :144]
    assert torch.equal(want, w.codes.float() * s)
    assert torch.equal(moe.fp8_dequantize(w), want.bfloat16())
    assert torch.equal(moe.fp8_dequantize(w, dtype=torch.float16), want.half())


@pytest.mark.parametrize("M", [3, 12, 70, 1500])
def test_small_products_beside_large_ones(M):
    """448 448 - 448 448 and one product more, in every place of a block of 128: fp32 results keep it whatever its
    size, and so do bf16 ones of few rows; the FP8 matrix unit from 2^-13 of 2^16 on, the power of two of the
    large ones' exponents, or in another eight of the block than theirs."""
    K, N, last = 128, 8504 if M == 1500 else 264, 127
    for s in (2.0 ** -6, 1.0, 8.0, 64.0):
        a = torch.zeros((M, K), device="cuda")
        b = torch.ones((N, K), device="cuda")
        place = torch.arange(M, device="cuda") % 126 + 1
        a[torch.arange(M), place] = s
        a[:, 0], a[:, last], b[:, 0], b[:, last] = 448, -448, 448, 448
        args = (moe.Fp8(a.to(E4M3), torch.ones(1, M, device="cuda"), 1),
                moe.Fp8(b.to(E4M3), torch.ones(-(-N // 128), 1, device="cuda"), 128))
        assert (moe.fp8_matmul(*args, dtype=torch.float32) == s).all()
        keeps = (place >= 8) & (place < 120) | (s >= 8) | (M <= 16)
        out = moe.fp8_matmul(*args)
        assert (out[keeps] == s).all() and (out[~keeps].float().abs() <= 8).all()
