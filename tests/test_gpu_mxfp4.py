"""MXFP4: quantisation bit for bit against its definition, the product and the feed-forward block
against fp64.

The product of two codes and their scales is exact; a fp32 sum of n of them is off by at most n 2^-24
of the sum of their magnitudes, a bf16 result by 2^-8 of itself more."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe

pytestmark = pytest.mark.gpu

BF, U, FN = 2.0 ** -8, 2.0 ** -24, 2.0 ** -20
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def rand(*shape, seed=0, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def quantize(x):
    """The definition on the CPU in fp64: (codes, scales)."""
    rows, width = x.shape
    v = x.double().cpu().reshape(rows, width // 32, 32)
    bad = ~torch.isfinite(v).all(dim=2)
    v = torch.where(bad.unsqueeze(2), torch.zeros_like(v), v)
    top = v.abs().amax(dim=2)
    power = torch.frexp(top).exponent.long() - 1
    byte = torch.where(top > 0, power - 2 + 127, torch.zeros_like(power)).clamp(0, 254)
    y = torch.ldexp(v, (127 - byte).unsqueeze(2))
    dist = (y.abs().unsqueeze(3) - GRID).abs()
    near = dist == dist.amin(dim=3, keepdim=True)
    index = torch.arange(8).expand_as(near)
    # of two equally near, the even code
    code = torch.where(near, index + 8 * (index % 2), torch.full_like(index, 99)).amin(dim=3) % 8
    code = code + 8 * torch.signbit(y).long()
    code = torch.where(bad.unsqueeze(2), torch.zeros_like(code), code).reshape(rows, width // 2, 2)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), byte.to(torch.uint8)


def values(codes, scales):
    codes, scales = codes.cpu().long(), scales.cpu().long()
    c = torch.stack([codes & 15, codes >> 4], dim=2).reshape(codes.shape[0], -1)
    v = GRID[c & 7] * torch.where(c >= 8, -1.0, 1.0).double()
    v = torch.ldexp(v, (scales - 127).repeat_interleave(32, dim=1))
    return torch.where(scales.repeat_interleave(32, dim=1) == 255, torch.full_like(v, float("nan")), v)


def q_values(x):
    return values(*quantize(x)).cuda()


@pytest.mark.parametrize("rows,width", [(1, 32), (1, 7168), (3, 96), (65, 1024), (257, 992), (1000, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantize(rows, width, dtype):
    x = rand(rows, width, seed=rows, dtype=dtype) * torch.exp2(
        torch.randint(-12, 12, (1, width), device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    x = x.to(dtype)
    q = moe.mxfp4_quantize(x)
    codes, scales = quantize(x)
    assert torch.equal(q.scales.cpu(), scales)
    assert torch.equal(q.codes.cpu(), codes)
    back = moe.mxfp4_dequantize(q, dtype=torch.float32)
    assert torch.equal(back.double().cpu(), values(codes, scales))
    assert torch.equal(moe.mxfp4_dequantize(q), back.bfloat16())
    assert torch.equal(moe.mxfp4_dequantize(q, dtype=torch.float16), back.half())


def test_quantize_borders():
    """Every border between codes and its neighbours, zeros of both signs, subnormals, the largest
    values, and blocks with infinities and NaN."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99]
    row = []
    for m in mids:
        m = torch.tensor(m)
        row += [m, torch.nextafter(m, torch.tensor(9.0)), torch.nextafter(m, torch.tensor(0.0))]
    row = torch.stack(row + [torch.tensor(0.0), torch.tensor(-0.0)])
    blocks = [row, -row, row * 2.0 ** -120, row * 2.0 ** -127, row * 2.0 ** -140, row * 2.0 ** 125,
              torch.zeros(32), -torch.zeros(32), torch.full((32,), 1e-45), torch.full((32,), 3.4e38)]
    for special in (float("inf"), float("-inf"), float("nan")):
        b = torch.ones(32)
        b[17] = special
        blocks.append(b)
    x = torch.stack(blocks).reshape(1, -1).float()
    q = moe.mxfp4_quantize(x.cuda())
    codes, scales = quantize(x)
    assert torch.equal(q.scales.cpu(), scales)
    assert torch.equal(q.codes.cpu(), codes)
    back = moe.mxfp4_dequantize(q, dtype=torch.float32).cpu()
    assert torch.equal(back.double().nan_to_num(nan=123.0), values(codes, scales).nan_to_num(nan=123.0))
    assert back[0, -96:].isnan().all()
    x16 = x.bfloat16()
    assert torch.equal(moe.mxfp4_quantize(x16.cuda()).codes.cpu(), quantize(x16)[0])


def test_every_code_and_scale_reads_back():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).repeat(16, 1).T.contiguous()
    q = moe.Mxfp4(codes.cuda(), scales.cuda())
    want = values(codes, scales).float()  # 6 * 2^127 and more: infinity; below 2^-149: 0
    got = moe.mxfp4_dequantize(q, dtype=torch.float32).cpu()
    assert torch.equal(got.nan_to_num(nan=5.0), want.nan_to_num(nan=5.0))


PRODUCTS = [(1, 8, 32), (1, 4096, 7168), (2, 264, 992), (7, 72, 256), (16, 512, 1024), (33, 136, 64),
            (64, 128, 2048), (128, 128, 256), (129, 1000, 480), (300, 264, 7168), (777, 72, 992), (17, 1000, 992), (48, 264, 704), (64, 4096, 1024),
            (151, 6304, 64), (791, 4800, 64), (2228, 3648, 64)]


def product_close(got, a, b, n, rounded):
    ref = a @ b.T
    tol = (n + 1) * U * (a.abs() @ b.abs().T) + (BF * ref.abs() if rounded else 0) + 1e-30
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(M, N, K, codes, dtype):
    x = rand(M, K, seed=M)
    w = rand(N, K, seed=N, dtype=torch.float32, scale=K ** -0.5)
    wq = moe.mxfp4_quantize(w)
    pad = 4096
    whole = torch.full((M * N + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    out = whole[pad:pad + M * N].view(M, N)
    moe.mxfp4_matmul(moe.mxfp4_quantize(x) if codes else x, wq, out=out)
    product_close(out, q_values(x), values(wq.codes, wq.scales).cuda(), K, dtype == torch.bfloat16)
    assert (whole[:pad] == 7).all() and (whole[pad + M * N:] == 7).all()


def test_a_nearly_empty_last_round_of_tiles():
    """A product of 272 and 289 tiles of 256 x 256: two launches, the second from row 3840 or 3855 on."""
    for M, N, K in ((4100, 4096, 544), (4300, 4232, 256)):
        x, w = rand(M, K, seed=1), rand(N, K, seed=2)
        got = moe.mxfp4_matmul(x, moe.mxfp4_quantize(w), dtype=torch.float32)
        product_close(got, q_values(x), q_values(w), K, False)


def test_product_of_row_slices_and_odd_scale_rows():
    """Rows taken out of larger matrices: scales then start at any byte."""
    x, w = rand(70, 96, seed=1), rand(40, 96, seed=2)
    xq, wq = moe.mxfp4_quantize(x), moe.mxfp4_quantize(w)
    a = moe.Mxfp4(xq.codes[1:68], xq.scales[1:68])
    b = moe.Mxfp4(wq.codes[3:35], wq.scales[3:35])
    product_close(moe.mxfp4_matmul(a, b, dtype=torch.float32), q_values(x)[1:68], q_values(w)[3:35], 96,
                  False)


@pytest.mark.parametrize("M", [3, 40, 150])
def test_scales_of_all_sizes(M):
    """Scales from 2^-40 to 2^40 in every block position, and NaN blocks, which reach their rows only."""
    K, N = 544, 72
    g = torch.Generator().manual_seed(3)
    codes = torch.randint(0, 256, (M, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(87, 167, (M, K // 32), generator=g, dtype=torch.uint8)
    w = rand(N, K, seed=4)
    wq = moe.mxfp4_quantize(w)
    out = moe.mxfp4_matmul(moe.Mxfp4(codes.cuda(), scales.cuda()), wq, dtype=torch.float32)
    product_close(out, values(codes, scales).cuda(), q_values(w), K, False)
    scales[1, K // 32 - 1] = 255
    marked = moe.mxfp4_matmul(moe.Mxfp4(codes.cuda(), scales.cuda()), wq, dtype=torch.float32)
    assert marked[1].isnan().all()
    keep = [m for m in range(M) if m != 1]
    assert torch.equal(marked[keep], out[keep])


FFN = [(1, 32, 32), (1, 7168, 256), (3, 96, 64), (8, 512, 256), (40, 992, 160), (130, 256, 736), (257, 64, 96),
       (20, 704, 256), (57, 1024, 2048), (64, 512, 160), (16, 7168, 2048), (66, 64, 64), (151, 6304, 64), (523, 64, 928), (1197, 64, 1632),
       (4146, 64, 928), (2228, 3648, 64), (523, 4800, 928)]


@pytest.mark.parametrize("T,H,I", FFN)
def test_block(T, H, I):
    """h is quantised from its fp32 value: where that value is nearer to a border between codes (or its
    block's maximum to a power of two) than its own error, either code is right, and the bound holds the
    difference."""
    x = rand(T, H, seed=T)
    w13 = moe.mxfp4_quantize(rand(2 * I, H, seed=5, dtype=torch.float32, scale=H ** -0.5))
    w2 = moe.mxfp4_quantize(rand(H, I, seed=6, dtype=torch.float32, scale=I ** -0.5))
    out = moe.mxfp4_ffn_forward(x, w13, w2)
    a, b = q_values(x), values(w13.codes, w13.scales).cuda()
    gu, gu_tol = a @ b.T, (H + 1) * U * (a.abs() @ b.abs().T)
    g, u = gu[:, :I], gu[:, I:]
    h = g * torch.sigmoid(g) * u
    h_tol = 1.1 * gu_tol[:, :I] * u.abs() + gu_tol[:, I:] * g.abs() + FN * (g * u).abs()
    q = q_values(h)
    sign = torch.where(h < 0, -1.0, 1.0).double()
    either = torch.maximum((q_values(h + sign * h_tol) - q).abs(), (q_values(h - sign * h_tol) - q).abs())
    w = values(w2.codes, w2.scales).cuda()
    ref = q @ w.T
    tol = BF * ref.abs() + 1.01 * (either @ w.abs().T) + (I + 1) * U * (q.abs() @ w.abs().T) + 1e-30
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max()


def test_block_is_the_products_in_turn():
    """The block against its own parts: quantise, product, SwiGLU, quantise, product."""
    T, H, I = 50, 512, 256
    x = rand(T, H, seed=7)
    w13, w2 = moe.mxfp4_quantize(rand(2 * I, H, seed=8)), moe.mxfp4_quantize(rand(H, I, seed=9))
    gu = moe.mxfp4_matmul(moe.mxfp4_quantize(x), w13, dtype=torch.float32)
    h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    want = moe.mxfp4_matmul(moe.mxfp4_quantize(h), w2).float()
    got = moe.mxfp4_ffn_forward(x, w13, w2).float()
    # codes that differ by the two ways to round silu: few, so the norms agree to a rounding
    assert ((got - want).norm() / want.norm()).item() <= 2 * BF


def test_trained_block_served_in_4_bits():
    """The operators together: a step of the bf16 block, its weights moved along the gradients,
    quantised, and served; the result stays within what the quantised weights and activations give."""
    T, H, I = 48, 256, 160
    x, w13 = rand(T, H, seed=10), rand(2 * I, H, seed=11, scale=H ** -0.5)
    w2, d = rand(H, I, seed=12, scale=I ** -0.5), rand(T, H, seed=13)
    gu = torch.empty(T, 2 * I, device="cuda")
    moe.ffn_forward(x, w13, w2, gate_up=gu)
    _, dw13, dw2 = moe.ffn_backward(d, x, gu, w13, w2)
    w13, w2 = w13 - 1e-3 * dw13, w2 - 1e-3 * dw2
    q13, q2 = moe.mxfp4_quantize(w13), moe.mxfp4_quantize(w2)
    served = moe.mxfp4_ffn_forward(x, q13, q2)
    wide = moe.ffn_forward(moe.mxfp4_dequantize(moe.mxfp4_quantize(x)), moe.mxfp4_dequantize(q13),
                           moe.mxfp4_dequantize(q2))
    # between the two lies the quantisation of h alone: an e2m1 value is off by at most half a step,
    # a third of the value above 0.5 of the unit and 0.25 units below; 6 to 8 units saturate (a quarter)
    h = torch.nn.functional.silu((a := moe.mxfp4_matmul(x, q13, dtype=torch.float32))[:, :I]) * a[:, I:]
    q = q_values(h)
    w = values(q2.codes, q2.scales).cuda()
    bound = 1.01 * ((q - h.double()).abs() @ w.abs().T) + 4 * BF * (h.double().abs() @ w.abs().T)
    assert ((served.double() - wide.double()).abs() <= bound).all()


def test_empty_and_repeated():
    w = moe.mxfp4_quantize(rand(64, 96))
    none = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    assert moe.mxfp4_matmul(none, w).shape == (0, 64)
    assert moe.mxfp4_quantize(none).shape == (0, 96)
    assert moe.mxfp4_dequantize(moe.mxfp4_quantize(none)).shape == (0, 96)
    x = rand(200, 96)
    assert torch.equal(moe.mxfp4_matmul(x, w), moe.mxfp4_matmul(x, w))
    assert torch.equal(moe.mxfp4_matmul(x, w), moe.mxfp4_matmul(moe.mxfp4_quantize(x), w))


@pytest.mark.parametrize("T", [1, 24, 140])
def test_captured_block_replays(T):
    H, I = 288, 160
    x = rand(T, H, seed=14)
    w13, w2 = moe.mxfp4_quantize(rand(2 * I, H, seed=15)), moe.mxfp4_quantize(rand(H, I, seed=16))
    out, prod = torch.empty_like(x), torch.empty(T, 2 * I, device="cuda")
    ws = torch.empty(max(moe.ffn_workspace_size(T, H, I, moe.MOE_FFN_FORWARD_MXFP4),
                         moe.mxfp4_matmul_workspace_size(T, 2 * I, H, True)), dtype=torch.uint8,
                     device="cuda")

    def step():
        moe.mxfp4_ffn_forward(x, w13, w2, out=out, workspace=ws)
        moe.mxfp4_matmul(x, w13, out=prod, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (17, 18, 19):
        x.copy_(rand(T, H, seed=seed))
        out.zero_()
        prod.zero_()
        graph.replay()
        got = out.clone(), prod.clone()
        torch.cuda.synchronize()
        step()
        assert torch.equal(got[0], out) and torch.equal(got[1], prod)


def test_refusals():
    x, w = rand(4, 64), moe.mxfp4_quantize(rand(8, 64))
    with pytest.raises(TypeError):
        moe.mxfp4_quantize(x.double())
    with pytest.raises(ValueError):
        moe.mxfp4_quantize(rand(4, 48))
    with pytest.raises(ValueError):
        moe.mxfp4_quantize(x.T)
    with pytest.raises(TypeError):
        moe.mxfp4_matmul(x.float(), w)
    with pytest.raises(TypeError):
        moe.mxfp4_matmul(x, x)
    with pytest.raises(TypeError):
        moe.mxfp4_matmul(x, w, dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.mxfp4_matmul(rand(4, 96), w)
    with pytest.raises(ValueError):
        moe.mxfp4_matmul(x, moe.Mxfp4(w.codes[:7], w.scales[:7]))
    with pytest.raises(ValueError):
        moe.mxfp4_matmul(rand(40, 64), w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        moe.Mxfp4(w.codes, w.scales[:, :1].contiguous())
    with pytest.raises(ValueError):
        moe.Mxfp4(w.codes[:, :24].contiguous(), w.scales)
    with pytest.raises(ValueError):
        moe.mxfp4_ffn_forward(x, w, w)
