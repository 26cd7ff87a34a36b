"""Every way the plans cut the products of the feed-forward block and of MXFP4 (tests/ffn_cuts.py), each
result and workspace between guards: nothing outside what the library asked for is written.

Tolerances are those of test_gpu_ffn.py and test_gpu_mxfp4.py."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe

from . import ffn_cuts
from .test_gpu_ffn import close, guarded, inputs, reference_backward, reference_forward
from .test_gpu_mxfp4 import BF, FN, U, product_close, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,I", list(ffn_cuts.FFN))
def test_block(T, H, I):
    x, w13, w2, d = inputs(T, H, I, seed=20)
    ref_gu, gu_tol, y, y_tol = reference_forward(x, w13, w2)
    out, out_ok = guarded((T, H), torch.bfloat16)
    gu, gu_ok = guarded((T, 2 * I), torch.float32)
    ws, ws_ok = guarded((moe.ffn_workspace_size(T, H, I, moe.MOE_FFN_FORWARD),), torch.uint8)
    close(moe.ffn_forward(x, w13, w2, out=out, gate_up=gu, workspace=ws), y, y_tol)
    assert ((gu.double() - ref_gu).abs() <= gu_tol).all()
    assert out_ok() and gu_ok() and ws_ok()
    del ref_gu, gu_tol, y, y_tol
    ws, ws_ok = guarded((moe.ffn_workspace_size(T, H, I, moe.MOE_FFN_BACKWARD),), torch.uint8)
    outs = [guarded(s, torch.bfloat16) for s in ((T, H), (2 * I, H), (H, I))]
    got = moe.ffn_backward(d, x, gu, w13, w2, *(o for o, _ in outs), workspace=ws)
    for value, (ref, tol), (_, ok) in zip(got, reference_backward(d, x, gu, w13, w2), outs):
        close(value, ref, tol)
        assert ok()
    assert ws_ok()


def quantized(x):
    """What the blocks of x stand for, in fp64: the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 units, ties to
    the even code (an even number of steps, as round() takes them), larger values to 6."""
    v = x.double().reshape(x.shape[0], -1, 32)
    top = v.abs().amax(dim=2, keepdim=True)
    power = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    unit = torch.ldexp(torch.ones_like(top), power)
    m = (v / unit).abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    return (torch.copysign((torch.round(m / step) * step).clamp(max=6.0), v) * unit).reshape(x.shape)


def weights(rows, width, seed):
    w = rand(rows, width, seed=seed, dtype=torch.float32, scale=width ** -0.5)
    return moe.mxfp4_quantize(w), quantized(w)


@pytest.mark.parametrize("M,N,K", list(ffn_cuts.MX))
@pytest.mark.parametrize("codes,dtype", [(False, torch.bfloat16), (True, torch.float32)])
def test_mxfp4_product(M, N, K, codes, dtype):
    x = rand(M, K, seed=21)
    wq, w = weights(N, K, 22)
    out, out_ok = guarded((M, N), dtype)
    ws, ws_ok = guarded((moe.mxfp4_matmul_workspace_size(M, N, K, not codes),), torch.uint8)
    moe.mxfp4_matmul(moe.mxfp4_quantize(x) if codes else x, wq, out=out, workspace=ws)
    product_close(out, quantized(x), w, K, dtype == torch.bfloat16)
    assert out_ok() and ws_ok()


# the few-row kernels beside the tiles' sizes: x quantised by them, and by a launch ahead
@pytest.mark.parametrize("T,H,I", [(1, 7168, 256), (9, 512, 288), (33, 992, 160), (64, 512, 160),
                                   *ffn_cuts.MX_FFN])
def test_mxfp4_block(T, H, I):
    x = rand(T, H, seed=23)
    (q13, b), (q2, w) = weights(2 * I, H, 24), weights(H, I, 25)
    out, out_ok = guarded((T, H), torch.bfloat16)
    ws, ws_ok = guarded((moe.ffn_workspace_size(T, H, I, moe.MOE_FFN_FORWARD_MXFP4),), torch.uint8)
    moe.mxfp4_ffn_forward(x, q13, q2, out=out, workspace=ws)
    assert out_ok() and ws_ok()
    a = quantized(x)
    gu, gu_tol = a @ b.T, (H + 1) * U * (a.abs() @ b.abs().T)
    g, u = gu[:, :I], gu[:, I:]
    h = g * torch.sigmoid(g) * u
    h_tol = 1.1 * gu_tol[:, :I] * u.abs() + gu_tol[:, I:] * g.abs() + FN * (g * u).abs()
    q = quantized(h)
    sign = torch.where(h < 0, -1.0, 1.0).double()
    # where h is nearer to a border between codes than its own error, either code is right
    either = torch.maximum((quantized(h + sign * h_tol) - q).abs(),
                           (quantized(h - sign * h_tol) - q).abs())
    ref = q @ w.T
    tol = BF * ref.abs() + 1.01 * (either @ w.abs().T) + (I + 1) * U * (q.abs() @ w.abs().T) + 1e-30
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max()
