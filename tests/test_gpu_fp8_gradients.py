"""One gradient of an FP8 product alone, as the C ABI offers it (da or db NULL, and with it what only it
reads)."""
import ctypes

import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe
from tests.test_gpu_fp8 import GRADS, published, rand
from w4a16_int4_grouped_moe_amd import _fp8

pytestmark = pytest.mark.gpu


def backward(d, a, w, scales, M, N, K, dtype, da, db, ws):
    at = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    kind = moe.MOE_TYPE_BF16 if dtype == torch.bfloat16 else moe.MOE_TYPE_FP32
    return _fp8._library().moe_fp8_matmul_backward(
        at(d), at(a), at(w), at(scales), M, N, K, kind, at(da), at(db), at(ws), 0 if ws is None else ws.numel(),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


@pytest.mark.parametrize("M,N,K", [*GRADS, (2000, 1360, 1008)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_gradient_alone(M, N, K, dtype):
    a, w, d = rand(M, K, seed=M), published(N, K, seed=N), rand(M, N, seed=K)
    want_a, want_b = moe.fp8_matmul_backward(d, a, w, dtype=dtype)
    need = moe.fp8_matmul_backward_workspace_size(M, N, K)
    room = torch.full((need + 512,), 0xff, dtype=torch.uint8, device="cuda")
    ws = room[256:256 + need]
    da, db = torch.full_like(want_a, 7), torch.full_like(want_b, 7)
    assert backward(d, None, w.codes, w.scales, M, N, K, dtype, da, None, ws) == moe.MOE_OK
    assert torch.equal(da, want_a)
    ws.fill_(0xff)
    assert backward(d, a, None, None, M, N, K, dtype, None, db, ws) == moe.MOE_OK
    assert torch.equal(db, want_b)
    assert (room[:256] == 0xff).all() and (room[256 + need:] == 0xff).all()


def test_no_tokens():
    """db alone is cleared, da alone nothing."""
    w = published(136, 144, seed=1)
    db = torch.full((136, 144), 3.0, device="cuda")
    assert backward(None, None, None, None, 0, 136, 144, torch.float32, None, db, None) == moe.MOE_OK
    assert (db == 0).all()
    da = torch.full((8,), 3.0, device="cuda")
    assert backward(None, None, w.codes, w.scales, 0, 136, 144, torch.float32, da, None, None) == moe.MOE_OK
    assert (da == 3).all()
