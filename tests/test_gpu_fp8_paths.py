"""Paths of the FP8 products and experts that depend on sizes: the kernels for a few rows and the tiles, at
the sizes where one ends and another begins."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe
from tests import fp8_oracle as o
from tests.test_gpu_fp8 import product_close, published, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 4096, 59392), (4, 4096, 15104), (4, 4096, 15360)])
def test_the_longest_rows_quantised_on_the_way(M, N, K):
    """The most that 64 KB of LDS hold with one and four rows (tests/test_fp8_rows_host.py), and one more."""
    x, w = rand(M, K, seed=M), published(N, K, seed=N)
    a, b = o.q_values(x), o.values(w.codes, w.scales, 128)
    for dtype in (torch.bfloat16, torch.float32):
        product_close(moe.fp8_matmul(x, w, dtype=dtype), a, b, K)


@pytest.mark.parametrize("M,N,K", [(1, 7168, 1024), (4, 7168, 2048), (1, 256, 8192), (3, 1024, 8192), (2, 7168, 7168),
                                   (1, 1024, 14336), (4, 8192, 1040), (5, 7168, 1024), (16, 512, 7168)])
def test_a_bf16_operand_and_its_codes_give_the_same_bits(M, N, K):
    x, w = rand(M, K, seed=M), published(N, K, seed=N)
    q = moe.fp8_quantize(x)
    for dtype in (torch.bfloat16, torch.float32):
        out = moe.fp8_matmul(x, w, dtype=dtype)
        assert torch.equal(out, moe.fp8_matmul(q, w, dtype=dtype)), dtype
        product_close(out, o.values(q.codes, q.scales, 1), o.values(w.codes, w.scales, 128), K)
