"""The largest sizes of include/moe_ffn.h on the host: refused before any launch, or launched whole."""
import ctypes

import pytest

import w4a16_int4_grouped_moe_amd as moe

from .test_ffn_boundary import A, B, C, D, W, lib  # noqa: F401 (lib: a fixture)

MOST = (1 << 31) - 256


@pytest.mark.parametrize("quantize", [0, 1])
def test_the_most_columns(lib, quantize):  # noqa: F811
    n = ctypes.c_size_t(0)
    assert lib.moe_mxfp4_matmul_workspace_size(65, MOST, 32, quantize, ctypes.byref(n)) == moe.MOE_OK
    for cols in (MOST + 8, (1 << 31) - 8):
        assert lib.moe_mxfp4_matmul_workspace_size(65, cols, 32, quantize, ctypes.byref(n)) == \
            moe.MOE_ERR_SHAPE
        assert lib.moe_mxfp4_matmul(A, None if quantize else B, C, D, 65, cols, 32, 0, W, W, 1 << 62,
                                    None) == moe.MOE_ERR_SHAPE
        with pytest.raises(ValueError):
            moe.mxfp4_matmul_workspace_size(65, cols, 32, bool(quantize))
