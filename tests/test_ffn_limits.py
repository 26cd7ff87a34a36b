"""The largest sizes of include/moe_ffn.h on the host: refused before any launch, or launched whole."""
import ctypes
import os
import shutil

import pytest

import w4a16_int4_grouped_moe_amd as moe

from .test_ffn_boundary import A, B, C, D, W, lib  # noqa: F401 (lib: a fixture)
from .test_sanitizers import CSRC, FLAGS, ROCM_INC, SAN, build, run

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


@pytest.mark.skipif(not shutil.which("g++") or not os.path.isdir(ROCM_INC),
                    reason="host compiler or HIP headers not found")
def test_more_tiles_than_a_launch_holds(tmp_path):
    """tests/sanitize/ffn_launches.cpp, under AddressSanitizer and UndefinedBehaviorSanitizer."""
    exe = str(tmp_path / "ffn_launches")
    build(["g++", "-std=c++17", "-I", ROCM_INC, "-I", CSRC, "-D__HIP_PLATFORM_AMD__", *FLAGS,
           os.path.join(CSRC, "ffn_plan.cpp"), os.path.join(SAN, "ffn_launches.cpp"), "-o", exe])
    rc, out = run(exe)
    assert rc == 0, out[-4000:]
    assert "failed: 0" in out and "runtime error" not in out and "Sanitizer" not in out, out[-4000:]


@pytest.mark.parametrize("wrap", [1 << 32, -(1 << 32), 1 << 64, -(1 << 64)])
def test_sizes_that_c_would_wrap(lib, wrap):  # noqa: F811
    """Python integers outside C's are refused, whatever they would be modulo 2^32 or 2^64."""
    for i in range(4):
        args = [4, 64, 32, moe.MOE_FFN_FORWARD]
        args[i] += wrap if i else wrap << 32  # the first is an int64_t
        with pytest.raises(ValueError):
            moe.ffn_workspace_size(*args)
    for i in range(3):
        args = [4, 64, 32, True]
        args[i] += wrap if i else wrap << 32  # the first is an int64_t
        with pytest.raises(ValueError):
            moe.mxfp4_matmul_workspace_size(*args)
