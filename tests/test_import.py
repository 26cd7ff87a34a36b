"""The package without torch: importing it, its constants, its size queries and its build need none,
and importing it where torch is installed does not load it."""
import os
import subprocess
import sys

import pytest

import w4a16_int4_grouped_moe_amd as moe

from .test_sanitizers import ROOT

QUERIES = """
import w4a16_int4_grouped_moe_amd as moe
import w4a16_int4_grouped_moe_amd.build
assert moe.workspace_size(moe.problem(4, 256, 128, 8, 2)) > 0
assert moe.ffn_workspace_size(100, 64, 32, moe.MOE_FFN_BACKWARD) >= 6 * 100 * 32
assert moe.mxfp4_matmul_workspace_size(100, 64, 96, True) >= 100 * 96 * 17 // 32
assert (moe.MOE_TYPE_BF16, moe.MOE_TYPE_FP16, moe.MOE_TYPE_FP32) == (0, 1, 2)
"""


def run(code):
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(moe.LIB_PATH):
        from w4a16_int4_grouped_moe_amd import build

        build.build()


def test_where_torch_is_missing():
    run("import sys\nsys.modules['torch'] = None\n" + QUERIES)


def test_torch_is_not_loaded():
    run(QUERIES + "import sys\nassert 'torch' not in sys.modules\n")


@pytest.mark.parametrize("name,count", [("ffn_forward", 3), ("ffn_backward", 5), ("Mxfp4", 2),
                                        ("mxfp4_quantize", 1), ("mxfp4_dequantize", 1),
                                        ("mxfp4_matmul", 2), ("mxfp4_ffn_forward", 3)])
def test_entry_points_load_it(monkeypatch, name, count):
    """The first call finds torch, whichever entry point it goes to."""
    from w4a16_int4_grouped_moe_amd import _ffn

    monkeypatch.setattr(_ffn, "torch", None)
    with pytest.raises(TypeError, match="must be"):
        getattr(moe, name)(*[1] * count)


def test_a_matrix_of_another_process(monkeypatch):
    """An Mxfp4 that arrived pickled is used before any other entry point ran."""
    import torch

    from w4a16_int4_grouped_moe_amd import _ffn

    q = object.__new__(moe.Mxfp4)
    q._codes, q._scales = torch.zeros(1, 16, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.uint8)
    q._shape = (1, 32)
    monkeypatch.setattr(_ffn, "torch", None)
    with pytest.raises(TypeError, match="dtype must be"):
        moe.mxfp4_dequantize(q, dtype=torch.float64)
