"""Wrong kinds of arguments to the MXFP4 entry points are TypeErrors that name the argument (no GPU)."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe


def on_the_host(rows, width):
    """An Mxfp4 that the constructor would refuse: its tensors are host tensors."""
    q = object.__new__(moe.Mxfp4)
    q._codes = torch.zeros(rows, width // 2, dtype=torch.uint8)
    q._scales = torch.zeros(rows, width // 32, dtype=torch.uint8)
    q._shape = (rows, width)
    return q


@pytest.mark.parametrize("out", [5, [[0.0] * 8], "cuda"])
@pytest.mark.parametrize("dtype", [None, torch.bfloat16])
def test_out_that_is_no_tensor(out, dtype):
    q = on_the_host(8, 64)
    with pytest.raises(TypeError, match="out must be a torch.Tensor"):
        moe.mxfp4_dequantize(q, dtype=dtype, out=out)
    with pytest.raises(TypeError, match="out must be a torch.Tensor"):
        moe.mxfp4_matmul(q, q, out=out, dtype=dtype)
