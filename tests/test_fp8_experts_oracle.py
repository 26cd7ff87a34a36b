"""The bound that the FP8 experts are held to (tests/fp8_experts_oracle.py) tells a right pass from passes with a
mistake in them, at the sizes of the GPU tests."""
import pytest
import torch

from tests import fp8_experts_oracle as x

SIZES = [  # T, H, I, local experts, all experts, k, base
    (1, 256, 128, 8, 8, 2, 0), (1, 7168, 256, 2, 2, 1, 0), (5, 512, 1024, 16, 16, 8, 0), (17, 1024, 1024, 2, 2, 2, 0),
    (64, 1024, 512, 6, 6, 2, 0), (300, 640, 256, 5, 5, 3, 0), (700, 256, 256, 2, 4, 2, 1),
    (1500, 128, 128, 7, 16, 8, 3)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_right_passes_are_near_and_mistakes_are_not(size):
    T, H, I, E, total, k, base = size
    args = (*x.inputs(*size, seed=T), base)
    right = x.forward(*args)[0]
    whole, each = x.distance(right.bfloat16(), *args)
    assert whole <= 0.46 and each <= 0.46  # the rounding to bf16 alone: 0.00226 / 0.005
    for mistake in x.MISTAKES:
        if mistake == "the last stage under the scales of the one before" and H == 128:
            continue  # has one stage
        whole, each = x.distance(x.forward(*args, mistake=mistake)[0].bfloat16(), *args)
        assert max(whole, each) > 1, mistake
