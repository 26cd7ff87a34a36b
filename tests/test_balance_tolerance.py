"""The tolerance of the balance loss's gradient tells a gradient that was lost or turned round, in every type
and for large batches, whose fp16 gradients are subnormal."""
import pytest
import torch

from tests.balance_oracle import LARGE, problem, tolerance
from tests.test_gpu_balance import reference


@pytest.mark.parametrize("T,S,k", [(64, 384, 8), *LARGE])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_lost_gradients_are_told(T, S, k, dtype):
    scores, ids, mask = problem(T, S, k, T, dtype, "cpu")
    for dloss in (1.7, 1.7 * 4096):
        _, _, _, grad, size = reference(scores, ids, mask, None, dloss)
        tol = tolerance(grad, size, dtype)
        over = lambda g: float(((g.to(dtype).double() - grad).abs() / tol).max())  # noqa: E731
        assert over(grad) <= 1
        for wrong in (torch.zeros_like(grad), -grad, 1.1 * grad):
            assert over(wrong) > 5, dloss
        tiny = torch.finfo(dtype).tiny
        flushed = torch.where(grad.abs() < tiny, torch.zeros_like(grad), grad)
        lost = (grad.to(dtype).double().abs() < tiny) & (grad.abs() > 4 * tol)
        assert not lost.any() or over(flushed) > 1
    if dtype == torch.float16 and (T, S, k) in LARGE:
        _, _, _, grad, _ = reference(scores, ids, mask, None, 1.7)
        assert (grad.abs() < torch.finfo(dtype).tiny).double().mean() > 0.5  # what this is about
