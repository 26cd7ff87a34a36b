"""The balance loss's gradient in every type, to half a step of its subnormals too (tests/balance_oracle.py), with
the gradient of the loss as it is and scaled up, as training in fp16 has it."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe
from tests.balance_oracle import LARGE, problem, tolerance
from tests.test_gpu_balance import SIZES, cuts, reference

pytestmark = pytest.mark.gpu


def check(scores, ids, mask, offsets, dloss):
    _, counts, tokens = moe.balance_loss(scores, ids, mask=mask, seq_offsets=offsets)
    grad = moe.balance_loss_backward(torch.full((), dloss, device="cuda"), scores, counts, tokens, ids.shape[1],
                                     mask=mask, seq_offsets=offsets)
    _, _, _, want, size = reference(scores, ids, mask, offsets, dloss)
    over = (grad.double() - want).abs() / tolerance(want, size, scores.dtype)
    assert over.max() <= 1, float(over.max())


@pytest.mark.parametrize("T,S,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dloss", [1.75, 4096.0])
def test_whole_batch(T, S, k, dtype, dloss):
    scores, ids, mask = problem(T, S, k, T, dtype, "cuda")
    check(scores, ids, None, None, dloss)
    check(scores, ids, mask, None, dloss)


@pytest.mark.parametrize("T,S,k", LARGE)
@pytest.mark.parametrize("B", [2, 40])
def test_sequences_in_fp16(T, S, k, B):
    scores, ids, mask = problem(T, S, k, T, torch.float16, "cuda")
    for dloss in (1.75, 4096.0):
        check(scores, ids, mask, cuts(T, B, 1), dloss)
