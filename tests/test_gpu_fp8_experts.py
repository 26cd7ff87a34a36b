"""The FP8 experts' values in the 2-norm (tests/fp8_experts_oracle.py: what the bound is made of; that it tells
mistakes is tested on the CPU), over their paths."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe
from tests import fp8_experts_oracle as x
from tests.fp8_rows_host import FEW_EXPERTS, PAIRS, SPANS
from tests.test_fp8_experts_oracle import SIZES

pytestmark = pytest.mark.gpu


def run(act, ids, weights, w13, w2, base, **given):
    return moe.fp8_experts_forward(act, ids, weights, moe.Fp8(*w13, block=128), moe.Fp8(*w2, block=128),
                                   expert_base=base, **given)


def check(args, bound=x.BOUND):
    out = run(*args)
    whole, each = x.distance(out, *args)
    assert whole <= bound / x.BOUND and each <= 1, (whole, each)
    assert torch.equal(out, run(*args))
    return out


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_experts_in_the_norm(size):
    args = (*x.inputs(*size, seed=size[0], device="cuda"), size[-1])
    check(args)
    ids = args[1]
    if len(ids) > 1:  # a token without experts, one of another GPU's alone, the same id twice
        ids[0] = -1
        ids[1] = size[4] + 3
        ids[-1] = size[-1]
        out = check(args)
        assert (out[:2] == 0).all()


@pytest.mark.parametrize("T", [1, 5, 90, 600])
def test_all_tokens_to_one_expert(T):
    args = [*x.inputs(T, 256, 512, 4, 4, 1, 0, seed=T, device="cuda"), 0]
    args[1] = torch.full_like(args[1], 2)
    check(args)


def test_a_run_and_a_shared_expert():
    """Ids and weights from route, weights quantised from bf16, and one more expert in a slot of every token."""
    T, H, I, E, k = 130, 512, 512, 8, 2
    g = torch.Generator("cuda").manual_seed(5)
    act, scores, w13, w2 = (torch.randn(s, generator=g, device="cuda") for s in ((T, H), (T, E), (E + 1, 2 * I, H), (E + 1, H, I)))
    ids, weights = moe.route(scores, k)
    ids = torch.cat([ids, torch.full_like(ids[:, :1], E)], dim=1)
    weights = torch.cat([weights, torch.ones_like(weights[:, :1])], dim=1)
    q13, q2 = (moe.fp8_quantize((w * w.shape[2] ** -0.5).bfloat16(), block=128) for w in (w13, w2))
    check((act.bfloat16(), ids, weights, (q13.codes, q13.scales), (q2.codes, q2.scales), 0))


@pytest.mark.parametrize("size", list(FEW_EXPERTS), ids=lambda s: "-".join(map(str, s)) + " " + FEW_EXPERTS[s])
def test_few_rows_deep_and_in_slices(size):
    """The few-row kernels as decoding uses them: several stages a wave, several slices a work-group, one to four
    pairs a bucket. They sum in fp32."""
    T, H, I, E, k = size
    args = [*x.inputs(T, H, I, E, E, k, 0, seed=T, device="cuda"), 0]
    check(args, x.FP32_SUMS)
    pair = torch.arange(T * k, device="cuda").reshape(T, k)
    for full in (2, 3, 4, 5):  # pairs of an expert; of five, one is in a bucket of its own
        args[1] = (pair // full % E).int()
        check(args, x.FP32_SUMS)


@pytest.mark.parametrize("size", list(SPANS), ids=lambda s: "%d-%d" % s + " %d in turn" % SPANS[s])
def test_column_tiles_in_turn(size):
    """The second product with one, two and four column tiles a work-group, over blocks of every filling."""
    (H, I), E, T = size, len(PAIRS), sum(PAIRS) // 2
    args = [*x.inputs(T, H, I, E, E, 2, 0, seed=H + I, device="cuda"), 0]
    owner = torch.repeat_interleave(torch.arange(E), torch.tensor(PAIRS))
    order = torch.randperm(len(owner), generator=torch.Generator().manual_seed(1))
    args[1] = owner[order].reshape(T, 2).int().cuda()
    out = check(args)
    # in a workspace of exactly the size asked for, full of NaN, with guards around it
    need = moe.fp8_experts_workspace_size(T, H, I, E, 2)
    room = torch.full((need + 512,), 0xff, dtype=torch.uint8, device="cuda")
    assert torch.equal(run(*args, workspace=room[256:256 + need]), out)
    assert (room[:256] == 0xff).all() and (room[256 + need:] == 0xff).all()
