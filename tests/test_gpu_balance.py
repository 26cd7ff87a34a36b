"""The balance loss, its counts and its gradient against fp64.

p is off by at most 2^-18 of itself (the exponential of a difference below 90 that was rounded once:
90 2^-24, and a dozen roundings in the sum over 1024 experts and the division), the loss, sums of p times exact counts, by as
much and its own rounding; the gradient p (c - sum c p) by 2^-17 of p (|c - mean| + sum |c - mean| p)."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe

pytestmark = pytest.mark.gpu

P = 2.0 ** -18


def reference(scores, ids, mask, offsets, dloss):
    z = scores.double()
    (T, S), k = z.shape, ids.shape[1]
    top = z.amax(dim=1, keepdim=True) if S else z
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(z - top)
    total = p.sum(dim=1, keepdim=True)
    p = torch.where(total == 0, torch.zeros_like(p), p / total)
    off = [0, T] if offsets is None else offsets.tolist()
    keep = torch.ones(T, dtype=torch.bool, device=z.device) if mask is None else mask
    groups = [torch.nonzero(keep[a:b]).squeeze(1) + a for a, b in zip(off[:-1], off[1:])]
    live = max(1, sum(g.numel() > 0 for g in groups))
    loss, grad, size = 0.0, torch.zeros_like(z), torch.zeros_like(z)
    counts = torch.zeros(len(groups), S, dtype=torch.int32, device=z.device)
    for i, g in enumerate(groups):
        n = g.numel()
        if n == 0:
            continue
        e = ids[g].reshape(-1).long()
        counts[i] = torch.bincount(e[(e >= 0) & (e < S)], minlength=S).int()
        f = S / (live * k * n * n)
        c = counts[i].double()
        loss = loss + f * (c * p[g].sum(dim=0)).sum()
        # less their mean, which changes nothing, as sum p = 1: the difference keeps its digits
        c = c - n * k // S
        grad[g] = dloss * f * p[g] * (c - (p[g] * c).sum(dim=1, keepdim=True))
        d = c.abs()
        size[g] = dloss * f * p[g] * (d + (p[g] * d).sum(dim=1, keepdim=True))
    tokens = torch.tensor([g.numel() for g in groups], dtype=torch.int32, device=z.device)
    return loss, counts, tokens, grad, size


def problem(T, S, k, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator("cuda").manual_seed(seed)
    scores = (torch.randn((T, S), generator=g, device="cuda") * spread + torch.randn((1, S), generator=g, device="cuda")).to(dtype)
    ids = torch.topk(scores.float(), k, dim=1).indices.int() if T else torch.empty((0, k), dtype=torch.int32, device="cuda")
    return scores, ids, torch.rand(T, generator=g, device="cuda") > 0.3, torch.full((), 1.7, device="cuda")


def check(scores, ids, mask=None, offsets=None, dloss=None):
    k = ids.shape[1]
    dloss = torch.full((), 1.7, device="cuda") if dloss is None else dloss
    loss, counts, tokens = moe.balance_loss(scores, ids, mask=mask, seq_offsets=offsets)
    grad = moe.balance_loss_backward(dloss, scores, counts, tokens, k, mask=mask, seq_offsets=offsets)
    rl, rc, rt, rg, size = reference(scores, ids, mask, offsets, float(dloss))
    assert torch.equal(counts if offsets is not None else counts[None], rc)
    assert torch.equal(tokens, rt)
    assert abs(float(loss) - float(rl)) <= (P + 2.0 ** -24) * abs(float(rl))
    # half a step of the type, and what is below its least normal number
    info = torch.finfo(scores.dtype)
    tol = 2 * P * size + info.eps / 2 * 1.01 * rg.abs() + info.tiny
    err = (grad.double() - rg).abs()
    assert (err <= tol).all(), (err / tol).max()
    again = moe.balance_loss(scores, ids, mask=mask, seq_offsets=offsets)
    assert torch.equal(again[0], loss) and torch.equal(again[1], counts)
    return loss, counts, tokens, grad


SIZES = [(1, 1, 1), (1, 2, 1), (3, 8, 2), (64, 384, 8), (127, 64, 4), (128, 65, 3), (129, 256, 8), (1000, 512, 6),
         (4097, 384, 8), (5000, 130, 16), (300, 1024, 8), (70000, 9, 2)]


@pytest.mark.parametrize("T,S,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_whole_batch(T, S, k, dtype):
    scores, ids, mask, dloss = problem(T, S, k, T, dtype)
    check(scores, ids, None, None, dloss)
    check(scores, ids, mask, None, dloss)


def cuts(T, B, seed, first=0, last=None):
    g = torch.Generator("cuda").manual_seed(seed)
    c = torch.sort(torch.randint(first, (T if last is None else last) + 1, (B + 1,), generator=g, device="cuda")).values
    return c.int()


@pytest.mark.parametrize("T,S,k", [(1, 2, 1), (50, 8, 2), (64, 384, 8), (1000, 384, 8), (5000, 64, 4), (9000, 130, 3)])
@pytest.mark.parametrize("B", [1, 2, 7, 300])
def test_sequences(T, S, k, B):
    scores, ids, mask, _ = problem(T, S, k, T + B)
    check(scores, ids, None, cuts(T, B, 1))  # sequences of length zero, tokens ahead of and behind them
    check(scores, ids, mask, cuts(T, B, 2, first=T // 3, last=T // 2))
    whole = torch.linspace(0, T, B + 1).int().cuda()
    check(scores, ids, mask, whole)


def test_one_sequence_is_the_whole_batch():
    scores, ids, mask, dloss = problem(700, 64, 4, 1)
    off = torch.tensor([0, 700], dtype=torch.int32, device="cuda")
    a, b = check(scores, ids, mask, None, dloss), check(scores, ids, mask, off, dloss)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1][0]) and torch.equal(a[3], b[3])


@pytest.mark.parametrize("T", [0, 1, 90, 3000])
@pytest.mark.parametrize("B", [None, 1, 3])
def test_nothing_takes_part(T, B):
    scores, ids, _, _ = problem(T, 48, 2, 1)
    off = None if B is None else torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    loss, counts, tokens, grad = check(scores, ids, mask, off)
    assert loss == 0 and (counts == 0).all() and (tokens == 0).all() and (grad == 0).all()
    if B is not None:  # behind and ahead of all sequences
        check(scores, ids, None, torch.full((B + 1,), T, dtype=torch.int32, device="cuda"))
        check(scores, ids, None, off)


@pytest.mark.parametrize("T", [100, 4000])
def test_special_scores(T):
    scores, ids, mask, _ = problem(T, 100, 4, 3, spread=30.0)
    scores[:, 7] = float("-inf")
    scores[5] = float("-inf")   # a token without any finite score
    scores[6, :50] = torch.finfo(torch.float32).min
    ids[9] = -1
    ids[10, 1], ids[10, 2], ids[10, 3] = 100, 1 << 30, -(1 << 31)
    ids[11] = 3                 # the same id in every slot
    mask[:12] = True
    mask[20], mask[21] = False, False
    scores[20], scores[21, 3] = float("nan"), float("inf")  # not looked at
    ids[20] = 5
    loss, counts, tokens, grad = check(scores, ids, mask)
    assert loss.isfinite() and (grad[5] == 0).all() and (grad[20] == 0).all()
    mask[21] = True
    loss, counts, tokens = moe.balance_loss(scores, ids, mask=mask)
    assert loss.isnan()
    grad = moe.balance_loss_backward(torch.ones((), device="cuda"), scores, counts, tokens, 4, mask=mask)
    assert grad[21].isnan().all() and not grad[:20].isnan().any() and not grad[22:].isnan().any()


def test_even_ids_have_loss_one_and_differences_agree():
    """Ids that spread evenly have loss 1 for any scores; the gradient agrees with central
    differences of the fp64 loss at fixed counts."""
    T, S, k = 96, 16, 2
    scores, ids, _, _ = problem(T, S, k, 5)
    even = ((torch.arange(T, device="cuda")[:, None] * k + torch.arange(k, device="cuda")) % S).int()
    loss, _, _, grad = check(scores, even)
    assert abs(float(loss) - 1) <= 2 * P and grad.abs().max() <= 2.0 ** -15 / T
    _, _, _, grad = check(scores, ids, dloss=torch.ones((), device="cuda"))
    for t, e in ((0, 0), (17, 3), (95, 15)):
        step = torch.zeros_like(scores).double()
        step[t, e] = 1e-5
        up, down = (reference(scores.double() + s * step, ids, None, None, 1.0)[0] for s in (1, -1))
        diff = float(up - down) / 2e-5
        assert abs(diff - float(grad[t, e])) <= 1e-6 * abs(diff) + 1e-9 + 2 * P * abs(diff)


def test_counts_are_the_bucketing():
    """The counts agree with the layer's bucketing of the same ids."""
    scores, _, _, _ = problem(500, 48, 4, 8)
    ids, _ = moe.route(scores, 4)
    _, counts, tokens = moe.balance_loss(scores, ids)
    sorted_ids, block_expert, n = moe.align(ids, 48, 1)
    assert int(n) == 2000 == int(counts.sum()) and int(tokens) == 500
    assert torch.equal(torch.bincount(block_expert[:2000].long(), minlength=48).int(), counts)
