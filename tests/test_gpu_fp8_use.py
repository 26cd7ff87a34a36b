"""The FP8 and balance-loss operators as programs use them: every cut of a product, captured and replayed
graphs, other streams, workspaces of the exact size, neighbours of the outputs, and a run of them together."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe
from tests import fp8_oracle as o
from tests.fp8_cuts import CUTS
from tests.test_gpu_balance import check as balance_check, reference as balance_reference
from tests.test_gpu_fp8 import E4M3, experts, experts_reference, product_close, published, rand, routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", list(CUTS), ids=lambda s: "-".join(map(str, s)) + "=" + CUTS[s])
def test_every_cut(sizes):
    wide, rows, M, N, K = sizes
    a = moe.fp8_quantize(rand(M, K, seed=M))
    b = moe.fp8_quantize(rand(N, K, seed=N)) if rows else published(N, K, seed=N)
    out = moe.fp8_matmul(a, b, dtype=torch.float32 if wide else torch.bfloat16)
    product_close(out, o.values(a.codes, a.scales, 1), o.values(b.codes, b.scales, b.block), K)


def calls():
    """name -> (a call, its outputs given), over the paths: few rows, tiles, shares of K, gradients,
    experts of both kinds, balance losses of one and of several work-groups."""
    table = {}
    for M, N, K in ((2, 264, 1008), (12, 136, 1008), (40, 4096, 1024), (300, 264, 1008), (69, 72, 1536)):
        for dtype in (torch.bfloat16, torch.float32):
            x, w = rand(M, K, seed=M), published(N, K, seed=N)
            out = torch.empty(M, N, dtype=dtype, device="cuda")
            need = moe.fp8_matmul_workspace_size(M, N, K, True)
            table["matmul", M, dtype] = (lambda ws, x=x, w=w, out=out: moe.fp8_matmul(x, w, out=out, workspace=ws), [out], need)
    x, w, d = rand(201, 272, seed=1), published(264, 272, seed=2), rand(201, 264, seed=3)
    da, db = torch.empty_like(x), torch.empty(264, 272, dtype=torch.bfloat16, device="cuda")
    table["backward"] = (lambda ws: moe.fp8_matmul_backward(d, x, w, da=da, db=db, workspace=ws), [da, db],
                         moe.fp8_matmul_backward_workspace_size(201, 264, 272))
    for T in (3, 200):
        y, (w13, w2), (ids, wt) = rand(T, 256, seed=T), experts(4, 256, 256, seed=5), routing(T, 2, 6, seed=T)
        out = torch.empty_like(y)
        table["experts", T] = (lambda ws, y=y, ids=ids, wt=wt, w13=w13, w2=w2, out=out:
                               moe.fp8_experts_forward(y, ids, wt, w13, w2, out=out, workspace=ws), [out],
                               moe.fp8_experts_workspace_size(T, 256, 256, 4, 2))
    for T, B in ((100, 1), (5000, 1), (5000, 5)):
        g = torch.Generator("cuda").manual_seed(T)
        scores = torch.randn(T, 48, generator=g, device="cuda")
        top = torch.topk(scores, 4, dim=1).indices.int()
        off = torch.linspace(0, T, B + 1).int().cuda()
        counts, tokens = torch.empty(B, 48, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        loss, grad, one = torch.empty((), device="cuda"), torch.empty_like(scores), torch.ones((), device="cuda")

        def step(ws, scores=scores, top=top, off=off, counts=counts, tokens=tokens, loss=loss, grad=grad, one=one):
            loss.copy_(moe.balance_loss(scores, top, seq_offsets=off, counts=counts, tokens=tokens, workspace=ws)[0])
            moe.balance_loss_backward(one, scores, counts, tokens, 4, seq_offsets=off, dscores=grad)
        table["balance", T, B] = (step, [loss, counts, tokens, grad], moe.balance_workspace_size(T, 48, 4, B))
    return table


def bits(outs):
    return [t.clone().view(torch.uint8) if t.dim() else t.clone() for t in outs]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


def test_exact_workspaces_of_any_contents():
    """A workspace of exactly the size asked for, full of 0xff bytes (NaN), with guards around it."""
    for name, (call, outs, need) in calls().items():
        call(None)
        want = bits(outs)
        room = torch.full((need + 512,), 0xff, dtype=torch.uint8, device="cuda")
        for t in outs:
            t.zero_()
        call(room[256:256 + need])
        assert same(bits(outs), want), name
        assert (room[:256] == 0xff).all() and (room[256 + need:] == 0xff).all(), name


def test_graph_replays():
    """All of them in one captured graph, replayed with other work between, against the eager results."""
    table = calls()
    spaces = {n: torch.empty(max(need, 1), dtype=torch.uint8, device="cuda") for n, (_, _, need) in table.items()}
    want = {}
    for name, (call, outs, _) in table.items():
        call(spaces[name])
        want[name] = bits(outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for name, (call, _, _) in table.items():
            call(spaces[name])
    for turn in range(4):
        for name, (_, outs, _) in table.items():
            for t in outs:
                t.zero_()
            spaces[name].fill_(turn)
        graph.replay()
        torch.cuda.synchronize()
        for name, (_, outs, _) in table.items():
            assert same(bits(outs), want[name]), (name, turn)
        x = torch.randn(512, 512, device="cuda")
        (x @ x).sum().item()


def test_two_streams_at_once():
    """Two sets of the calls on two streams, each with its own workspaces, many times over."""
    sets = [calls(), calls()]
    want = []
    for table in sets:
        for call, outs, _ in table.values():
            call(None)
        want.append({n: bits(outs) for n, (_, outs, _) in table.items()})
    spaces = [{n: torch.empty(max(need, 1), dtype=torch.uint8, device="cuda") for n, (_, _, need) in t.items()} for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for table, space, stream in zip(sets, spaces, streams):
            with torch.cuda.stream(stream):
                for name, (call, _, _) in table.items():
                    call(space[name])
    torch.cuda.synchronize()
    for table, w in zip(sets, want):
        for name, (_, outs, _) in table.items():
            assert same(bits(outs), w[name]), name


@pytest.mark.parametrize("M", [1, 3, 17, 70, 300])
def test_neighbours_of_the_outputs(M):
    """What lies behind an output in its allocation stays as it was."""
    def room(rows, cols, dtype):
        t = torch.full((rows + 8, cols), 7.0, device="cuda").to(dtype)
        return t, t[:rows], lambda: bool((t[rows:].float() == 7.0).all())

    x, w, d = rand(M, 144, seed=M), published(136, 144, seed=1), rand(M, 136, seed=2)
    for dtype in (torch.bfloat16, torch.float32):
        _, out, intact = room(M, 136, dtype)
        moe.fp8_matmul(x, w, out=out)
        assert intact()
        _, da, intact_a = room(M, 144, dtype)
        _, db, intact_b = room(136, 144, dtype)
        moe.fp8_matmul_backward(d, x, w, da=da, db=db)
        assert intact_a() and intact_b()
    for block in (1, 128):
        codes, c, intact_c = room(M, 144, E4M3)
        shape = (2, M) if block == 1 else (-(-M // 128), 2)
        _, s, intact_s = room(*shape, torch.float32)
        moe.fp8_quantize(x, block=block, codes=c, scales=s)
        assert intact_c() and intact_s()
        _, back, intact = room(M, 144, torch.float16)
        moe.fp8_dequantize(moe.Fp8(c, s, block), out=back)
        assert intact()
    y, (w13, w2), (ids, wt) = rand(M, 256, seed=M), experts(4, 128, 256, seed=5), routing(M, 2, 6, seed=M)
    _, out, intact = room(M, 256, torch.bfloat16)
    moe.fp8_experts_forward(y, ids, wt, w13, w2, out=out)
    assert intact()
    scores = rand(M, 24, seed=M, dtype=torch.float32)
    top = torch.topk(scores, 2, dim=1).indices.int()
    off = torch.tensor([0, M // 2, M // 2], dtype=torch.int32, device="cuda")  # tokens behind the last sequence
    _, grad, intact = room(M, 24, torch.float32)
    _, counts, tokens = moe.balance_loss(scores, top, seq_offsets=off)
    moe.balance_loss_backward(torch.ones(1, device="cuda"), scores, counts, tokens, 2, seq_offsets=off, dscores=grad)
    assert intact() and (grad[M // 2:] == 0).all()


def test_offsets_that_are_not_in_order():
    """Sequence borders that decrease or lie outside give unspecified values, but an answer, and leave the
    other results of the process alone."""
    scores = rand(3000, 64, seed=1, dtype=torch.float32)
    top = torch.topk(scores, 2, dim=1).indices.int()
    good = moe.balance_loss(scores, top)[0].clone()
    for off in ([3000, 0], [-5, 10, 4], [0, 1 << 30, 7, 2000], [-(1 << 31), (1 << 31) - 1], [2000, 100, 2500, 50, 3000]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        _, counts, tokens = moe.balance_loss(scores, top, seq_offsets=off)
        grad = moe.balance_loss_backward(torch.ones((), device="cuda"), scores, counts, tokens, 2, seq_offsets=off)
        assert grad.shape == scores.shape
    torch.cuda.synchronize()
    assert torch.equal(moe.balance_loss(scores, top)[0], good)


def test_refusals():
    x, w = rand(4, 256, seed=1), published(136, 256, seed=1)
    q = moe.fp8_quantize(x)
    wide = rand(4, 512, seed=1)
    for call, kind in (
            (lambda: moe.fp8_quantize(wide[:, :256]), ValueError),             # strided
            (lambda: moe.fp8_quantize(x, block=64), ValueError),
            (lambda: moe.fp8_quantize(x[:, :24].contiguous()), ValueError),    # width 24
            (lambda: moe.fp8_quantize(x.reshape(2, 2, 256)), ValueError),      # matrices in 1 x 128 blocks
            (lambda: moe.fp8_quantize(rand(2, 100, 256, seed=1), block=128), ValueError),
            (lambda: moe.fp8_quantize(x.double()), TypeError),
            (lambda: moe.fp8_quantize(x, scales=torch.empty(4, 2, device="cuda")), ValueError),
            (lambda: moe.Fp8(q.codes, q.scales, 128), ValueError),
            (lambda: moe.Fp8(q.codes.view(torch.uint8), q.scales, 1), TypeError),
            (lambda: moe.Fp8(q.codes, q.scales.double(), 1), TypeError),
            (lambda: moe.Fp8(q.codes, q.scales.cpu(), 1), ValueError),
            (lambda: moe.fp8_matmul(w, w), ValueError),                        # a in 128 x 128 blocks
            (lambda: moe.fp8_matmul(x.half(), w), TypeError),
            (lambda: moe.fp8_matmul(wide, w), ValueError),                     # widths differ
            (lambda: moe.fp8_matmul(x, x), TypeError),
            (lambda: moe.fp8_matmul(x, w, dtype=torch.float16), TypeError),
            (lambda: moe.fp8_matmul(x, w, out=torch.empty(4, 128, device="cuda")), ValueError),
            (lambda: moe.fp8_matmul(x, moe.fp8_quantize(rand(12, 256, seed=1))), ValueError),  # cols 12
            (lambda: moe.fp8_matmul_backward(x, x, w), ValueError),
            (lambda: moe.fp8_matmul_backward(rand(4, 136), x, moe.fp8_quantize(rand(136, 256))), ValueError),
            (lambda: moe.fp8_matmul_backward(rand(4, 136), q, w), TypeError),
            (lambda: moe.fp8_matmul(x, w, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), ValueError)):
        with pytest.raises(kind):
            call()
    w13, w2 = experts(4, 128, 256, seed=1)
    ids, wt = routing(4, 2, 4, seed=1)
    for call, kind in (
            (lambda: moe.fp8_experts_forward(x, ids.long(), wt, w13, w2), TypeError),
            (lambda: moe.fp8_experts_forward(x, ids, wt.bfloat16(), w13, w2), TypeError),
            (lambda: moe.fp8_experts_forward(x, ids[:2], wt, w13, w2), ValueError),
            (lambda: moe.fp8_experts_forward(x, ids, wt, w2, w13), ValueError),
            (lambda: moe.fp8_experts_forward(x, ids, wt, w13, w), ValueError),
            (lambda: moe.fp8_experts_forward(x, ids, wt, w13, w2, expert_base=-1), ValueError),
            (lambda: moe.fp8_experts_forward(x, ids, wt, w13, w2, expert_base=1 << 40), ValueError)):
        with pytest.raises(kind):
            call()
    s = rand(6, 8, seed=1, dtype=torch.float32)
    top = torch.topk(s, 2, dim=1).indices.int()
    one = torch.ones((), device="cuda")
    _, counts, tokens = moe.balance_loss(s, top)
    for call, kind in (
            (lambda: moe.balance_loss(s.double(), top), TypeError),
            (lambda: moe.balance_loss(s.t(), top), ValueError),
            (lambda: moe.balance_loss(s, top.long()), TypeError),
            (lambda: moe.balance_loss(s, top[:3]), ValueError),
            (lambda: moe.balance_loss(s, top, mask=torch.ones(6, dtype=torch.uint8, device="cuda")), TypeError),
            (lambda: moe.balance_loss(s, top, mask=torch.ones(5, dtype=torch.bool, device="cuda")), ValueError),
            (lambda: moe.balance_loss(s, top, seq_offsets=torch.zeros(1, dtype=torch.int32, device="cuda")), ValueError),
            (lambda: moe.balance_loss(s, top, seq_offsets=torch.zeros(9000, dtype=torch.int32, device="cuda")), ValueError),
            (lambda: moe.balance_loss(s, torch.zeros(6, 9, dtype=torch.int32, device="cuda")), ValueError),  # k > S
            (lambda: moe.balance_loss_backward(one, s, counts[:4], tokens, 2), ValueError),
            (lambda: moe.balance_loss_backward(torch.ones(2, device="cuda"), s, counts, tokens, 2), ValueError),
            (lambda: moe.balance_loss_backward(one.cpu(), s, counts, tokens, 2), ValueError),
            (lambda: moe.balance_loss_backward(one, s, counts, tokens, 0), ValueError)):
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("T", [1, 6, 130])
def test_a_run_of_them(T):
    """A router's step and the experts it picks, a padded batch: scores -> ids and weights, the balance
    loss with its counts and gradient, the experts on weights quantised from bf16, an FP8 projection
    after them and its gradients."""
    H, I, E, k = 256, 128, 8, 2
    x = rand(T, H, seed=T)
    scores = rand(T, E, seed=T + 1, dtype=torch.float32)
    ids, weights = moe.route(scores, k)
    mask = torch.arange(T, device="cuda") < max(1, T - 3)  # padding at the end
    dloss = torch.full((), 0.01, device="cuda")
    loss, counts, tokens, dscores = balance_check(scores, ids, mask, None, dloss)
    assert int(tokens) == int(mask.sum()) and int(counts.sum()) == k * int(tokens)
    assert (dscores[~mask] == 0).all()
    ids = torch.where(mask[:, None], ids, torch.full_like(ids, -1))
    w13 = moe.fp8_quantize(rand(E, 2 * I, H, seed=2, scale=H ** -0.5), block=128)
    w2 = moe.fp8_quantize(rand(E, H, I, seed=3, scale=I ** -0.5), block=128)
    y = moe.fp8_experts_forward(x, ids, weights, w13, w2)
    ref, tol = experts_reference(x, ids, weights, w13, w2, 0)
    assert ((y.double() - ref).abs() <= tol).all() and (y[~mask] == 0).all()
    sorted_ids, block_expert, n = moe.align(ids, E, 1)
    assert int(n) == int(counts.sum())
    wo = moe.fp8_quantize(rand(136, H, seed=4), block=128)
    z = moe.fp8_matmul(y, wo)
    product_close(z, o.q_values(y), o.values(wo.codes, wo.scales, 128), H)
    dz = rand(T, 136, seed=5)
    dy, dwo = moe.fp8_matmul_backward(dz, y, wo)
    product_close(dy, o.q_values(dz), o.values(wo.codes, wo.scales, 128).T, 136)
    product_close(dwo, o.q_values(dz.T), o.q_values(y.T), T)
    rl, rc, rt, rg, _ = balance_reference(scores, ids, mask, None, 0.01)
    assert torch.equal(rc[0], counts)


def test_a_shared_expert_is_one_more():
    """An expert in a slot of every token, with weight 1, beside the routed ones."""
    x, (w13, w2) = rand(9, 256, seed=1), experts(5, 128, 256, seed=1)
    ids, wt = routing(9, 2, 4, seed=2)
    ids = torch.cat([ids, torch.full((9, 1), 4, dtype=torch.int32, device="cuda")], dim=1)
    wt = torch.cat([wt, torch.ones(9, 1, device="cuda")], dim=1)
    out = moe.fp8_experts_forward(x, ids, wt, w13, w2)
    ref, tol = experts_reference(x, ids, wt, w13, w2, 0)
    assert ((out.double() - ref).abs() <= tol).all()
