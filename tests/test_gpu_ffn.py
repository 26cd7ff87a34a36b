"""The feed-forward block and its gradients against fp64.

Tolerances. A bf16 rounding is off by at most 2^-8 of the value, a fp32 sum of n products by at most
n 2^-24 of the sum of their magnitudes; a result's bound is its own rounding plus, through the product
that follows, those of the bf16 values it is made of (h, and the gradients of g and u). Function
values (exp, the division) are taken to 2^-20 of the larger of their factors' products."""
import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe

pytestmark = pytest.mark.gpu

BF, U, FN = 2.0 ** -8, 2.0 ** -24, 2.0 ** -20
SHAPES = [(1, 8, 8), (1, 64, 32), (2, 72, 40), (5, 136, 264), (17, 64, 2048), (64, 256, 128),
          (127, 128, 128), (129, 520, 72), (200, 1000, 680), (256, 640, 384), (300, 64, 64),
          (33, 7168, 256), (31, 696, 256), (48, 1000, 680), (64, 2048, 512)]


def inputs(T, H, I, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731
    return (bf(n(T, H) * scale), bf(n(2 * I, H) * H ** -0.5), bf(n(H, I) * I ** -0.5), bf(n(T, H)))


def guarded(shape, dtype):
    """A tensor inside a larger one, and a check that nothing around it was written."""
    n = int(torch.tensor(shape).prod())
    pad = 4096
    whole = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device="cuda")
    view = whole[pad:pad + n].view(shape)

    def intact():
        return bool((whole[:pad] == 7).all()) and bool((whole[pad + n:] == 7).all())

    return view, intact


def reference_forward(x, w13, w2):
    x, w13, w2 = x.double(), w13.double(), w2.double()
    I = w2.shape[1]
    gu = x @ w13.T
    gu_tol = (x.shape[1] + 1) * U * (x.abs() @ w13.abs().T)
    g, u = gu[:, :I], gu[:, I:]
    s = torch.sigmoid(g)
    h = g * s * u
    # |silu'| <= 1.1, |silu(g)| <= |g|
    h_tol = BF * h.abs() + 1.1 * gu_tol[:, :I] * u.abs() + gu_tol[:, I:] * g.abs() + FN * (g * u).abs()
    y = h @ w2.T
    y_tol = BF * y.abs() + 1.01 * (h_tol @ w2.abs().T) + (I + 1) * U * (h.abs() @ w2.abs().T) + 1e-30
    return gu, gu_tol + 1e-30, y, y_tol


def reference_backward(d, x, gu, w13, w2):
    d, x, gu, w13, w2 = (t.double() for t in (d, x, gu, w13, w2))
    (T, H), I = x.shape, w2.shape[1]
    g, u = gu[:, :I], gu[:, I:]
    s = torch.sigmoid(g)
    dh = d @ w2
    dh_tol = (H + 1) * U * (d.abs() @ w2.abs())
    slope = s * (1 + g * (1 - s))
    dgu = torch.cat([dh * u * slope, dh * g * s], dim=1)
    tol = torch.cat([(1.1 * dh_tol + FN * dh.abs() * (1 + g.abs())) * u.abs(),
                     (dh_tol + FN * dh.abs()) * g.abs()], dim=1) + BF * dgu.abs()
    h, h_tol = g * s * u, (BF + FN) * (g * u * s).abs() + FN * (g * u).abs()

    def product(a, a_tol, b, n):
        out = a @ b
        return out, BF * out.abs() + 1.01 * (a_tol @ b.abs()) + (n + 1) * U * (a.abs() @ b.abs()) + 1e-30

    dx = product(dgu, tol, w13, 2 * I)
    dw13 = product(dgu.T, tol.T, x, T)
    out = d.T @ h
    dw2 = (out, BF * out.abs() + 1.01 * (d.abs().T @ h_tol) + (T + 1) * U * (d.abs().T @ h.abs()) + 1e-30)
    return dx, dw13, dw2


def close(got, ref, tol):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, worst
    if err.numel() and ref.norm() > 0:  # two roundings of 2^-8 at most, in the 2-norm
        assert (err.norm() / ref.norm()).item() <= 2 * BF


@pytest.mark.parametrize("T,H,I", SHAPES)
@pytest.mark.parametrize("keep", [False, True])
def test_forward(T, H, I, keep):
    x, w13, w2, _ = inputs(T, H, I)
    gu, gu_tol, y, y_tol = reference_forward(x, w13, w2)
    out, out_ok = guarded((T, H), torch.bfloat16)
    kept, kept_ok = guarded((T, 2 * I), torch.float32)
    assert moe.ffn_forward(x, w13, w2, out=out, gate_up=kept if keep else None) is out
    close(out, y, y_tol)
    assert out_ok() and kept_ok()
    if keep:
        err = (kept.double() - gu).abs()
        assert (err <= gu_tol).all(), (err / gu_tol).max()


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_backward(T, H, I):
    x, w13, w2, d = inputs(T, H, I, seed=1)
    gu = x.float() @ w13.float().T
    want = reference_backward(d, x, gu, w13, w2)
    outs = [guarded(s, torch.bfloat16) for s in ((T, H), (2 * I, H), (H, I))]
    got = moe.ffn_backward(d, x, gu, w13, w2, *(o for o, _ in outs))
    for value, (ref, tol), (_, intact) in zip(got, want, outs):
        close(value, ref, tol)
        assert intact()


# between them every tile of every product, with shares of its sums and without
CUTS = [(66, 72, 72), (66, 232, 712), (2740, 72, 328), (4146, 232, 72), (66, 2120, 1224),
        (3370, 4808, 72), (4146, 72, 936), (99, 3656, 1224), (2740, 72, 712), (4146, 1640, 168),
        (151, 6312, 552), (2228, 3656, 72), (2740, 328, 1640)]


@pytest.mark.parametrize("T,H,I", CUTS)
def test_every_cut(T, H, I):
    x, w13, w2, d = inputs(T, H, I, seed=16)
    ref_gu, gu_tol, y, y_tol = reference_forward(x, w13, w2)
    out, out_ok = guarded((T, H), torch.bfloat16)
    gu, gu_ok = guarded((T, 2 * I), torch.float32)
    ws, ws_ok = guarded((moe.ffn_workspace_size(T, H, I, moe.MOE_FFN_FORWARD),), torch.uint8)
    close(moe.ffn_forward(x, w13, w2, out=out, gate_up=gu, workspace=ws), y, y_tol)
    assert ((gu.double() - ref_gu).abs() <= gu_tol).all()
    assert out_ok() and gu_ok() and ws_ok()
    ws, ws_ok = guarded((moe.ffn_workspace_size(T, H, I, moe.MOE_FFN_BACKWARD),), torch.uint8)
    outs = [guarded(s, torch.bfloat16) for s in ((T, H), (2 * I, H), (H, I))]
    got = moe.ffn_backward(d, x, gu, w13, w2, *(o for o, _ in outs), workspace=ws)
    for value, (ref, tol), (_, ok) in zip(got, reference_backward(d, x, gu, w13, w2), outs):
        close(value, ref, tol)
        assert ok()
    assert ws_ok()


@pytest.mark.parametrize("T,H,I", [(20, 696, 256), (201, 1000, 680), (1500, 1024, 256),
                                   (4000, 200, 64), (1000, 1000, 680), (300, 4096, 512)])
def test_backward_products_in_one_launch(T, H, I):
    """Sizes at which dx, dw13 and dw2 share a launch, with and without shares of their sums, in a
    workspace of just the size asked for."""
    x, w13, w2, d = inputs(T, H, I, seed=12)
    gu = x.float() @ w13.float().T
    want = reference_backward(d, x, gu, w13, w2)
    need = moe.ffn_workspace_size(T, H, I, 1)
    ws, ws_ok = guarded((need,), torch.uint8)
    outs = [guarded(s, torch.bfloat16) for s in ((T, H), (2 * I, H), (H, I))]
    got = moe.ffn_backward(d, x, gu, w13, w2, *(o for o, _ in outs), workspace=ws)
    for value, (ref, tol), (_, intact) in zip(got, want, outs):
        close(value, ref, tol)
        assert intact()
    assert ws_ok()
    first = [v.clone() for v in got]
    again = moe.ffn_backward(d, x, gu, w13, w2)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("T,H,I", [(20, 696, 256), (201, 1000, 680), (300, 64, 64)])
@pytest.mark.parametrize("part", ["dx", "weights"])
def test_parts_of_the_gradients(T, H, I, part):
    """dx alone, or dw13 and dw2 alone: those are right and nothing else is written."""
    from w4a16_int4_grouped_moe_amd import _ffn

    x, w13, w2, d = inputs(T, H, I, seed=13)
    gu = x.float() @ w13.float().T
    want = reference_backward(d, x, gu, w13, w2)
    outs = [guarded(s, torch.bfloat16) for s in ((T, H), (2 * I, H), (H, I))]
    asked = [part == "dx", part != "dx", part != "dx"]
    p, need = _ffn._problem(T, H, I, moe.MOE_FFN_BACKWARD)
    ws, ws_ok = guarded((need,), torch.uint8)
    _ffn._launch(x.device, _ffn._library().moe_ffn_backward, d.data_ptr(), x.data_ptr(),
                 gu.data_ptr(), w13.data_ptr(), w2.data_ptr(),
                 *(o.data_ptr() if a else None for (o, _), a in zip(outs, asked)), p,
                 ws.data_ptr(), need)
    for (value, intact), (ref, tol), a in zip(outs, want, asked):
        if a:
            close(value, ref, tol)
        else:
            assert (value == 7).all()
        assert intact()
    assert ws_ok()


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with a workspace of its own."""
    T, H, I = 201, 1000, 680
    sets = [inputs(T, H, I, seed=s) for s in (14, 15)]

    def step(x, w13, w2, d):
        gu = torch.empty(T, 2 * I, device="cuda")
        return (moe.ffn_forward(x, w13, w2, gate_up=gu), *moe.ffn_backward(d, x, gu, w13, w2))

    alone = [step(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for stream, s in zip(streams, sets):
            with torch.cuda.stream(stream):
                got.append(step(*s))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(v, w) for v, w in zip(a, b))


def test_gradients_against_differences():
    """sum(out * dout) changes along a direction as the gradients say (central differences of the
    fp64 block; the gradients' own error is their bound summed over the direction)."""
    T, H, I = 6, 48, 32
    x, w13, w2, d = inputs(T, H, I, seed=2)
    gu = torch.empty(T, 2 * I, device="cuda")
    moe.ffn_forward(x, w13, w2, gate_up=gu)
    got = moe.ffn_backward(d, x, gu, w13, w2)
    tols = [t for _, t in reference_backward(d, x, gu, w13, w2)]

    def loss(a, b, c):
        p = a @ b.T
        g, u = p[:, :I], p[:, I:]
        return ((g * torch.sigmoid(g) * u) @ c.T * d.double()).sum().item()

    base = [t.double() for t in (x, w13, w2)]
    for i in range(3):
        v = torch.randn(base[i].shape, generator=torch.Generator(device="cuda").manual_seed(i),
                        device="cuda").double()
        step = 1e-5
        moved = [[b + sign * step * v if j == i else b for j, b in enumerate(base)]
                 for sign in (1, -1)]
        slope = (loss(*moved[0]) - loss(*moved[1])) / (2 * step)
        assert abs(slope - (got[i].double() * v).sum().item()) <= \
            (tols[i] * v.abs()).sum().item() + 1e-6 * abs(slope)


def test_no_tokens():
    _, w13, w2, _ = inputs(1, 64, 32)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gu = torch.empty(0, 64, device="cuda")
    assert moe.ffn_forward(x, w13, w2, gate_up=gu).shape == (0, 64)
    dw13, dw2 = torch.ones_like(w13), torch.ones_like(w2)
    dx, _, _ = moe.ffn_backward(x, x, gu, w13, w2, dw13=dw13, dw2=dw2)
    assert dx.shape == (0, 64)
    assert not dw13.any() and not dw2.any()


@pytest.mark.parametrize("T", [3, 40, 150])
def test_a_row_keeps_its_own_infinities(T):
    """A token that holds NaN or infinity changes no other token's output."""
    x, w13, w2, _ = inputs(T, 264, 136, seed=3)
    clean = moe.ffn_forward(x, w13, w2)
    x2 = x.clone()
    x2[1, 5], x2[2, 7] = float("nan"), float("inf")
    out = moe.ffn_forward(x2, w13, w2)
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(out[keep], clean[keep])
    assert torch.isnan(out[1]).all() and not torch.isfinite(out[2]).all()


@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_saturated_and_small_gates(scale):
    x, w13, w2, d = inputs(70, 128, 96, seed=4, scale=scale)
    gu = torch.empty(70, 192, device="cuda")
    out = moe.ffn_forward(x, w13, w2, gate_up=gu)
    _, _, y, tol = reference_forward(x, w13, w2)
    close(out, y, tol)
    for value, (ref, t) in zip(moe.ffn_backward(d, x, gu, w13, w2),
                               reference_backward(d, x, gu, w13, w2)):
        close(value, ref, t)


def test_same_bits_again_and_on_another_stream():
    x, w13, w2, d = inputs(150, 512, 264, seed=5)
    gu = torch.empty(150, 528, device="cuda")

    def once():
        return (moe.ffn_forward(x, w13, w2, gate_up=gu), *moe.ffn_backward(d, x, gu, w13, w2))

    first = once()
    for a, b in zip(first, once()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = once()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 48, 200])
def test_captured_step_replays(T):
    """A step captured into a graph, replayed on new inputs between eager work."""
    H, I = 256, 136
    x, w13, w2, d = inputs(T, H, I, seed=6)
    gu = torch.empty(T, 2 * I, device="cuda")
    outs = [torch.empty_like(t) for t in (x, x, w13, w2)]
    ws = torch.empty(max(moe.ffn_workspace_size(T, H, I, k) for k in (0, 1)), dtype=torch.uint8,
                     device="cuda")

    def step():
        moe.ffn_forward(x, w13, w2, out=outs[0], gate_up=gu, workspace=ws)
        moe.ffn_backward(d, x, gu, w13, w2, *outs[1:], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (7, 8, 9):
        nx, _, _, nd = inputs(T, H, I, seed=seed)
        x.copy_(nx)
        d.copy_(nd)
        for o in outs:
            o.zero_()
        graph.replay()
        got = [o.clone() for o in outs]
        torch.cuda.synchronize()
        step()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)


def test_many_rows_past_2_gib():
    """gate_up of 2.1 GiB and an x of 1.1 GiB: the last rows are right."""
    T, H, I = 2 ** 21 + 3, 264, 136
    x, w13, w2, d = inputs(256, H, I, seed=10)
    big = x.repeat((T + 255) // 256, 1)[:T].contiguous()
    gu = torch.empty(T, 2 * I, device="cuda")
    out = moe.ffn_forward(big, w13, w2, gate_up=gu)
    ref_gu, gu_tol, y, tol = reference_forward(big[-300:], w13, w2)
    close(out[-300:], y, tol)
    assert ((gu[-300:].double() - ref_gu).abs() <= gu_tol).all()
    dx, _, _ = moe.ffn_backward(big, big, gu, w13, w2)
    (ref, t), _, _ = reference_backward(big[-300:], big[-300:], gu[-300:], w13, w2)
    close(dx[-300:], ref, t)


@pytest.mark.parametrize("T,H,I", [(260, 16640, 64), (4100, 136, 2112), (8200, 520, 1032)])
def test_a_nearly_empty_last_round_of_tiles(T, H, I):
    """Products of a little more than a whole number of rounds of tiles run as two launches."""
    x, w13, w2, d = inputs(T, H, I, seed=11)
    gu = torch.empty(T, 2 * I, device="cuda")
    out = moe.ffn_forward(x, w13, w2, gate_up=gu)
    ref_gu, gu_tol, y, tol = reference_forward(x, w13, w2)
    close(out, y, tol)
    assert ((gu.double() - ref_gu).abs() <= gu_tol).all()
    got = moe.ffn_backward(d, x, gu, w13, w2)
    for value, (ref, t) in zip(got, reference_backward(d, x, gu, w13, w2)):
        close(value, ref, t)


def test_refusals():
    x, w13, w2, d = inputs(4, 64, 32)
    gu = torch.empty(4, 64, device="cuda")
    with pytest.raises(TypeError):
        moe.ffn_forward(x.float(), w13, w2)
    with pytest.raises(ValueError):
        moe.ffn_forward(x, w13[:62], w2)
    with pytest.raises(ValueError):
        moe.ffn_forward(x.T.contiguous().T, w13, w2)
    with pytest.raises(ValueError):
        moe.ffn_forward(x, w13, w2, out=torch.empty_like(x)[:3])
    with pytest.raises(ValueError):
        moe.ffn_forward(x, w13, w2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        moe.ffn_forward(x, w13, w2, gate_up=gu.bfloat16())
    with pytest.raises(ValueError):
        moe.ffn_backward(d, x, gu[:, :32].contiguous(), w13, w2)
    with pytest.raises(ValueError):
        moe.ffn_backward(d[:3], x, gu, w13, w2)
    odd = torch.zeros(4, 60, dtype=torch.bfloat16, device="cuda")  # 60 % 8
    with pytest.raises(ValueError):
        moe.ffn_forward(odd, torch.zeros(64, 60, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(60, 32, dtype=torch.bfloat16, device="cuda"))
    flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):  # 2-byte aligned
        moe.ffn_forward(flat[1:].view(4, 64), w13, w2)
