"""Cases of the FP8 block, FP8 expert and balance-loss operators, with their plain forms.

The operators (`w4a16_int4_grouped_moe_amd`):

  fp8_quantize,           blocks of 1 x 128 or 128 x 128 values as one power-of-two fp32 scale and
  fp8_dequantize          e4m3 codes, and back
  fp8_matmul              a W^T with W in 128 x 128 blocks and a in 1 x 128 blocks, or in bf16 and
                          quantised on the way
  fp8_matmul_backward     gradients of a and W from the gradient of the product: each operand in
                          blocks of 128 along the axis that is summed over
  fp8_experts_forward     the routed experts on FP8 weights: x and h are quantised on the way
  balance_loss,           the router's balance loss with per-expert counts, and the gradient of the
  balance_loss_backward   scores; a loss for each sequence, masked tokens left out

A case names its operator in "op". The plain forms are elementary torch operations in fp32, rounded
once at the end (the long sums of the balance loss in fp64).
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": BF16, "fp16": F16, "fp32": F32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # the activations of a small decode batch
        {"name": "fp8 tokens 8", "op": "fp8_quantize", "rows": 8, "width": 7168, "block": 1, "type": "bf16"},
        # a gate/up matrix quantised from its master weights
        {"name": "fp8 weights 4096", "op": "fp8_quantize", "rows": 4096, "width": 7168, "block": 128, "type": "fp32"},
        # one decode token against the gate/up matrix: latency and the weight stream
        {"name": "fp8 product 1", "op": "fp8_matmul", "rows": 1, "cols": 4096, "width": 7168, "codes": False, "out": "bf16"},
        # both operands in codes, ragged everywhere, fp32 result
        {"name": "fp8 product ragged 777", "op": "fp8_matmul", "rows": 777, "cols": 1000, "width": 1008, "codes": True, "out": "fp32"},
        # a prefill batch against the gate/up matrix
        {"name": "fp8 product 4096", "op": "fp8_matmul", "rows": 4096, "cols": 4096, "width": 7168, "codes": False, "out": "bf16"},
        # a small ragged training batch (an odd token count is the weight gradient's sum length)
        {"name": "fp8 gradients ragged 201", "op": "fp8_matmul_backward", "rows": 201, "cols": 1360, "width": 1008, "out": "bf16"},
        # a training batch against the gate/up matrix, fp32 gradients for accumulation
        {"name": "fp8 gradients 4096", "op": "fp8_matmul_backward", "rows": 4096, "cols": 4096, "width": 7168, "out": "fp32"},
        # one decode token: eight experts' weights
        {"name": "fp8 experts decode 1", "op": "fp8_experts_forward", "tokens": 1, "hidden": 7168, "inter": 2048, "experts": 48, "global": 48, "top_k": 8},
        # one GPU's share of 384 experts: about 43 rows an expert
        {"name": "fp8 experts share 2048", "op": "fp8_experts_forward", "tokens": 2048, "hidden": 7168, "inter": 2048, "experts": 48, "global": 384, "top_k": 8},
        # a prefill batch with every expert here
        {"name": "fp8 experts 4096", "op": "fp8_experts_forward", "tokens": 4096, "hidden": 7168, "inter": 2048, "experts": 48, "global": 48, "top_k": 8},
        # the router of a small step: latency
        {"name": "balance 64", "op": "balance_loss", "tokens": 64, "experts": 384, "top_k": 8, "sequences": 0, "masked": False, "type": "fp32"},
        # a training batch of ragged sequences with padding
        {"name": "balance 32768", "op": "balance_loss", "tokens": 32768, "experts": 384, "top_k": 8, "sequences": 24, "masked": True, "type": "fp32"},
    ]


def _log(rng, lo, hi, step):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["fp8_quantize", "fp8_matmul", "fp8_matmul_backward", "fp8_experts_forward", "balance_loss"])
    rows = _log(rng, 1, 4096, 1)
    if op == "fp8_quantize":
        return {"op": op, "rows": rows, "width": _log(rng, 16, 7168, 16), "block": rng.choice([1, 128]),
                "type": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "fp8_matmul":
        return {"op": op, "rows": rows, "cols": _log(rng, 32, 4096, 8), "width": _log(rng, 32, 7168, 16),
                "codes": rng.random() < 0.5, "out": rng.choice(["bf16", "fp32"])}
    if op == "fp8_matmul_backward":
        return {"op": op, "rows": rows, "cols": _log(rng, 32, 4096, 8), "width": _log(rng, 32, 7168, 16),
                "out": rng.choice(["bf16", "fp32"])}
    if op == "fp8_experts_forward":
        experts = _log(rng, 1, 48, 1)
        whole = experts * rng.choice([1, 8])
        return {"op": op, "tokens": rows, "hidden": _log(rng, 128, 7168, 128), "inter": _log(rng, 128, 2048, 128),
                "experts": experts, "global": whole, "top_k": rng.randint(1, min(8, whole))}
    experts = _log(rng, 2, 512, 1)
    return {"op": op, "tokens": _log(rng, 1, 32768, 1), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
            "sequences": rng.choice([0, _log(rng, 1, 64, 1)]), "masked": rng.random() < 0.5,
            "type": rng.choice(["fp32", "bf16"])}


# ---------------------------------------------------------------- inputs


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32)


def _activations(gen, rows, width):
    """N(0, 1) with a few loud channels, as hidden states have them."""
    x = _normal(gen, rows, width)
    loud = torch.rand(width, generator=gen, device=DEV) < 0.01
    return torch.where(loud, 8 * x, x)


def _weights(gen, rows, width):
    return _normal(gen, rows, width) * width ** -0.5


def _published(gen, rows, width):
    """A weight matrix as checkpoints hold it: its block scales are the largest magnitude over 448,
    not powers of two."""
    w = _blocks(_weights(gen, rows, width), 128)
    scale = w.abs().amax(dim=(1, 3)).clamp(min=2.0 ** -100) / 448.0
    codes = (w / scale[:, None, :, None]).clamp(-448.0, 448.0)
    return _unblocks(codes, rows, width).to(E4M3), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    state = {"op": op}
    if op == "fp8_quantize":
        kind = TYPES[case["type"]]
        make = _activations if case["block"] == 1 else _weights
        state["x"] = make(gen, case["rows"], case["width"]).to(kind)
        state["block"] = case["block"]
        state["values"] = F32 if kind == F32 else BF16
    elif op in ("fp8_matmul", "fp8_matmul_backward"):
        m, n, k = case["rows"], case["cols"], case["width"]
        a = _activations(gen, m, k).to(BF16)
        state["a"] = _plain_quantize(a, 1) if case.get("codes") else a
        state["w"] = _published(gen, n, k)
        state["out"] = TYPES[case["out"]]
        if op == "fp8_matmul_backward":
            state["dout"] = _activations(gen, m, n).to(BF16)
    elif op == "fp8_experts_forward":
        t, h, i, e, k = (case[x] for x in ("tokens", "hidden", "inter", "experts", "top_k"))
        state["x"] = _activations(gen, t, h).to(BF16)
        scores = _normal(gen, t, case["global"])
        top, ids = torch.topk(scores, k, dim=1)
        state["ids"], state["weights"] = ids.to(torch.int32), torch.softmax(top, dim=1)
        for name, rows, width in (("w13", 2 * i, h), ("w2", h, i)):
            codes = torch.empty((e, rows, width), dtype=E4M3, device=DEV)
            scales = torch.empty((e, rows // 128, width // 128), dtype=F32, device=DEV)
            for x in range(e):
                codes[x], scales[x] = _published(gen, rows, width)
            state[name] = (codes, scales)
    else:
        t, s, k = case["tokens"], case["experts"], case["top_k"]
        # a router that prefers some experts
        scores = (1.5 * _normal(gen, t, s) + _normal(gen, 1, s)).to(TYPES[case["type"]])
        state["scores"] = scores
        state["ids"] = torch.topk(scores.to(F32), k, dim=1).indices.to(torch.int32)
        state["mask"] = torch.rand(t, generator=gen, device=DEV) >= 0.1 if case["masked"] else None
        state["offsets"] = None
        if case["sequences"]:
            # ragged, some of them empty, tokens behind the last one
            cuts = torch.rand(case["sequences"] + 1, generator=gen, device=DEV) * (t + 1)
            cuts[0] = 0
            cuts = torch.sort(cuts.floor().clamp(max=t)).values
            state["offsets"] = cuts.to(torch.int32)
        state["dloss"] = torch.rand((), generator=gen, device=DEV) + 0.5
    return state


# ---------------------------------------------------------------- the plain forms


def _blocks(x, high):
    """x padded with zeros to whole blocks of high x 128: [R, high, C, 128]."""
    rows, width = x.shape
    r, c = -(-rows // high), -(-width // 128)
    out = x.new_zeros((r * high, c * 128))
    out[:rows, :width] = x
    return out.reshape(r, high, c, 128)


def _unblocks(x, rows, width):
    r, high, c, _ = x.shape
    return x.reshape(r * high, c * 128)[:rows, :width].contiguous()


def _plain_quantize(x, high):
    """codes e4m3 [R, K]; scales fp32 [K/128, R] (high 1) or [R/128, K/128]."""
    rows, width = x.shape
    v = _blocks(x.to(F32), high)
    top = v.abs().amax(dim=(1, 3))
    mantissa, power = torch.frexp(top)  # top = mantissa 2^power, mantissa in [0.5, 1): 448 = 0.875 2^9
    power = (power - 9 + (mantissa > 0.875)).clamp(min=-126)
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), power), torch.ones_like(top))
    codes = _unblocks(v / scale[:, None, :, None], rows, width).to(E4M3)
    return codes, scale.t().contiguous() if high == 1 else scale


def _plain_values(codes, scales, high):
    rows, width = codes.shape
    s = scales.t() if high == 1 else scales
    return _unblocks(_blocks(codes.to(F32), high) * s[:, None, :, None], rows, width)


def _plain_experts(state):
    x, ids = state["x"], state["ids"].to(torch.int64)
    (c13, s13), (c2, s2) = state["w13"], state["w2"]
    experts, t, k = c13.shape[0], x.shape[0], ids.shape[1]
    xq = _plain_values(*_plain_quantize(x, 1), 1)
    flat = ids.reshape(-1).clamp(max=experts)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=experts + 1).tolist()
    y = torch.zeros((t * k, x.shape[1]), dtype=F32, device=DEV)
    at = 0
    for e in range(experts):
        pairs = order[at:at + counts[e]]
        at += counts[e]
        if counts[e] == 0:
            continue
        gu = xq[pairs // k] @ _plain_values(c13[e], s13[e], 128).t()
        g, u = gu.chunk(2, dim=1)
        h = g / (1 + torch.exp(-g)) * u
        h = _plain_values(*_plain_quantize(h, 1), 1)
        y[pairs] = h @ _plain_values(c2[e], s2[e], 128).t()
    return (y.reshape(t, k, -1) * state["weights"].unsqueeze(2)).sum(dim=1).to(BF16)


def _sequences(state, t):
    """Which sequence each token is in, one-hot [B, T] in fp64; masked tokens are in none."""
    at = torch.arange(t, device=DEV)
    if state["offsets"] is None:
        member = torch.ones((1, t), dtype=torch.bool, device=DEV)
    else:
        off = state["offsets"].to(torch.int64)
        member = (at >= off[:-1, None]) & (at < off[1:, None])
    if state["mask"] is not None:
        member = member & state["mask"]
    return member.to(F64)


def _plain_balance(state):
    scores, ids = state["scores"], state["ids"].to(torch.int64)
    (t, s), k = scores.shape, ids.shape[1]
    z = scores.to(F32)
    z = torch.exp(z - z.amax(dim=1, keepdim=True))
    p = z / z.sum(dim=1, keepdim=True)
    member = _sequences(state, t)
    picked = torch.zeros((t, s), dtype=F64, device=DEV).scatter_add_(1, ids, torch.ones_like(ids, dtype=F64))
    counts, tokens, sums = member @ picked, member.sum(dim=1), member @ p.to(F64)
    some = tokens > 0
    factor = torch.where(some, s / (k * tokens.clamp(min=1) ** 2), torch.zeros_like(tokens)) / some.sum().clamp(min=1)
    loss = (factor * (counts * sums).sum(dim=1)).sum()
    pull = (member.t() @ (factor[:, None] * counts)) * state["dloss"].to(F64)  # [T, S]
    pull = pull - (pull * p).sum(dim=1, keepdim=True)
    grad = torch.where(member.sum(dim=0)[:, None] > 0, p * pull, torch.zeros_like(pull))
    if state["offsets"] is None:
        counts = counts[0]
    return {"loss": loss.to(F32), "counts": counts.to(torch.int32), "tokens": tokens.to(torch.int32),
            "dscores": grad.to(scores.dtype)}


def _plain(state):
    op = state["op"]
    if op == "fp8_quantize":
        codes, scales = _plain_quantize(state["x"], state["block"])
        return {"values": _plain_values(codes, scales, state["block"]).to(state["values"]), "scales": scales}
    if op == "fp8_matmul":
        a = state["a"]
        a = a if isinstance(a, tuple) else _plain_quantize(a, 1)
        return {"out": (_plain_values(*a, 1) @ _plain_values(*state["w"], 128).t()).to(state["out"])}
    if op == "fp8_matmul_backward":
        a, d = state["a"], state["dout"]
        dq = _plain_values(*_plain_quantize(d, 1), 1)
        da = dq @ _plain_values(*state["w"], 128)
        dt = _plain_values(*_plain_quantize(d.t(), 1), 1)
        at = _plain_values(*_plain_quantize(a.t(), 1), 1)
        return {"da": da.to(state["out"]), "db": (dt @ at.t()).to(state["out"])}
    return {"out": _plain_experts(state)} if op == "fp8_experts_forward" else _plain_balance(state)


# ---------------------------------------------------------------- the operators


def run(state):
    if not own:
        return _plain(state)
    import w4a16_int4_grouped_moe_amd as moe

    op = state["op"]
    if op == "fp8_quantize":
        q = moe.fp8_quantize(state["x"], block=state["block"])
        return {"values": moe.fp8_dequantize(q, dtype=state["values"]), "scales": q.scales}
    if op == "fp8_matmul":
        a = state["a"]
        a = moe.Fp8(*a, block=1) if isinstance(a, tuple) else a
        return {"out": moe.fp8_matmul(a, moe.Fp8(*state["w"], block=128), dtype=state["out"])}
    if op == "fp8_matmul_backward":
        w = moe.Fp8(*state["w"], block=128)
        da, db = moe.fp8_matmul_backward(state["dout"], state["a"], w, dtype=state["out"])
        return {"da": da, "db": db}
    if op == "fp8_experts_forward":
        w13, w2 = moe.Fp8(*state["w13"], block=128), moe.Fp8(*state["w2"], block=128)
        return {"out": moe.fp8_experts_forward(state["x"], state["ids"], state["weights"], w13, w2)}
    scores, mask, offsets = state["scores"], state["mask"], state["offsets"]
    loss, counts, tokens = moe.balance_loss(scores, state["ids"], mask=mask, seq_offsets=offsets)
    grad = moe.balance_loss_backward(state["dloss"], scores, counts, tokens, state["ids"].shape[1], mask=mask,
                                     seq_offsets=offsets)
    return {"loss": loss, "counts": counts, "tokens": tokens, "dscores": grad}


# ---------------------------------------------------------------- work and exact results


def work(case):
    """Inputs once, outputs once, and the products' operations."""
    op = case["op"]
    if op == "fp8_quantize":
        n = case["rows"] * case["width"]
        return {"bytes": n * (SIZE[case["type"]] + (4 if case["type"] == "fp32" else 2)), "flops": 2 * n}
    if op == "fp8_matmul":
        m, n, k = case["rows"], case["cols"], case["width"]
        return {"bytes": m * k * (1 if case["codes"] else 2) + n * k + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    if op == "fp8_matmul_backward":
        m, n, k, size = case["rows"], case["cols"], case["width"], SIZE[case["out"]]
        return {"bytes": 2 * m * (n + k) + n * k + (m + n) * k * size, "flops": 4 * m * n * k}
    if op == "fp8_experts_forward":
        t, h, i, e, k = (case[x] for x in ("tokens", "hidden", "inter", "experts", "top_k"))
        share = k / case["global"]
        hit = e * (1 - (1 - share) ** t)  # expected, of a uniform routing
        return {"bytes": int(4 * t * h + 8 * t * k + 3 * h * i * hit), "flops": int(6 * h * i * t * e * share)}
    t, s = case["tokens"], case["experts"]
    return {"bytes": 3 * t * s * SIZE[case["type"]] + 4 * t * case["top_k"], "flops": 12 * t * s}


def _exact_values(x, high):
    """What the blocks of high x 128 of x stand for once quantised, in fp64, and their scales: the
    least power of two that brings the largest magnitude to 448 at most, each value to the nearest
    multiple of its step (an eighth of its power of two, 2^-9 at least), ties to even multiples."""
    rows, width = x.shape
    v = _blocks(x.to(F64), high)
    top = v.abs().amax(dim=(1, 3), keepdim=True)
    power = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
    power = torch.where(448.0 * torch.exp2(power) < top, power + 1, power)
    power = torch.where(448.0 * torch.exp2(power - 1) >= top, power - 1, power)
    power = torch.where(top > 0, power.clamp(min=-126.0), torch.zeros_like(power))
    unit = torch.exp2(power)
    y = (v / unit).abs()
    octave = torch.floor(torch.log2(y.clamp(min=2.0 ** -6)))
    octave = torch.where(torch.exp2(octave) > y, octave - 1, octave)
    octave = torch.where(torch.exp2(octave + 1) <= y, octave + 1, octave).clamp(min=-6.0)
    step = torch.exp2(octave - 3)
    q = torch.round(y / step) * step * torch.sign(v) * unit
    scale = unit.squeeze(3).squeeze(1)
    return _unblocks(q, rows, width), scale.t().contiguous() if high == 1 else scale


def _exact_decoded(codes, scales):
    """The values of a weight matrix, from the codes' bits."""
    c = codes.view(torch.uint8).to(torch.int32)
    e, m = (c // 8) % 16, (c % 8).to(F64)
    size = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).to(F64)))
    v = torch.where(c >= 128, -size, size)
    high, wide = torch.repeat_interleave(scales.to(F64), 128, dim=0)[:v.shape[0]], v.shape[1]
    return v * torch.repeat_interleave(high, 128, dim=1)[:, :wide]


def _exact_experts(state):
    x, ids = _exact_values(state["x"], 1)[0], state["ids"].to(torch.int64)
    out = torch.zeros(x.shape, dtype=F64, device=DEV)
    for e in range(state["w13"][0].shape[0]):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if token.numel() == 0:
            continue
        w13 = _exact_decoded(state["w13"][0][e], state["w13"][1][e])
        gate, up = torch.matmul(x[token], w13.t()).chunk(2, dim=1)
        h = _exact_values(gate * torch.sigmoid(gate) * up, 1)[0]
        y = torch.matmul(h, _exact_decoded(state["w2"][0][e], state["w2"][1][e]).t())
        out.index_add_(0, token, y * state["weights"][token, slot].to(F64)[:, None])
    return out


def _exact_balance(state):
    scores, ids = state["scores"].to(F64), state["ids"].to(torch.int64)
    (t, s), k = scores.shape, ids.shape[1]
    offsets = [0, t] if state["offsets"] is None else state["offsets"].tolist()
    keep = torch.ones(t, dtype=torch.bool, device=DEV) if state["mask"] is None else state["mask"]
    p = torch.softmax(scores, dim=1)
    groups = [torch.nonzero(keep[a:b]).squeeze(1) + a for a, b in zip(offsets[:-1], offsets[1:])]
    live = max(1, sum(g.numel() > 0 for g in groups))
    loss, grad = torch.zeros((), dtype=F64, device=DEV), torch.zeros_like(scores)
    counts = torch.zeros((len(groups), s), dtype=torch.int32, device=DEV)
    for i, g in enumerate(groups):
        n = g.numel()
        if n == 0:
            continue
        counts[i] = torch.bincount(ids[g].reshape(-1), minlength=s).to(torch.int32)
        share = counts[i].to(F64) / (k * n) * s / live
        loss = loss + (share * p[g].mean(dim=0)).sum()
        pull = share / n
        grad[g] = state["dloss"].to(F64) * p[g] * (pull - (p[g] * pull).sum(dim=1, keepdim=True))
    tokens = torch.tensor([g.numel() for g in groups], dtype=torch.int32, device=DEV)
    return {"loss": loss, "counts": counts[0] if state["offsets"] is None else counts, "tokens": tokens, "dscores": grad}


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "fp8_quantize":
        values, scales = _exact_values(state["x"], state["block"])
        return {"values": values, "scales": scales}
    if op == "fp8_experts_forward":
        return {"out": _exact_experts(state)}
    if op == "balance_loss":
        return _exact_balance(state)
    w = _exact_decoded(*state["w"])
    if op == "fp8_matmul":
        if case["codes"]:
            codes, scales = state["a"]
            a = codes.to(F64) * torch.repeat_interleave(scales.to(F64).t(), 128, dim=1)[:, :codes.shape[1]]
        else:
            a = _exact_values(state["a"], 1)[0]
        return {"out": torch.matmul(a, w.t())}
    d, a = state["dout"], state["a"]
    return {"da": torch.matmul(_exact_values(d, 1)[0], w),
            "db": torch.matmul(_exact_values(d.t(), 1)[0], _exact_values(a.t(), 1)[0].t())}
