"""Cases of the feed-forward and MXFP4 operators, with their plain forms.

The operators (`w4a16_int4_grouped_moe_amd`):

  ffn_forward        y = W2 (silu(W1 x) * (W3 x)), bf16, W13 = [W1; W3]; on request the fp32
                     pre-activations [W1 x, W3 x] that the backward pass reads
  ffn_backward       gradients of x, W13 and W2 from the gradient of y
  mxfp4_quantize,    blocks of 32 values along a row as one power-of-two scale (e8m0) and 32
  mxfp4_dequantize   e2m1 codes, and back
  mxfp4_matmul       a W^T with W in MXFP4 and a in MXFP4, or in bf16 and quantised on the way
  mxfp4_ffn_forward  the feed-forward block on MXFP4 weights: x and h are quantised on the way

A case names its operator in "op". The plain forms are elementary torch operations in fp32 (the
quantisation in fp64: its borders decide codes), rounded once at the end.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "fp16": F16, "fp32": F32}


def listed():
    return [
        # one decode token through the shared expert's widths: latency and the weight stream
        {"name": "ffn decode 1", "op": "ffn_forward", "tokens": 1, "hidden": 7168, "inter": 2048, "keep": False},
        # a small ragged training batch, forward with the pre-activations kept
        {"name": "ffn ragged 333", "op": "ffn_forward", "tokens": 333, "hidden": 1000, "inter": 680, "keep": True},
        # the prefill batch of the layer
        {"name": "ffn prefill 4096", "op": "ffn_forward", "tokens": 4096, "hidden": 7168, "inter": 2048, "keep": False},
        # the same ragged batch's gradients (an odd token count is the weight gradients' sum length)
        {"name": "ffn grad ragged 201", "op": "ffn_backward", "tokens": 201, "hidden": 1000, "inter": 680},
        # a training batch of the shared expert
        {"name": "ffn grad 4096", "op": "ffn_backward", "tokens": 4096, "hidden": 7168, "inter": 2048},
        # the activations of a small decode batch
        {"name": "mxfp4 tokens 8", "op": "mxfp4_quantize", "rows": 8, "width": 7168, "type": "bf16"},
        # a gate/up matrix quantised from its master weights
        {"name": "mxfp4 weights 4096", "op": "mxfp4_quantize", "rows": 4096, "width": 7168, "type": "fp32"},
        # a decode batch against the gate/up matrix
        {"name": "mxfp4 product 32", "op": "mxfp4_matmul", "rows": 32, "cols": 4096, "width": 7168, "codes": False, "out": "bf16"},
        # both operands in codes, ragged everywhere, fp32 result
        {"name": "mxfp4 product ragged 777", "op": "mxfp4_matmul", "rows": 777, "cols": 1000, "width": 992, "codes": True, "out": "fp32"},
        # a prefill batch against the gate/up matrix
        {"name": "mxfp4 product 4096", "op": "mxfp4_matmul", "rows": 4096, "cols": 4096, "width": 7168, "codes": False, "out": "bf16"},
        # a small decode batch through the block
        {"name": "mxfp4 ffn decode 8", "op": "mxfp4_ffn_forward", "tokens": 8, "hidden": 7168, "inter": 2048},
        # a prefill batch through the block
        {"name": "mxfp4 ffn 4096", "op": "mxfp4_ffn_forward", "tokens": 4096, "hidden": 7168, "inter": 2048},
    ]


def _log(rng, lo, hi, step):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["ffn_forward", "ffn_backward", "mxfp4_quantize", "mxfp4_matmul", "mxfp4_ffn_forward"])
    tokens = _log(rng, 1, 4096, 1)
    if op in ("ffn_forward", "ffn_backward"):
        case = {"op": op, "tokens": tokens, "hidden": _log(rng, 64, 7168, 8), "inter": _log(rng, 32, 2048, 8)}
        if op == "ffn_forward":
            case["keep"] = rng.random() < 0.5 and tokens < 2048
        return case
    if op == "mxfp4_quantize":
        return {"op": op, "rows": tokens, "width": _log(rng, 32, 7168, 32), "type": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "mxfp4_matmul":
        return {"op": op, "rows": tokens, "cols": _log(rng, 32, 4096, 8), "width": _log(rng, 32, 7168, 32),
                "codes": rng.random() < 0.5, "out": rng.choice(["bf16", "fp32"])}
    return {"op": op, "tokens": tokens, "hidden": _log(rng, 64, 7168, 32), "inter": _log(rng, 32, 2048, 32)}


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


def _mx(gen, rows, width):
    codes, scales = _plain_quantize(_weights(gen, rows, width))
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    state = {"op": op}
    if op in ("ffn_forward", "ffn_backward", "mxfp4_ffn_forward"):
        t, h, i = case["tokens"], case["hidden"], case["inter"]
        state["x"] = _activations(gen, t, h).to(BF16)
        if op == "mxfp4_ffn_forward":
            state["w13"], state["w2"] = _mx(gen, 2 * i, h), _mx(gen, h, i)
            return state
        state["w13"], state["w2"] = _weights(gen, 2 * i, h).to(BF16), _weights(gen, h, i).to(BF16)
        if op == "ffn_forward":
            state["keep"] = case["keep"]
        else:
            state["gate_up"] = state["x"].to(F32) @ state["w13"].to(F32).T
            state["dout"] = _normal(gen, t, h).to(BF16)
    elif op == "mxfp4_quantize":
        kind = TYPES[case["type"]]
        state["x"] = _activations(gen, case["rows"], case["width"]).to(kind)
        state["values"] = F32 if kind == F32 else BF16
    else:
        x = _activations(gen, case["rows"], case["width"]).to(BF16)
        state["a"] = _plain_quantize(x) if case["codes"] else x
        state["w"] = _mx(gen, case["cols"], case["width"])
        state["out"] = TYPES[case["out"]]
    return state


# ---------------------------------------------------------------- the plain forms


def _e2m1():
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        dtype=F32, device=DEV)


def _plain_quantize(x):
    """codes uint8 [R, K/2] (the even input in the low four bits), scales uint8 [R, K/32]."""
    rows, width = x.shape
    v = x.to(F64).reshape(rows, width // 32, 32)
    top = v.abs().amax(dim=2)
    power = torch.frexp(top).exponent - 1  # floor(log2(top))
    scale = torch.where(top > 0, power - 2 + 127, torch.zeros_like(power)).clamp(0, 254)
    y = v * torch.exp2((127 - scale).to(F64)).unsqueeze(2)
    m = y.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).reshape(rows, width // 2, 2)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).contiguous(), scale.to(torch.uint8)


def _plain_values(codes, scales):
    rows, half = codes.shape
    code = torch.stack([codes & 15, codes >> 4], dim=2).reshape(rows, half // 16, 32)
    power = torch.exp2(scales.to(F64) - 127).to(F32)
    return (_e2m1()[code.to(torch.int64)] * power.unsqueeze(2)).reshape(rows, 2 * half)


def _plain_swiglu(gu):
    g, u = gu.chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


def _plain_backward(dout, x, gate_up, w13, w2):
    d, x, w13, w2 = dout.to(F32), x.to(F32), w13.to(F32), w2.to(F32)
    g, u = gate_up.chunk(2, dim=1)
    s = 1 / (1 + torch.exp(-g))
    dh = d @ w2
    dgu = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], dim=1)
    return (dgu @ w13).to(BF16), (dgu.T @ x).to(BF16), (d.T @ (g * s * u)).to(BF16)


def _plain(state):
    op = state["op"]
    if op == "ffn_forward":
        gu = state["x"].to(F32) @ state["w13"].to(F32).T
        out = (_plain_swiglu(gu) @ state["w2"].to(F32).T).to(BF16)
        return {"out": out, "gate_up": gu} if state["keep"] else {"out": out}
    if op == "ffn_backward":
        dx, dw13, dw2 = _plain_backward(*(state[k] for k in ("dout", "x", "gate_up", "w13", "w2")))
        return {"dx": dx, "dw13": dw13, "dw2": dw2}
    if op == "mxfp4_quantize":
        codes, scales = _plain_quantize(state["x"])
        return {"values": _plain_values(codes, scales).to(state["values"]), "scales": scales}
    if op == "mxfp4_matmul":
        a = state["a"]
        a = a if isinstance(a, tuple) else _plain_quantize(a)
        return {"out": (_plain_values(*a) @ _plain_values(*state["w"]).T).to(state["out"])}
    gu = _plain_values(*_plain_quantize(state["x"])) @ _plain_values(*state["w13"]).T
    h = _plain_values(*_plain_quantize(_plain_swiglu(gu)))
    return {"out": (h @ _plain_values(*state["w2"]).T).to(BF16)}


# ---------------------------------------------------------------- the operators


def run(state):
    if not own:
        return _plain(state)
    import w4a16_int4_grouped_moe_amd as moe

    op = state["op"]
    if op == "ffn_forward":
        x = state["x"]
        if not state["keep"]:
            return {"out": moe.ffn_forward(x, state["w13"], state["w2"])}
        gate_up = torch.empty((x.shape[0], state["w13"].shape[0]), dtype=F32, device=x.device)
        return {"out": moe.ffn_forward(x, state["w13"], state["w2"], gate_up=gate_up), "gate_up": gate_up}
    if op == "ffn_backward":
        dx, dw13, dw2 = moe.ffn_backward(state["dout"], state["x"], state["gate_up"], state["w13"], state["w2"])
        return {"dx": dx, "dw13": dw13, "dw2": dw2}
    if op == "mxfp4_quantize":
        q = moe.mxfp4_quantize(state["x"])
        return {"values": moe.mxfp4_dequantize(q, dtype=state["values"]), "scales": q.scales}
    if op == "mxfp4_matmul":
        a = state["a"]
        a = moe.Mxfp4(*a) if isinstance(a, tuple) else a
        return {"out": moe.mxfp4_matmul(a, moe.Mxfp4(*state["w"]), dtype=state["out"])}
    return {"out": moe.mxfp4_ffn_forward(state["x"], moe.Mxfp4(*state["w13"]), moe.Mxfp4(*state["w2"]))}


# ---------------------------------------------------------------- work and exact results


def work(case):
    """Inputs once, outputs once, and the products' operations."""
    op = case["op"]
    if op == "mxfp4_quantize":
        n = case["rows"] * case["width"]
        per = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
        out = 4 if case["type"] == "fp32" else 2
        return {"bytes": n * (per + out) + n // 32, "flops": 2 * n}
    if op == "mxfp4_matmul":
        m, n, k = case["rows"], case["cols"], case["width"]
        a = m * k * 17 // 32 if case["codes"] else 2 * m * k
        return {"bytes": a + n * k * 17 // 32 + m * n * (4 if case["out"] == "fp32" else 2), "flops": 2 * m * n * k}
    t, h, i = case["tokens"], case["hidden"], case["inter"]
    if op == "mxfp4_ffn_forward":
        return {"bytes": 4 * t * h + 3 * h * i * 17 // 32, "flops": 6 * t * h * i}
    if op == "ffn_forward":
        return {"bytes": 4 * t * h + 6 * h * i + (8 * t * i if case["keep"] else 0), "flops": 6 * t * h * i}
    return {"bytes": 6 * t * h + 8 * t * i + 12 * h * i, "flops": 12 * t * h * i}


def _exact_values(x):
    """What the blocks of 32 of x stand for once quantised, in fp64, and their scales: the largest
    magnitude's power of two, two below it the scale, each value to the nearest of 0, 0.5, 1, 1.5,
    2, 3, 4, 6 (ties to the even code, larger ones to 6)."""
    v = x.to(F64).reshape(x.shape[0], -1, 32)
    top = v.abs().amax(dim=2, keepdim=True)
    power = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    power = torch.where(torch.exp2(power) > top, power - 1, power)
    power = torch.where(torch.exp2(power + 1) <= top, power + 1, power)
    power = torch.where(top > 0, power - 2, torch.full_like(power, -127.0)).clamp(-127, 127)
    unit = torch.exp2(power)
    y = (v / unit).abs()
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).to(F64)
    q = (torch.round(y / step) * step).clamp(max=6.0) * torch.sign(v) * unit
    return q.reshape(x.shape), (power.squeeze(2) + 127).to(torch.uint8)


def _exact_decoded(codes, scales):
    low, high = codes.to(torch.int32) % 16, codes.to(torch.int32) // 16
    c = torch.stack([low, high], dim=2).reshape(codes.shape[0], -1)
    e, m = (c % 8) // 2, (c % 2).to(F64)
    size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).to(F64)))
    sign = torch.where(c >= 8, -1.0, 1.0).to(F64)
    return sign * size * torch.exp2(scales.to(F64) - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "mxfp4_quantize":
        values, scales = _exact_values(state["x"])
        return {"values": values, "scales": scales}
    if op == "mxfp4_matmul":
        a = _exact_decoded(*state["a"]) if case["codes"] else _exact_values(state["a"])[0]
        return {"out": torch.matmul(a, _exact_decoded(*state["w"]).t())}
    x, i = state["x"].to(F64), case["inter"]
    if op == "mxfp4_ffn_forward":
        x = _exact_values(x)[0]
        w13, w2 = _exact_decoded(*state["w13"]), _exact_decoded(*state["w2"])
    else:
        w13, w2 = state["w13"].to(F64), state["w2"].to(F64)
    if op != "ffn_backward":
        gate, up = torch.matmul(x, w13[:i].t()), torch.matmul(x, w13[i:].t())
        h = gate * torch.sigmoid(gate) * up
        if op == "mxfp4_ffn_forward":
            return {"out": torch.matmul(_exact_values(h)[0], w2.t())}
        out = torch.matmul(h, w2.t())
        return {"out": out, "gate_up": torch.cat([gate, up], dim=1)} if case["keep"] else {"out": out}
    d, gu = state["dout"].to(F64), state["gate_up"].to(F64)
    gate, up = gu[:, :i], gu[:, i:]
    sig = torch.sigmoid(gate)
    swish = gate * sig
    dh = torch.matmul(d, w2)
    dgate = dh * up * (sig + swish * (1 - sig))
    dup = dh * swish
    return {"dx": torch.matmul(dgate, w13[:i]) + torch.matmul(dup, w13[i:]),
            "dw13": torch.cat([torch.matmul(dgate.t(), x), torch.matmul(dup.t(), x)]),
            "dw2": torch.matmul(d.t(), swish * up)}
