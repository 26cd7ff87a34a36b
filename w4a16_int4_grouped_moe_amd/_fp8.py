"""ctypes binding of include/moe_fp8.h: FP8 blocks, their products and the routed experts on
them (argument marshalling only)."""
from __future__ import annotations

import ctypes
import functools

from . import _binding, _ffn
from ._binding import _check, _need
from ._ffn import MAX_INT32, _dtype_of, _gpu, _in_range, _launch, _result, _scratch, _shaped, _type_of

MOE_FP8_ROW_BLOCKS = 1
MOE_FP8_SQUARE_BLOCKS = 128

FP8_BLOCK = 128


class Fp8ExpertsProblem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int32),
        ("inter", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("expert_base", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
    ]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = _binding.library()
        P, PP = ctypes.c_void_p, ctypes.POINTER(Fp8ExpertsProblem)
        PS = ctypes.POINTER(ctypes.c_size_t)
        N, I, L = ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        lib.moe_fp8_quantize.argtypes = [P, I, L, I, I, P, P, P]
        lib.moe_fp8_dequantize.argtypes = [P, P, L, I, I, I, P, P]
        lib.moe_fp8_matmul_workspace_size.argtypes = [L, I, I, ctypes.c_int, PS]
        lib.moe_fp8_matmul.argtypes = [P] * 4 + [I, L, I, I, I, P, P, N, P]
        lib.moe_fp8_matmul_backward_workspace_size.argtypes = [L, I, I, PS]
        lib.moe_fp8_matmul_backward.argtypes = [P] * 4 + [L, I, I, I, P, P, P, N, P]
        lib.moe_fp8_experts_workspace_size.argtypes = [PP, PS]
        lib.moe_fp8_experts_forward.argtypes = [P] * 8 + [PP, P, N, P]
        for f in ("quantize", "dequantize", "matmul_workspace_size", "matmul",
                  "matmul_backward_workspace_size", "matmul_backward", "experts_workspace_size",
                  "experts_forward"):
            getattr(lib, "moe_fp8_" + f).restype = ctypes.c_int
        _lib = lib
    return _lib


def _scales_shape(shape, block):
    """The scales' shape of a matrix [rows, width], or of matrices [n, rows, width]."""
    *n, rows, width = shape
    across = -(-width // FP8_BLOCK)
    return (across, rows) if block == 1 else (*n, -(-rows // FP8_BLOCK), across)


def _check_shape(shape, block, name):
    if block not in (MOE_FP8_ROW_BLOCKS, MOE_FP8_SQUARE_BLOCKS):
        raise ValueError(f"block must be 1 or 128, got {block}")
    if len(shape) not in ((2, 3) if block == 128 else (2,)):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [rows, width]"
                         + (" or [n, rows, width]" if block == 128 else " for blocks of 1 x 128"))
    if shape[-1] % 16 or shape[-1] > MAX_INT32:
        raise ValueError(f"{name} has width {shape[-1]}, not a multiple of 16 in range")
    if len(shape) == 3 and shape[1] % FP8_BLOCK:
        raise ValueError(f"{name} has matrices of {shape[1]} rows, not a multiple of {FP8_BLOCK}")


class Fp8:
    """A matrix in FP8: codes float8_e4m3fn [rows, width] and scales fp32, one for each block
    of 1 x 128 values (block=1: [ceil(width/128), rows]) or 128 x 128 (block=128:
    [ceil(rows/128), ceil(width/128)]); with block=128 also matrices [n, rows, width] with
    scales [n, rows/128, ceil(width/128)], rows a multiple of 128."""

    __slots__ = ("_codes", "_scales", "_block")

    def __init__(self, codes, scales, block):
        dev = _gpu(codes, "codes")
        torch = _ffn.torch
        shape = tuple(codes.shape)
        _need(codes, "codes", torch.float8_e4m3fn, None, dev)
        _check_shape(shape, block, "codes")
        _shaped(scales, "scales", torch.float32, _scales_shape(shape, block), dev)
        self._codes = codes
        self._scales = scales
        self._block = block

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    block = property(lambda self: self._block)
    shape = property(lambda self: tuple(self._codes.shape))
    device = property(lambda self: self._codes.device)


def _is_fp8(q, name, block=None, dims=None, device=None):
    if not isinstance(q, Fp8):
        raise TypeError(f"{name} must be an Fp8")
    if device is not None and q.device != device:
        raise ValueError(f"{name} is on {q.device}, expected {device}")
    if block is not None and q.block != block:
        raise ValueError(f"{name} has block={q.block}, expected {block}")
    if dims is not None and len(q.shape) != dims:
        raise ValueError(f"{name} has shape {q.shape}, expected {dims} dims")
    return q


def _rows(shape):
    n = 1
    for d in shape[:-1]:
        n *= d
    return n


def fp8_quantize(x, block=1, codes=None, scales=None) -> Fp8:
    """x [rows, width] (bf16, fp16 or fp32; width a multiple of 16) in FP8 with power-of-two
    scales (moe_fp8_quantize): block=1 for 1 x 128 blocks along a row, 128 for 128 x 128
    blocks, then also of matrices [n, rows, width]. codes, scales: optional output tensors."""
    dev = _gpu(x, "x")
    torch = _ffn.torch
    kind = _type_of(x.dtype)
    _need(x, "x", x.dtype, None, dev)
    shape = tuple(x.shape)
    _check_shape(shape, block, "x")
    codes = _result(codes, "codes", torch.float8_e4m3fn, shape, dev)
    scales = _result(scales, "scales", torch.float32, _scales_shape(shape, block), dev)
    _launch(dev, _library().moe_fp8_quantize, x.data_ptr(), kind, _rows(shape), shape[-1], block,
            codes.data_ptr(), scales.data_ptr())
    q = object.__new__(Fp8)  # checked above
    q._codes, q._scales, q._block = codes, scales, block
    return q


def fp8_dequantize(q: Fp8, dtype=None, out=None):
    """The values of q as dtype (default bfloat16; moe_fp8_dequantize)."""
    _is_fp8(q, "q")
    if dtype is None:
        dtype = _dtype_of(out)
    kind = _type_of(dtype)
    out = _result(out, "out", dtype, q.shape, q.device)
    _launch(q.device, _library().moe_fp8_dequantize, q.codes.data_ptr(), q.scales.data_ptr(),
            _rows(q.shape), q.shape[-1], q.block, kind, out.data_ptr())
    return out


@functools.lru_cache(maxsize=4096)
def fp8_matmul_workspace_size(rows: int, cols: int, width: int, quantize: bool) -> int:
    """Bytes of workspace of fp8_matmul (quantize: a is a bf16 tensor)."""
    _in_range(rows=rows, cols=cols, width=width)
    n = ctypes.c_size_t(0)
    _check(_library().moe_fp8_matmul_workspace_size(rows, cols, width, int(quantize),
                                                    ctypes.byref(n)))
    return n.value


def _out_type(dtype, default_of=None):
    torch = _ffn.torch
    if dtype is None:
        dtype = _dtype_of(default_of)
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    return dtype


def fp8_matmul(a, b: Fp8, out=None, dtype=None, workspace=None):
    """a [M, K] times the transpose of b [N, K] (moe_fp8_matmul) -> [M, N] in dtype (bfloat16,
    the default, or float32). a: an Fp8 with block=1, or a bf16 tensor that is quantised as by
    fp8_quantize, with the same result; b: an Fp8 of either block. float32 results are summed in
    fp32 throughout, bfloat16 ones of more than a few rows in the FP8 matrix units, which cut
    small products off (moe_fp8.h). Autograd records nothing."""
    if isinstance(a, Fp8):
        _is_fp8(a, "a", 1, 2)
        dev, (M, K), codes, scales = a.device, a.shape, a.codes, a.scales.data_ptr()
    else:
        dev = _gpu(a, "a")
        _need(a, "a", _ffn.torch.bfloat16, 2, dev)
        (M, K), codes, scales = a.shape, a, None
    _is_fp8(b, "b", None, 2, dev)
    N, Kb = b.shape
    if K != Kb:
        raise ValueError(f"a has width {K}, b {Kb}")
    dtype = _out_type(dtype, out)
    out = _result(out, "out", dtype, (M, N), dev)
    ws = _scratch(workspace, fp8_matmul_workspace_size(M, N, K, scales is None), dev)
    _launch(dev, _library().moe_fp8_matmul, codes.data_ptr(), scales, b.codes.data_ptr(),
            b.scales.data_ptr(), b.block, M, N, K, _type_of(dtype), out.data_ptr(), ws.data_ptr(),
            ws.numel())
    return out


@functools.lru_cache(maxsize=4096)
def fp8_matmul_backward_workspace_size(rows: int, cols: int, width: int) -> int:
    """Bytes of workspace of fp8_matmul_backward."""
    _in_range(rows=rows, cols=cols, width=width)
    n = ctypes.c_size_t(0)
    _check(_library().moe_fp8_matmul_backward_workspace_size(rows, cols, width, ctypes.byref(n)))
    return n.value


def fp8_matmul_backward(dout, a, b: Fp8, da=None, db=None, dtype=None, workspace=None):
    """Gradients of fp8_matmul(a, b) for a and b's matrix (moe_fp8_matmul_backward): dout bf16
    [M, N], a bf16 [M, K], b an Fp8 with block=128 of [N, K] -> (da [M, K], db [N, K]) in dtype
    (bfloat16, the default, or float32, which also sums in fp32 throughout). Both operands of
    each product are quantised in blocks of 128 along the axis that it sums over. Given output
    tensors are overwritten."""
    dev = _gpu(a, "a")
    torch = _ffn.torch
    _need(a, "a", torch.bfloat16, 2, dev)
    M, K = a.shape
    _is_fp8(b, "b", 128, 2, dev)
    N = b.shape[0]
    if b.shape != (N, K):
        raise ValueError(f"a has width {K}, b {b.shape[1]}")
    _shaped(dout, "dout", torch.bfloat16, (M, N), dev)
    dtype = _out_type(dtype, da if da is not None else db)
    da = _result(da, "da", dtype, (M, K), dev)
    db = _result(db, "db", dtype, (N, K), dev)
    ws = _scratch(workspace, fp8_matmul_backward_workspace_size(M, N, K), dev)
    _launch(dev, _library().moe_fp8_matmul_backward, dout.data_ptr(), a.data_ptr(),
            b.codes.data_ptr(), b.scales.data_ptr(), M, N, K, _type_of(dtype), da.data_ptr(),
            db.data_ptr(), ws.data_ptr(), ws.numel())
    return da, db


@functools.lru_cache(maxsize=4096)
def _experts(num_tokens, hidden, inter, num_experts, expert_base, top_k):
    """The sizes as the library takes them, and the workspace bytes."""
    _in_range(num_tokens=num_tokens, hidden=hidden, inter=inter, num_experts=num_experts,
              expert_base=expert_base, top_k=top_k)
    p = Fp8ExpertsProblem(num_tokens, hidden, inter, num_experts, expert_base, top_k)
    n = ctypes.c_size_t(0)
    _check(_library().moe_fp8_experts_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return ctypes.byref(p), n.value


def fp8_experts_workspace_size(num_tokens: int, hidden: int, inter: int, num_experts: int,
                               top_k: int) -> int:
    """Bytes of workspace of fp8_experts_forward (host only)."""
    return _experts(num_tokens, hidden, inter, num_experts, 0, top_k)[1]


def fp8_experts_forward(x, topk_ids, topk_weights, w13: Fp8, w2: Fp8, out=None,
                        expert_base: int = 0, workspace=None):
    """The routed experts on FP8 weights (moe_fp8_experts_forward): x bf16 [T, H]; topk_ids
    int32 [T, k]; topk_weights fp32 [T, k]; w13 of [E, 2I, H] and w2 of [E, H, I], block=128
    (hidden and inter multiples of 128) -> out bf16 [T, H]. Ids outside [expert_base,
    expert_base + E) contribute nothing. A shared expert is one more expert, with weight 1 in a
    slot of every token."""
    dev = _gpu(x, "x")
    torch = _ffn.torch
    _need(x, "x", torch.bfloat16, 2, dev)
    T, H = x.shape
    _is_fp8(w13, "w13", 128, 3, dev)
    _is_fp8(w2, "w2", 128, 3, dev)
    E, I = w13.shape[0], w2.shape[2]
    if w13.shape != (E, 2 * I, H) or w2.shape != (E, H, I):
        raise ValueError(f"w13 is {w13.shape} and w2 {w2.shape}, "
                         f"expected (E, 2I, {H}) and (E, {H}, I)")
    _need(topk_ids, "topk_ids", torch.int32, 2, dev)
    k = topk_ids.shape[1]
    _shaped(topk_ids, "topk_ids", torch.int32, (T, k), dev)
    _shaped(topk_weights, "topk_weights", torch.float32, (T, k), dev)
    out = _result(out, "out", torch.bfloat16, (T, H), dev)
    p, need = _experts(T, H, I, E, expert_base, k)
    ws = _scratch(workspace, need, dev)
    _launch(dev, _library().moe_fp8_experts_forward, x.data_ptr(), topk_ids.data_ptr(),
            topk_weights.data_ptr(), w13.codes.data_ptr(), w13.scales.data_ptr(),
            w2.codes.data_ptr(), w2.scales.data_ptr(), out.data_ptr(), p, ws.data_ptr(),
            ws.numel())
    return out
