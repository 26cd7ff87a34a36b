"""ctypes binding of include/moe_ffn.h: the gated feed-forward block and MXFP4
(argument marshalling only)."""
from __future__ import annotations

import ctypes
import functools

from . import _binding
from ._binding import _check, _need

MOE_TYPE_BF16 = 0
MOE_TYPE_FP16 = 1
MOE_TYPE_FP32 = 2
MOE_FFN_FORWARD = 0
MOE_FFN_BACKWARD = 1
MOE_FFN_FORWARD_MXFP4 = 2

MX_BLOCK = 32
MAX_INT32 = 0x7fffffff
MAX_INT64 = 0x7fffffffffffffff

torch = None  # loaded by an entry point's first check: sizes, constants and the build need none


class FfnProblem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int32),
        ("inter", ctypes.c_int32),
    ]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = _binding.library()
        P, PP = ctypes.c_void_p, ctypes.POINTER(FfnProblem)
        PS = ctypes.POINTER(ctypes.c_size_t)
        N, I, L = ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        lib.moe_ffn_workspace_size.argtypes = [PP, ctypes.c_int, PS]
        lib.moe_ffn_forward.argtypes = [P] * 5 + [PP, P, N, P]
        lib.moe_ffn_backward.argtypes = [P] * 8 + [PP, P, N, P]
        lib.moe_mxfp4_quantize.argtypes = [P, I, L, I, P, P, P]
        lib.moe_mxfp4_dequantize.argtypes = [P, P, L, I, I, P, P]
        lib.moe_mxfp4_matmul_workspace_size.argtypes = [L, I, I, ctypes.c_int, PS]
        lib.moe_mxfp4_matmul.argtypes = [P] * 4 + [L, I, I, I, P, P, N, P]
        lib.moe_mxfp4_ffn_forward.argtypes = [P] * 6 + [PP, P, N, P]
        for f in ("ffn_workspace_size", "ffn_forward", "ffn_backward", "mxfp4_quantize",
                  "mxfp4_dequantize", "mxfp4_matmul_workspace_size", "mxfp4_matmul",
                  "mxfp4_ffn_forward"):
            getattr(lib, "moe_" + f).restype = ctypes.c_int
        _lib = lib
    return _lib


def _launch(device, fn, *args):
    """fn on the device's current stream, with that device current."""
    index = device.index
    if torch.cuda.current_device() == index:
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(index)))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, torch._C._cuda_getCurrentRawStream(index)))


def _load_torch():
    global torch
    torch = _binding._torch()


def _gpu(t, name):
    if torch is None:
        _load_torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _shaped(t, name, dtype, shape, device):
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_contiguous() and t.device == device):
        return t
    _need(t, name, dtype, len(shape), device)  # says what is wrong
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _result(t, name, dtype, shape, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _shaped(t, name, dtype, shape, device)


def _scratch(workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    _need(workspace, "workspace", torch.uint8, 1, device)
    return workspace


def _in_range(**sizes):
    """Sizes that a C int64_t (num_tokens, rows) or int holds: others would reach it wrapped."""
    for name, n in sizes.items():
        most = MAX_INT64 if name in ("num_tokens", "rows") else MAX_INT32
        if not -most <= n <= most:
            raise ValueError(f"{name} {n} is out of range")


@functools.lru_cache(maxsize=4096)
def _problem(num_tokens, hidden, inter, kind):
    """The sizes as the library takes them, and the workspace bytes (a pure
    function of the sizes)."""
    _in_range(num_tokens=num_tokens, hidden=hidden, inter=inter, kind=kind)
    p = FfnProblem(num_tokens, hidden, inter)
    n = ctypes.c_size_t(0)
    _check(_library().moe_ffn_workspace_size(ctypes.byref(p), kind, ctypes.byref(n)))
    return ctypes.byref(p), n.value


def ffn_workspace_size(num_tokens: int, hidden: int, inter: int, kind: int) -> int:
    """Bytes of workspace of one call (kind: MOE_FFN_*; host only)."""
    return _problem(num_tokens, hidden, inter, kind)[1]


def _block(x, w13, w2):
    """The feed-forward block's shapes: (device, T, H, I)."""
    dev = _gpu(x, "x")
    if x.dim() != 2 or not isinstance(w2, torch.Tensor) or w2.dim() != 2:
        _need(x, "x", torch.bfloat16, 2, dev)
        _need(w2, "w2", torch.bfloat16, 2, dev)
    T, H = x.shape
    I = w2.shape[1]
    _shaped(x, "x", torch.bfloat16, (T, H), dev)
    _shaped(w13, "w13", torch.bfloat16, (2 * I, H), dev)
    _shaped(w2, "w2", torch.bfloat16, (H, I), dev)
    return dev, T, H, I


def ffn_forward(x, w13, w2, out=None, gate_up=None, workspace=None):
    """The gated feed-forward block (moe_ffn_forward): x bf16 [T, H], w13 bf16
    [2I, H] (gate rows, then up rows), w2 bf16 [H, I] -> out bf16 [T, H].
    gate_up: optional fp32 [T, 2I], receives the pre-activations that
    ffn_backward reads. Like every call here it takes the tensors' values alone:
    autograd records nothing, also for tensors that require grad."""
    dev, T, H, I = _block(x, w13, w2)
    out = _result(out, "out", torch.bfloat16, (T, H), dev)
    if gate_up is not None:
        _shaped(gate_up, "gate_up", torch.float32, (T, 2 * I), dev)
    p, need = _problem(T, H, I, MOE_FFN_FORWARD)
    ws = _scratch(workspace, need, dev)
    _launch(dev, _library().moe_ffn_forward, x.data_ptr(), w13.data_ptr(), w2.data_ptr(),
            out.data_ptr(), None if gate_up is None else gate_up.data_ptr(), p,
            ws.data_ptr(), ws.numel())
    return out


def ffn_backward(dout, x, gate_up, w13, w2, dx=None, dw13=None, dw2=None, workspace=None):
    """Gradients of the block (moe_ffn_backward): dout bf16 [T, H] and
    gate_up as ffn_forward wrote it -> (dx, dw13, dw2), bf16 of the shapes of
    x, w13 and w2. Given output tensors are overwritten."""
    dev, T, H, I = _block(x, w13, w2)
    _shaped(dout, "dout", torch.bfloat16, (T, H), dev)
    _shaped(gate_up, "gate_up", torch.float32, (T, 2 * I), dev)
    dx = _result(dx, "dx", torch.bfloat16, (T, H), dev)
    dw13 = _result(dw13, "dw13", torch.bfloat16, (2 * I, H), dev)
    dw2 = _result(dw2, "dw2", torch.bfloat16, (H, I), dev)
    p, need = _problem(T, H, I, MOE_FFN_BACKWARD)
    ws = _scratch(workspace, need, dev)
    _launch(dev, _library().moe_ffn_backward, dout.data_ptr(), x.data_ptr(), gate_up.data_ptr(),
            w13.data_ptr(), w2.data_ptr(), dx.data_ptr(), dw13.data_ptr(), dw2.data_ptr(),
            p, ws.data_ptr(), ws.numel())
    return dx, dw13, dw2


class Mxfp4:
    """A matrix in MXFP4: codes uint8 [rows, width/2] (two e2m1 codes a byte,
    the even input low) and scales uint8 [rows, width/32] (e8m0)."""

    __slots__ = ("_codes", "_scales", "_shape")

    def __init__(self, codes, scales):
        dev = _gpu(codes, "codes")
        if codes.dim() != 2:
            _need(codes, "codes", torch.uint8, 2, dev)
        rows, half = codes.shape
        _shaped(codes, "codes", torch.uint8, (rows, half), dev)
        if half % (MX_BLOCK // 2) or 2 * half > MAX_INT32:
            raise ValueError(f"codes hold {half} bytes a row, not whole blocks of 16 in range")
        _shaped(scales, "scales", torch.uint8, (rows, half // (MX_BLOCK // 2)), dev)
        self._codes = codes
        self._scales = scales
        self._shape = (rows, 2 * half)

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    shape = property(lambda self: self._shape)
    device = property(lambda self: self._codes.device)


def _type_of(dtype):
    if dtype is torch.bfloat16:
        return MOE_TYPE_BF16
    if dtype is torch.float16:
        return MOE_TYPE_FP16
    if dtype is torch.float32:
        return MOE_TYPE_FP32
    raise TypeError(f"dtype must be bfloat16, float16 or float32, got {dtype}")


def _dtype_of(out):
    if out is None:
        return torch.bfloat16
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a torch.Tensor")
    return out.dtype


def _is_mx(q, name, device=None):
    if torch is None:
        _load_torch()
    if not isinstance(q, Mxfp4):
        raise TypeError(f"{name} must be an Mxfp4")
    if device is not None and q.device != device:
        raise ValueError(f"{name} is on {q.device}, expected {device}")
    return q


def mxfp4_quantize(x, codes=None, scales=None) -> Mxfp4:
    """x [rows, width] (bf16, fp16 or fp32; width a multiple of 32) in MXFP4
    (moe_mxfp4_quantize). codes, scales: optional output tensors."""
    dev = _gpu(x, "x")
    kind = _type_of(x.dtype)
    _need(x, "x", x.dtype, 2, dev)
    rows, width = x.shape
    if width % MX_BLOCK or width > MAX_INT32:
        raise ValueError(f"x has width {width}, not a multiple of {MX_BLOCK} in range")
    codes = _result(codes, "codes", torch.uint8, (rows, width // 2), dev)
    scales = _result(scales, "scales", torch.uint8, (rows, width // MX_BLOCK), dev)
    _launch(dev, _library().moe_mxfp4_quantize, x.data_ptr(), kind, rows, width,
            codes.data_ptr(), scales.data_ptr())
    q = object.__new__(Mxfp4)  # checked above
    q._codes, q._scales, q._shape = codes, scales, (rows, width)
    return q


def mxfp4_dequantize(q: Mxfp4, dtype=None, out=None):
    """The values of q as dtype (default bfloat16; moe_mxfp4_dequantize)."""
    _is_mx(q, "q")
    if dtype is None:
        dtype = _dtype_of(out)
    kind = _type_of(dtype)
    out = _result(out, "out", dtype, q.shape, q.device)
    _launch(q.device, _library().moe_mxfp4_dequantize, q.codes.data_ptr(), q.scales.data_ptr(),
            *q.shape, kind, out.data_ptr())
    return out


@functools.lru_cache(maxsize=4096)
def mxfp4_matmul_workspace_size(rows: int, cols: int, width: int, quantize: bool) -> int:
    """Bytes of workspace of mxfp4_matmul (quantize: a is a bf16 tensor)."""
    _in_range(rows=rows, cols=cols, width=width)
    n = ctypes.c_size_t(0)
    _check(_library().moe_mxfp4_matmul_workspace_size(rows, cols, width, int(quantize),
                                                      ctypes.byref(n)))
    return n.value


def mxfp4_matmul(a, b: Mxfp4, out=None, dtype=None, workspace=None):
    """a [M, K] times the transpose of b [N, K] (moe_mxfp4_matmul) -> [M, N]
    in dtype (bfloat16, the default, or float32). a: an Mxfp4, or a bf16
    tensor that is quantised as by mxfp4_quantize."""
    if isinstance(a, Mxfp4):
        dev, (M, K), codes, scales = a.device, a.shape, a.codes, a.scales.data_ptr()
    else:
        dev = _gpu(a, "a")
        _need(a, "a", torch.bfloat16, 2, dev)
        (M, K), codes, scales = a.shape, a, None
    _is_mx(b, "b", dev)
    N, Kb = b.shape
    if K != Kb:
        raise ValueError(f"a has width {K}, b {Kb}")
    if dtype is None:
        dtype = _dtype_of(out)
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    out = _result(out, "out", dtype, (M, N), dev)
    ws = _scratch(workspace, mxfp4_matmul_workspace_size(M, N, K, scales is None), dev)
    _launch(dev, _library().moe_mxfp4_matmul, codes.data_ptr(), scales, b.codes.data_ptr(),
            b.scales.data_ptr(), M, N, K, _type_of(dtype), out.data_ptr(), ws.data_ptr(),
            ws.numel())
    return out


def mxfp4_ffn_forward(x, w13: Mxfp4, w2: Mxfp4, out=None, workspace=None):
    """The gated feed-forward block on MXFP4 weights (moe_mxfp4_ffn_forward):
    x bf16 [T, H], w13 of [2I, H], w2 of [H, I] -> out bf16 [T, H]."""
    dev = _gpu(x, "x")
    _need(x, "x", torch.bfloat16, 2, dev)
    T, H = x.shape
    _is_mx(w13, "w13", dev)
    _is_mx(w2, "w2", dev)
    I = w2.shape[1]
    if w13.shape != (2 * I, H) or w2.shape != (H, I):
        raise ValueError(f"w13 is {w13.shape} and w2 {w2.shape}, expected (2I, {H}) and ({H}, I)")
    out = _result(out, "out", torch.bfloat16, (T, H), dev)
    p, need = _problem(T, H, I, MOE_FFN_FORWARD_MXFP4)
    ws = _scratch(workspace, need, dev)
    _launch(dev, _library().moe_mxfp4_ffn_forward, x.data_ptr(), w13.codes.data_ptr(),
            w13.scales.data_ptr(), w2.codes.data_ptr(), w2.scales.data_ptr(), out.data_ptr(),
            p, ws.data_ptr(), ws.numel())
    return out
