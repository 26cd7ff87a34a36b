"""ctypes binding of include/moe_balance.h: the router's balance loss, its counts and its
gradient (argument marshalling only)."""
from __future__ import annotations

import ctypes
import functools

from . import _binding, _ffn
from ._binding import _check, _need
from ._ffn import _gpu, _in_range, _launch, _result, _scratch, _shaped, _type_of

MOE_MAX_SEQUENCES = 8192


class BalanceProblem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("num_sequences", ctypes.c_int32),
        ("type", ctypes.c_int32),
    ]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = _binding.library()
        P, PP = ctypes.c_void_p, ctypes.POINTER(BalanceProblem)
        N = ctypes.c_size_t
        lib.moe_balance_workspace_size.argtypes = [PP, ctypes.POINTER(N)]
        lib.moe_balance_loss.argtypes = [P] * 7 + [PP, P, N, P]
        lib.moe_balance_loss_backward.argtypes = [P] * 7 + [PP, P]
        for f in ("workspace_size", "loss", "loss_backward"):
            getattr(lib, "moe_balance_" + f).restype = ctypes.c_int
        _lib = lib
    return _lib


@functools.lru_cache(maxsize=4096)
def _problem(num_tokens, num_experts, top_k, num_sequences, kind):
    """The sizes as the library takes them, and the workspace bytes."""
    _in_range(num_tokens=num_tokens, num_experts=num_experts, top_k=top_k,
              num_sequences=num_sequences)
    p = BalanceProblem(num_tokens, num_experts, top_k, num_sequences, kind)
    n = ctypes.c_size_t(0)
    _check(_library().moe_balance_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return ctypes.byref(p), n.value


def balance_workspace_size(num_tokens: int, num_experts: int, top_k: int,
                           num_sequences: int = 1) -> int:
    """Bytes of workspace of balance_loss (host only)."""
    return _problem(num_tokens, num_experts, top_k, num_sequences, _ffn.MOE_TYPE_FP32)[1]


def _inputs(scores, mask, seq_offsets):
    """Checks what both calls take: (device, T, S, sequences, mask and offsets as pointers)."""
    dev = _gpu(scores, "scores")
    torch = _ffn.torch
    _type_of(scores.dtype)
    _need(scores, "scores", scores.dtype, 2, dev)
    T, S = scores.shape
    if mask is not None:
        _shaped(mask, "mask", torch.bool, (T,), dev)
    B = 1
    if seq_offsets is not None:
        _need(seq_offsets, "seq_offsets", torch.int32, 1, dev)
        B = seq_offsets.shape[0] - 1
        if B < 1:
            raise ValueError("seq_offsets must hold at least 2 values")
    return (dev, T, S, B, None if mask is None else mask.data_ptr(),
            None if seq_offsets is None else seq_offsets.data_ptr())


def balance_loss(scores, topk_ids, mask=None, seq_offsets=None, counts=None, tokens=None,
                 workspace=None):
    """The router's balance loss (moe_balance_loss): scores [T, S] (fp32, bf16 or fp16),
    topk_ids int32 [T, k], mask bool [T] (False: the token takes no part), seq_offsets int32
    [B + 1] (a loss for each sequence, averaged; tokens outside take no part) -> (loss fp32 [],
    counts int32 [S], or [B, S] with seq_offsets, tokens int32 [B]: those that took part).
    counts, tokens: optional output tensors. Autograd records nothing: balance_loss_backward
    is the gradient."""
    dev, T, S, B, m, off = _inputs(scores, mask, seq_offsets)
    torch = _ffn.torch
    _need(topk_ids, "topk_ids", torch.int32, 2, dev)
    k = topk_ids.shape[1]
    _shaped(topk_ids, "topk_ids", torch.int32, (T, k), dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    counts = _result(counts, "counts", torch.int32, (S,) if off is None else (B, S), dev)
    tokens = _result(tokens, "tokens", torch.int32, (B,), dev)
    p, need = _problem(T, S, k, B, _type_of(scores.dtype))
    ws = _scratch(workspace, need, dev)
    _launch(dev, _library().moe_balance_loss, scores.data_ptr(), topk_ids.data_ptr(), m, off,
            loss.data_ptr(), counts.data_ptr(), tokens.data_ptr(), p, ws.data_ptr(), ws.numel())
    return loss, counts, tokens


def balance_loss_backward(dloss, scores, counts, tokens, top_k: int, mask=None, seq_offsets=None,
                          dscores=None):
    """The gradient of the scores (moe_balance_loss_backward) from dloss fp32 (one value, on
    the GPU) and counts and tokens as balance_loss gave them for the same scores, mask and
    seq_offsets -> dscores of the scores' shape and type."""
    dev, T, S, B, m, off = _inputs(scores, mask, seq_offsets)
    torch = _ffn.torch
    _need(dloss, "dloss", torch.float32, None, dev)
    if dloss.numel() != 1:
        raise ValueError(f"dloss has shape {tuple(dloss.shape)}, expected one value")
    _shaped(counts, "counts", torch.int32, (S,) if off is None else (B, S), dev)
    _shaped(tokens, "tokens", torch.int32, (B,), dev)
    dscores = _result(dscores, "dscores", scores.dtype, (T, S), dev)
    p, _ = _problem(T, S, top_k, B, _type_of(scores.dtype))
    _launch(dev, _library().moe_balance_loss_backward, dloss.data_ptr(), scores.data_ptr(),
            counts.data_ptr(), tokens.data_ptr(), m, off, dscores.data_ptr(), p)
    return dscores
