"""MI355X (gfx950) W4A16 INT4 grouped MoE layer.

A thin binding over the C ABI declared in include/moe_w4a16.h: argument
marshalling only, every step of the layer runs in the library's HIP kernels.
PyTorch supplies device memory and the current stream.

    out = forward(x, topk_ids, topk_weights, packed_w13, scales_w13,
                  packed_w2, scales_w2, shared_w=None, out=None, expert_base=0)
    ids, weights = route(scores, top_k)              # router step
    out, ids, weights = forward_scores(x, scores, top_k, packed_w13, ...)
    pk = prepack(packed_w13, scales_w13, packed_w2, scales_w2)   # once
    out = forward_prepacked(x, topk_ids, topk_weights, pk, shared_w=None)

The shared expert's feed-forward block on its own, with gradients, and MXFP4
(include/moe_ffn.h):

    out = ffn_forward(x, w13, w2, gate_up=None)
    dx, dw13, dw2 = ffn_backward(dout, x, gate_up, w13, w2)
    q = mxfp4_quantize(w)                            # Mxfp4: codes, scales
    w = mxfp4_dequantize(q)
    out = mxfp4_matmul(a, q)                         # a: Mxfp4 or bf16
    out = mxfp4_ffn_forward(x, w13_q, w2_q)

No call records an autograd graph, also for tensors that require grad:
ffn_backward is how the block's gradients are had.
"""
from ._binding import (  # noqa: F401
    MOE_ERR_ALIGNMENT,
    MOE_ERR_HIP,
    MOE_ERR_NULL,
    MOE_ERR_SHAPE,
    MOE_ERR_UNSUPPORTED,
    MOE_ERR_WORKSPACE,
    MOE_OK,
    LIB_PATH,
    MoeError,
    Prepacked,
    Problem,
    align,
    align_capacity,
    align_scratch_size,
    forward,
    forward_block_m,
    forward_split_max_pairs,
    forward_noalloc,
    forward_prepacked,
    forward_scores,
    library,
    noalloc_workspace_limit,
    prepack,
    prepack_size,
    problem,
    route,
    status_string,
    workspace_size,
)
from ._ffn import (  # noqa: F401
    MOE_FFN_BACKWARD,
    MOE_FFN_FORWARD,
    MOE_FFN_FORWARD_MXFP4,
    MOE_TYPE_BF16,
    MOE_TYPE_FP16,
    MOE_TYPE_FP32,
    FfnProblem,
    Mxfp4,
    ffn_backward,
    ffn_forward,
    ffn_workspace_size,
    mxfp4_dequantize,
    mxfp4_ffn_forward,
    mxfp4_matmul,
    mxfp4_matmul_workspace_size,
    mxfp4_quantize,
)
