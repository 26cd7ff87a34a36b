// balance_api.cpp -- host side of include/moe_balance.h: argument checks and
// workspace layout. Every check runs before the first launch.
#include "../../include/moe_balance.h"
#include "balance_internal.h"
#include "internal.h"

namespace {

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

int check_problem(const moe_balance_problem* p) {
  if (!p) return MOE_ERR_NULL;
  if (p->num_tokens < 0 || p->num_experts < 1 || p->num_experts > MOE_MAX_SCORED ||
      p->top_k < 1 || p->top_k > p->num_experts || p->num_sequences < 1 ||
      p->num_sequences > MOE_MAX_SEQUENCES || p->num_tokens > 0x7fffffff / p->top_k)
    return MOE_ERR_SHAPE;
  if (p->type < MOE_TYPE_BF16 || p->type > MOE_TYPE_FP32) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

balance::Sizes sizes_of(const moe_balance_problem* p) {
  return {p->num_tokens, p->num_experts, p->top_k, p->num_sequences, p->type};
}

int done(hipError_t e) { return e == hipSuccess ? MOE_OK : moe::report_hip(e); }

}  // namespace

extern "C" {

int moe_balance_workspace_size(const moe_balance_problem* p, size_t* bytes) {
  if (!p || !bytes) return MOE_ERR_NULL;
  const int st = check_problem(p);
  if (st != MOE_OK) return st;
  *bytes = balance::Workspace(sizes_of(p)).bytes;
  return MOE_OK;
}

int moe_balance_loss(const void* scores, const int32_t* topk_ids, const uint8_t* mask,
                     const int32_t* seq_offsets, float* loss, int32_t* counts, int32_t* tokens,
                     const moe_balance_problem* p, void* workspace, size_t workspace_bytes,
                     void* stream) {
  size_t need = 0;
  const int st = moe_balance_workspace_size(p, &need);
  if (st != MOE_OK) return st;
  if (!seq_offsets && p->num_sequences != 1) return MOE_ERR_NULL;
  if (!loss || !counts || !tokens || (p->num_tokens > 0 && (!scores || !topk_ids)) ||
      (need && !workspace))
    return MOE_ERR_NULL;
  if (!aligned(scores, 16) || !aligned(topk_ids, 4) || !aligned(seq_offsets, 4) ||
      !aligned(loss, 4) || !aligned(counts, 4) || !aligned(tokens, 4) ||
      (need && !aligned(workspace, 16)))
    return MOE_ERR_ALIGNMENT;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  return done(balance::launch_forward(sizes_of(p), scores, topk_ids, mask, seq_offsets, loss,
                                      counts, tokens, workspace, (hipStream_t)stream));
}

int moe_balance_loss_backward(const float* dloss, const void* scores, const int32_t* counts,
                              const int32_t* tokens, const uint8_t* mask,
                              const int32_t* seq_offsets, void* dscores,
                              const moe_balance_problem* p, void* stream) {
  const int st = check_problem(p);
  if (st != MOE_OK) return st;
  if (!seq_offsets && p->num_sequences != 1) return MOE_ERR_NULL;
  if (p->num_tokens == 0) return MOE_OK;
  if (!dloss || !scores || !counts || !tokens || !dscores) return MOE_ERR_NULL;
  if (!aligned(scores, 16) || !aligned(dscores, 16) || !aligned(dloss, 4) ||
      !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(seq_offsets, 4))
    return MOE_ERR_ALIGNMENT;
  return done(balance::launch_backward(sizes_of(p), dloss, scores, counts, tokens, mask,
                                       seq_offsets, dscores, (hipStream_t)stream));
}

}  // extern "C"
