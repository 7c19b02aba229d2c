// C ABI of the training operators: argument validation, then the launchers.  Nothing is
// enqueued when validation fails; see include/moeskew_train.h for the contract.
#include <cfloat>
#include <cmath>
#include <initializer_list>

#include "train_common.cuh"

namespace moe {
namespace {

constexpr int kMaxSeq = 1 << 20;
// The step divides by a root plus eps with a reciprocal that is 0 from 2^126 on; a root is below
// 2^64 (1 - beta2)^-1/2.
constexpr float kMaxEps = 0x1p100f;
constexpr long long kMaxTensor = 1LL << 40;

int check_optional(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
int check_seq(const int32_t* seq_off, int32_t n_seq) {
  if (n_seq < 1 || n_seq > kMaxSeq || (!seq_off && n_seq != 1)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
bool is_weight_type(int32_t t) { return t == MOET_F32 || t == MOET_BF16; }
int check_norm(const moe_cfg* c, const moet_norm* n) {
  const int rc = check_cfg(c);
  if (rc != MOE_OK) return rc;
  if (!n || !is_weight_type(n->h_dtype) || !is_weight_type(n->w_dtype) || !(n->eps > 0.f) ||
      !std::isfinite(n->eps) || !std::isfinite(n->w_offset) || !std::isfinite(n->res_scale) ||
      !std::isfinite(n->out_scale))
    return MOE_ERR_INVALID_ARG;
  if (c->d % 8 || c->d > MOET_MAX_NORM_D) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moet_workspace_size(const moe_cfg* cfg, int32_t n_seq, int which) {
  if (check_cfg(cfg) != MOE_OK) return 0;
  if (which == MOET_WS_BALANCE)
    return n_seq < 1 || n_seq > kMaxSeq ? 0 : balance_workspace_bytes(*cfg, n_seq);
  if (which == MOET_WS_NORM_BWD)
    return cfg->d % 8 || cfg->d > MOET_MAX_NORM_D ? 0 : norm_bwd_workspace_bytes(*cfg);
  return 0;
}

int moet_balance_loss(const moe_cfg* cfg, const float* logits, const int32_t* topk_ids,
                      const uint8_t* token_mask, const int32_t* seq_off, int32_t n_seq,
                      float* losses, int32_t* counts, float* probs, int32_t* seq_info,
                      float* lse, void* workspace, int32_t* status, moe_stream_t stream) {
  int rc = check_cfg(cfg);
  if (rc == MOE_OK) rc = check_seq(seq_off, n_seq);
  if (rc == MOE_OK)
    rc = check_ptrs({logits, topk_ids, losses, counts, probs, seq_info, lse, workspace,
                       status});
  if (rc == MOE_OK) rc = check_optional({token_mask, seq_off});
  if (rc != MOE_OK) return rc;
  return cuda_result(launch_balance_loss(*cfg, logits, topk_ids, token_mask, seq_off, n_seq,
                                         losses, counts, probs, seq_info, lse, workspace,
                                         status, (cudaStream_t)stream));
}

int moet_router_backward(const moe_cfg* cfg, const float* logits, const int32_t* topk_ids,
                         const float* topk_gates, const float* dy, const uint16_t* o,
                         const int32_t* tok_row, const uint8_t* token_mask,
                         const int32_t* seq_off, int32_t n_seq, const int32_t* counts,
                         const int32_t* seq_info, const float* lse, const float* dloss,
                         float* dgates, float* dlogits, int32_t* status,
                         moe_stream_t stream) {
  int rc = check_cfg(cfg);
  if (rc != MOE_OK) return rc;
  const bool through_gates = dy || o || tok_row;
  if (!through_gates && !dloss) return MOE_ERR_INVALID_ARG;
  if (!through_gates && dgates) return MOE_ERR_INVALID_ARG;
  rc = check_ptrs({dlogits, status});
  if (rc == MOE_OK && through_gates) {
    rc = check_ptrs({dy, o, tok_row, topk_ids, topk_gates});
    if (rc == MOE_OK && cfg->d % 8) rc = MOE_ERR_UNSUPPORTED;
  }
  if (rc == MOE_OK && dloss) {
    rc = check_seq(seq_off, n_seq);
    if (rc == MOE_OK) rc = check_ptrs({dloss, logits, lse, counts, seq_info});
    if (rc == MOE_OK) rc = check_optional({token_mask, seq_off});
  }
  if (rc == MOE_OK) rc = check_optional({dgates});
  if (rc != MOE_OK) return rc;
  return cuda_result(launch_router_backward(*cfg, logits, topk_ids, topk_gates, dy, o, tok_row,
                                            token_mask, seq_off, n_seq, counts, seq_info, lse,
                                            dloss, dgates, dlogits, status,
                                            (cudaStream_t)stream));
}

int moet_block_norm(const moe_cfg* cfg, const moet_norm* norm, const void* h, const float* y,
                    const float* gate, const void* w_post, const void* w_next, void* h_out,
                    uint16_t* x, moe_stream_t stream) {
  int rc = check_norm(cfg, norm);
  if (rc != MOE_OK) return rc;
  if ((!y && !w_next) || (!y && (gate || w_post || h_out)) || (!w_next != !x))
    return MOE_ERR_INVALID_ARG;
  rc = check_ptrs({h});
  if (rc == MOE_OK && y) rc = check_ptrs({y, h_out});
  if (rc == MOE_OK) rc = check_optional({gate, w_post, w_next, x});
  if (rc != MOE_OK) return rc;
  return cuda_result(launch_block_norm(*cfg, *norm, h, y, gate, w_post, w_next, h_out, x,
                                       (cudaStream_t)stream));
}

int moet_block_norm_backward(const moe_cfg* cfg, const moet_norm* norm, const void* h_out,
                             const float* y, const float* gate, const void* w_post,
                             const void* w_next, const void* dh_out, const float* dx, void* dh,
                             float* dy, float* dgate, float* dw_post, float* dw_next,
                             void* workspace, moe_stream_t stream) {
  int rc = check_norm(cfg, norm);
  if (rc != MOE_OK) return rc;
  if ((!y && (gate || w_post || dy)) || (!w_next != !dx) || (!dh_out && !dx) ||
      (!gate != !dgate) || (!w_post != !dw_post) || (!w_next != !dw_next))
    return MOE_ERR_INVALID_ARG;
  rc = check_ptrs({h_out, dh, workspace});
  if (rc == MOE_OK && y) rc = check_ptrs({y, dy});
  if (rc == MOE_OK)
    rc = check_optional({gate, w_post, w_next, dh_out, dx, dgate, dw_post, dw_next});
  if (rc != MOE_OK) return rc;
  return cuda_result(launch_block_norm_backward(*cfg, *norm, h_out, y, gate, w_post, w_next,
                                                dh_out, dx, dh, dy, dgate, dw_post, dw_next,
                                                workspace, (cudaStream_t)stream));
}

int moet_adamw_step(const moet_adamw_tensor* tensors, int32_t count, const moet_adamw* opt,
                    const float* lr, const float* grad_scale, int32_t* step,
                    moe_stream_t stream) {
  if (count < 0 || (count > 0 && !tensors) || !opt) return MOE_ERR_INVALID_ARG;
  if (!(opt->beta1 >= 0. && opt->beta1 < 1.) || !(opt->beta2 >= 0. && opt->beta2 < 1.) ||
      !((float)opt->eps >= FLT_MIN && (float)opt->eps <= kMaxEps))
    return MOE_ERR_INVALID_ARG;
  int rc = check_ptrs({lr, step});
  if (rc == MOE_OK) rc = check_optional({grad_scale});
  for (int i = 0; rc == MOE_OK && i < count; ++i) {
    const moet_adamw_tensor& t = tensors[i];
    if (t.n < 0 || !is_weight_type(t.p_dtype) || !is_weight_type(t.g_dtype) ||
        (t.state_dtype != MOET_F32 && t.state_dtype != MOET_E4M3) ||
        (t.master && t.p_dtype != MOET_BF16) || !std::isfinite(t.weight_decay))
      return MOE_ERR_INVALID_ARG;
    if (t.n > kMaxTensor) return MOE_ERR_UNSUPPORTED;
    if (t.n == 0) continue;
    rc = check_ptrs({t.p, t.g, t.m, t.v});
    if (rc == MOE_OK && (t.state_dtype == MOET_E4M3) != (t.m_scale && t.v_scale))
      rc = MOE_ERR_INVALID_ARG;
    if (rc == MOE_OK && t.state_dtype == MOET_F32 && (t.m_scale || t.v_scale))
      rc = MOE_ERR_INVALID_ARG;
    // the scales are read one at a time
    if (rc == MOE_OK && ((reinterpret_cast<uintptr_t>(t.m_scale) |
                          reinterpret_cast<uintptr_t>(t.v_scale)) & 3u))
      rc = MOE_ERR_UNSUPPORTED;
    if (rc == MOE_OK) rc = check_optional({t.master});
  }
  if (rc != MOE_OK) return rc;
  return cuda_result(launch_adamw(tensors, count, *opt, lr, grad_scale, step,
                                  (cudaStream_t)stream));
}

}  // extern "C"
