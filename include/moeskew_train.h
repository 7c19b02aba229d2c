/*
 * moeskew_train.h - C ABI of the operators that train the block around the expert
 * computation of moeskew.h, in the same library: the router's balance loss with the
 * per-expert counts, the gradient of the router's logits, the norms before and after the
 * block with its gate and residual scale (forward and backward), and an AdamW step over
 * many tensors.
 *
 * The conventions of moeskew.h hold: device pointers owned by the caller and 16-byte
 * aligned, every call asynchronous on `stream` with the device of its arrays current,
 * MOE_OK or a negative MOE_ERR_* with nothing enqueued, problems only the device can see
 * OR-ed into `status`, no memory allocated or kept, no host synchronisation (every call can
 * be captured into a CUDA graph).  Calls that may run at the same time need workspaces of
 * their own.  Outputs may not overlap inputs or one another unless an entry point says so.
 * The results of every call here are the same bits on every run (no floating-point atomics).
 */
#ifndef MOESKEW_TRAIN_H
#define MOESKEW_TRAIN_H

#include "moeskew.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of the arrays that come in more than one */
enum { MOET_F32 = 0, MOET_BF16 = 1, MOET_E4M3 = 2 };

/* device-detected problem next to the MOE_STATUS_* bits: seq_off falls or leaves [0, T] */
enum { MOET_STATUS_BAD_SEQ = 32 };

/* moet_workspace_size(which): bytes of the `workspace` argument */
enum {
  MOET_WS_BALANCE = 0,  /* moet_balance_loss (of n_seq sequences) */
  MOET_WS_NORM_BWD = 1  /* moet_block_norm_backward (n_seq is not looked at) */
};

/* Widest row the block norms take. */
#define MOET_MAX_NORM_D 8192

/* Returns 0 for an invalid cfg, n_seq or which. */
MOE_API size_t moet_workspace_size(const moe_cfg* cfg, int32_t n_seq, int which);

/* Balance loss, z loss and per-expert counts of the router, over packed sequences.
 * Sequence s holds the tokens [seq_off[s], seq_off[s+1]); a token counts when it lies in a
 * sequence and its mask is not 0.  With n_s counted tokens in s, n = sum n_s, S+ sequences
 * that have any, p_t the softmax of logits[t] over all E experts, and c_se the counted
 * tokens' choices of expert e in s:
 *   P_se = (1/n_s) sum_t p_te,   f_se = E c_se / (k n_s),
 *   balance loss = (1/S+) sum_s sum_e f_se P_se   (1 where routing is uniform),
 *   z loss = (1/n) sum_t (log sum_e exp logits[t, e])^2;  both 0 when n = 0.
 *   logits     fp32 [T, E] (rows of tokens that do not count are not looked at).
 *   topk_ids   int32 [T, k] from moe_route_hist.
 *   token_mask uint8 [T], or NULL: every token counts.
 *   seq_off    int32 [n_seq + 1], rising from >= 0 to <= T, or NULL with n_seq = 1: one
 *              sequence of all T tokens.  1 <= n_seq <= 2^20.
 *   losses     fp32 [2]: balance loss, z loss.
 *   counts     int32 [n_seq, E]: c_se.     probs fp32 [n_seq, E]: P_se (0 when n_s = 0).
 *   seq_info   int32 [n_seq + 2]: n_s, then n, then S+.
 *   lse        fp32 [T]: log sum exp of a counted token's logits, 0 for the others.
 * A counted token's NaN or infinite logit sets MOE_STATUS_NONFINITE, an id outside [0, E)
 * MOE_STATUS_BAD_ID, a seq_off that falls or leaves [0, T] MOET_STATUS_BAD_SEQ. */
MOE_API int moet_balance_loss(const moe_cfg* cfg, const float* logits, const int32_t* topk_ids,
                              const uint8_t* token_mask, const int32_t* seq_off,
                              int32_t n_seq, float* losses, int32_t* counts, float* probs,
                              int32_t* seq_info, float* lse, void* workspace,
                              int32_t* status, moe_stream_t stream);

/* Gradient of the router's logits: the gates' part, the losses' part, or their sum.
 * Gates' part (dy, o and tok_row given; all three NULL leaves it out), of every token:
 *   dgates[t, j] = <dy[t], O[tok_row[t, j]]>,
 *   dlogits[t, id_j] += g_j (dgates[t, j] - sum_i g_i dgates[t, i])   (softmax over the k).
 * Losses' part (dloss given, with what moet_balance_loss wrote for the same logits, ids,
 * mask and sequences; dloss = NULL leaves it out), of every token that counted:
 *   dlogits[t, e] += p_te (a_se - sum_i a_si p_ti + 2 dloss[1] lse_t / n),
 *   a_se = dloss[0] E c_se / (S+ k n_s^2)   (the counts carry no gradient).
 *   dy      fp32 [T, d]: gradient of the layer's y.   o bf16 [R_max, d]: the expert output
 *           rows (MOE_FFN_WRITE_O).   tok_row int32 [T, k] from moe_dispatch_permute.
 *   dloss   fp32 [2]: gradient of the two losses.
 *   dgates  fp32 [T, k], written with the gates' part; may be NULL.
 *   dlogits fp32 [T, E], written in full (0 where nothing reaches).
 * logits, lse, counts and seq_info are needed with dloss only, topk_ids and topk_gates with
 * the gates' part only.  The gates' part needs d % 8 == 0.  A row outside [0, R_max) sets
 * MOE_STATUS_BAD_ID and counts as zeros; so does an id outside [0, E), which is left out. */
MOE_API int moet_router_backward(const moe_cfg* cfg, const float* logits,
                                 const int32_t* topk_ids, const float* topk_gates,
                                 const float* dy, const uint16_t* o, const int32_t* tok_row,
                                 const uint8_t* token_mask, const int32_t* seq_off,
                                 int32_t n_seq, const int32_t* counts,
                                 const int32_t* seq_info, const float* lse,
                                 const float* dloss, float* dgates, float* dlogits,
                                 int32_t* status, moe_stream_t stream);

/* The block norms' constants: n(v; w) = v * rsqrt(mean(v^2) + eps) * (w + w_offset), the
 * residual stream's scale and the block output's scale, and the element types of the
 * residual stream (h, h_out, dh_out, dh) and of the norm weights (MOET_F32 or MOET_BF16). */
typedef struct moet_norm {
  float eps, w_offset, res_scale, out_scale;
  int32_t h_dtype, w_dtype;
} moet_norm;

/* Behind a block and before the next, in one pass over the rows (cfg's T and d):
 *   h_out[t] = res_scale h[t] + out_scale gate[t] n(y[t]; w_post),
 *   x[t] = bf16(n(h_out[t]; w_next)), from h_out before its rounding.
 *   h      [T, d] residual stream.      y fp32 [T, d]: the layer's output, or NULL: h_out
 *          is h and is not written (a norm before the first block).
 *   gate   fp32 [T], or NULL: 1.        w_post [d], or NULL: y is added as it is.
 *   w_next [d], or NULL: no x (behind the last block).
 *   h_out  [T, d]; may be h itself.     x bf16 [T, d].
 * At least one of y and w_next is given.  Needs d % 8 == 0 and d <= MOET_MAX_NORM_D; eps
 * > 0.  Sums in fp32. */
MOE_API int moet_block_norm(const moe_cfg* cfg, const moet_norm* norm, const void* h,
                            const float* y, const float* gate, const void* w_post,
                            const void* w_next, void* h_out, uint16_t* x,
                            moe_stream_t stream);

/* Gradients of moet_block_norm.  h_out is the stream as the forward stored it (h itself when
 * there was no y); the gradient is taken at its stored values.  With u = dh_out +
 * (gradient of x through n(.; w_next)):
 *   dh = res_scale u when there is a y, u when there is none,
 *   dy fp32 [T, d], dgate fp32 [T] (NULL when gate is), dw_post, dw_next fp32 [d] (each
 *   NULL when its weight is).
 *   dh_out [T, d] in the stream's type, or NULL: 0.   dx fp32 [T, d]: gradient of x (NULL
 *   exactly when w_next is).  At least one of the two is given.
 *   dh may be dh_out itself.   workspace: MOET_WS_NORM_BWD bytes (partial weight
 *   gradients, added in a fixed order). */
MOE_API int moet_block_norm_backward(const moe_cfg* cfg, const moet_norm* norm,
                                     const void* h_out, const float* y, const float* gate,
                                     const void* w_post, const void* w_next,
                                     const void* dh_out, const float* dx, void* dh, float* dy,
                                     float* dgate, float* dw_post, float* dw_next,
                                     void* workspace, moe_stream_t stream);

/* Elements that share one scale of an 8-bit AdamW state. */
#define MOET_ADAMW_BLOCK 256

/* One tensor of an AdamW step (arrays on the device; n = 0 is left out).
 *   p      [n] weights of p_dtype (MOET_F32, MOET_BF16), updated.
 *   master fp32 [n], updated, or NULL.  With it, bf16 weights are its rounding and are only
 *          written; fp32 weights have none.
 *   g      [n] gradient of g_dtype (MOET_F32, MOET_BF16).
 *   m, v   the moments, updated.  state_dtype MOET_F32: fp32 [n] each, v the second moment.
 *          MOET_E4M3: one byte an element; block b of MOET_ADAMW_BLOCK elements stands for
 *          m[i] * m_scale[b], and v for the second moment's root, v[i] * v_scale[b].
 *   m_scale, v_scale fp32 [ceil(n / MOET_ADAMW_BLOCK)], updated, 4-byte aligned (NULL with
 *          MOET_F32). */
typedef struct moet_adamw_tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  int64_t n;
  float weight_decay;
  int32_t p_dtype, g_dtype, state_dtype;
} moet_adamw_tensor;

typedef struct moet_adamw {
  double beta1, beta2, eps; /* 0 <= beta < 1; 2^-126 <= eps <= 2^100 */
} moet_adamw;

/* One AdamW step over `count` tensors (a HOST array, read before the call returns):
 *   t = step + 1, g = grad * grad_scale,
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
 *   p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps),
 * in fp32; the weights use m and v before those are rounded to their stored form.
 * An 8-bit block's scale is its largest |m| (or root of v) over 448; values are rounded to
 * the nearest e4m3 code, and a root above 0 never to code 0; a block whose largest is below
 * 1e-30 is stored as zeros.  An infinite or NaN gradient makes its element infinite or NaN,
 * with 8-bit states its whole block's moments; a finite one whose (1 - beta2) g^2 leaves fp32
 * makes v infinite: the weight stands still but for its decay, an 8-bit block's moments are NaN.
 *   lr         fp32 [1].
 *   grad_scale fp32 [1], or NULL: 1.  When it is infinite or NaN the step is left out:
 *              nothing is written, the step count included.
 *   step       int32 [4]: step[0] counts the steps taken and is raised by the call;
 *              step[1] must be 0 before the first call and is 0 after every call.
 * lr, grad_scale and the step count are read on the device, so a captured step replays with
 * their current values.  No array may be shared by two tensors of a call. */
MOE_API int moet_adamw_step(const moet_adamw_tensor* tensors, int32_t count,
                            const moet_adamw* opt, const float* lr, const float* grad_scale,
                            int32_t* step, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOESKEW_TRAIN_H */
