/*
 * libsvq, the feed-forward block around the decode-and-multiply: a product
 * with bias, activation and residual, the gated pair of an FFN, the router
 * of a mixture of experts and a whole expert layer.  Same library, same
 * packed matrices, same rules as svq.h (ownership, errors, streams,
 * workspaces: a call with workspace == NULL only reports the bytes needed
 * and validates what it is given; a workspace starts on 16 bytes; calls that share a workspace must be
 * ordered on one stream; nothing is kept from one call for the next).
 *
 * Numerics.  Up to 16 rows products are those of svq.h, except that calls of
 * 5..16 rows that round to bf16 take weights as fp16 (R*D rounded to 11 bits
 * under the matrix's power-of-two scale).  Beyond 16 rows weights
 * enter the matrix cores as fp16 (R*D rounded to 11 bits under the matrix's
 * power-of-two scale) and activations as fp16 after a power-of-two scale per
 * row (a bf16 value keeps its bits down to 2^-29 of the row's largest finite
 * magnitude; below, the error is at most 2^-38 of it); matrices whose tables
 * admit no exact split run svq.h's bf16 form.  Accumulation is fp32.  Scales are taken from finite
 * magnitudes; an infinite activation gives the infinite or NaN output that
 * the products and sums have (NaN also where its weight rounds to zero in
 * fp16).  Bias, activation, gating, residual and the sum over a token's experts are fp32;
 * each output is rounded once, to nearest even.  The inner activation of an
 * expert layer (act(gate) * up) enters the down product as fp16 (11
 * significant bits) after a power-of-two scale: for few slots
 * (m * topk up to 64 or 5/4 num_experts) one per 512 permuted channels, beyond
 * one per row, and there all three products run in the form for more than 16
 * rows.
 */
#ifndef SVQ_FFN_H
#define SVQ_FFN_H

#include "svq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* silu(v) = v / (1 + e^-v); gelu(v) = v/2 (1 + erf(v / sqrt 2));
 * gelu_tanh(v) = v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))). */
typedef enum {
  SVQ_ACT_NONE = 0,
  SVQ_ACT_RELU = 1,
  SVQ_ACT_SILU = 2,
  SVQ_ACT_GELU = 3,
  SVQ_ACT_GELU_TANH = 4
} svq_act;

/* What happens to a product before it is stored: act(p + bias) + residual.
 *   bias:     device [n] of bias_dt (4-byte or 2-byte aligned), or NULL.
 *   residual: device [m][ldr] of residual_dt, ldr >= n, or NULL.  It may be
 *             the output itself (y, with ldr == ldy and the same type); it
 *             must not overlap the output otherwise. */
typedef struct {
  const void *bias;
  svq_dtype bias_dt;
  svq_act act;
  const void *residual;
  int64_t ldr;
  svq_dtype residual_dt;
} svq_epilogue;

/* svq_linear_epilogue: y = act(x * What^T + bias) + residual for one packed
 * matrix; svq_linear with the epilogue applied to the fp32 sums.
 *   w, x, m, ldx, y, ldy, ydt, workspace, stream: as for svq_linear; y must
 *             not overlap x.
 *   ep: host, not NULL (a zeroed struct means no epilogue). */
svq_status svq_linear_epilogue(const svq_handle *w, const void *x, int64_t m, int64_t ldx,
                               const svq_epilogue *ep, void *y, int64_t ldy, svq_dtype ydt,
                               void *workspace, size_t *workspace_bytes, void *stream);

/* svq_linear_glu: the gated pair of an FFN,
 *   y = act(x * Gate^T + bias_gate) * (x * Up^T + bias_up)   (element by element)
 *   gate, up:  packed matrices of one n and k (bd may differ).
 *   x, m, ldx, y, ldy, ydt, workspace, stream: as for svq_linear.
 *   bias_gate, bias_up: device [n] of bias_dt, each may be NULL.
 * x, y, the biases and the workspace must not overlap. */
svq_status svq_linear_glu(const svq_handle *gate, const svq_handle *up, const void *x, int64_t m,
                          int64_t ldx, svq_act act, const void *bias_gate, const void *bias_up,
                          svq_dtype bias_dt, void *y, int64_t ldy, svq_dtype ydt,
                          void *workspace, size_t *workspace_bytes, void *stream);

/* svq_moe_route: the router of a mixture of experts.  For token t and expert
 * e the logit is l = sum_j x[t][j] * w[e][j], summed in double precision;
 * the score is softmax over all experts or sigmoid(l), the key is the score
 * plus select_bias[e] (the logit itself when select_bias is NULL).  A token
 * takes the topk experts of largest key, in decreasing order, equal keys by
 * increasing index; a NaN key is below every number.  Its weights are those
 * experts' scores (without select_bias), divided by their sum when
 * renormalize is 1, times scale.
 *   x:           device bf16 [m][ldx], ldx >= k.
 *   w:           device [num_experts][ldw] of wdt, ldw >= k.
 *   num_experts: 1..256; topk: 1..min(num_experts, 32); k >= 1.
 *   select_bias: device fp32 [num_experts] or NULL.
 *   ids:         device int32 [m][topk], out; weights: device fp32 [m][topk], out.
 * ids and weights feed svq_moe_ffn; ids feed svq_moe_linear. */
typedef enum { SVQ_ROUTE_SOFTMAX = 0, SVQ_ROUTE_SIGMOID = 1 } svq_route_score;
svq_status svq_moe_route(const void *x, int64_t m, int64_t ldx, const void *w, svq_dtype wdt,
                         int32_t num_experts, int32_t k, int64_t ldw, const float *select_bias,
                         svq_route_score score, int32_t renormalize, float scale, int32_t topk,
                         int32_t *ids, float *weights, void *workspace, size_t *workspace_bytes,
                         void *stream);

/* svq_moe_ffn: a whole expert layer,
 *   y[t] = residual[t] + sum_j weights[t][j] * Down_e (act(Gate_e x[t]) * (Up_e x[t])),
 *   e = expert_ids[t][j], summed over j in order, in fp32.
 *   gate, up, down: host arrays of num_experts (1..256) packed matrices; gate
 *                   and up share n (the inner width) and k (the columns of
 *                   x), down has k = that inner width; one n and k per
 *                   projection, bd may differ per matrix.
 *   expert_ids:     device int32 [m*topk]; weights: device fp32 [m*topk].  A
 *                   slot whose id is outside [0, num_experts) contributes
 *                   nothing, whatever its weight.
 *   residual:       device [m][ldr] of residual_dt, ldr >= down's n, or NULL;
 *                   it may be y itself (ldr == ldy, same type), no other
 *                   overlap with y is allowed.
 *   y:              device [m][ldy] of type ydt, ldy >= down's n.  It may be x
 *                   itself (ldx == ldy, bf16, down's n the columns of x), with
 *                   or without x as the residual; no other overlap with x.
 *   workspace, stream: as for svq_moe_linear.
 * SVQ_ERR_UNSUPPORTED: up to 64 slots, an inner width beyond 36864, or, with
 * matrices that admit no exact split, rows too long for a block's LDS (an
 * inner width beyond about 20000). */
svq_status svq_moe_ffn(const svq_handle *gate, const svq_handle *up, const svq_handle *down,
                       int32_t num_experts, const void *x, int64_t ldx, const int32_t *expert_ids,
                       const float *weights, int64_t m, int32_t topk, svq_act act,
                       const void *residual, int64_t ldr, svq_dtype residual_dt, void *y,
                       int64_t ldy, svq_dtype ydt, void *workspace, size_t *workspace_bytes,
                       void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SVQ_FFN_H */
