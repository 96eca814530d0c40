/*
 * so2model.h -- model operators of libso2conv that run beside the SO(2) edge
 * convolution (so2conv.h): element embedding, routing to experts, mixing of
 * the experts' convolution weights, and dropout.
 *
 * They share the library's rules: the caller owns every buffer and the
 * stream; the library allocates nothing; all work is enqueued on `stream`
 * asynchronously and can be captured into a CUDA graph; outputs are
 * overwritten, never accumulated; argument problems are returned at once and
 * problems only the device can see go to the status word at the head of the
 * workspace (so2conv_check), for the operators that take one.  A workspace
 * belongs to one stream, or to one captured graph, at a time.  Sums, softmax
 * statistics and gradients are f32 or wider; a bf16 output is rounded once.
 * Results do not depend on scheduling: repeated calls give the same bits.
 *
 * None of the operators depends on edge vectors, so force training (the
 * double backward of the convolution) needs only their first derivatives:
 * the gradients handed to them may come from so2conv_backward or
 * so2conv_double_backward alike.  Dropout is linear with a mask that does not
 * depend on its input: its backward, of any order, is the same call.
 */
#ifndef SO2MODEL_H
#define SO2MODEL_H

#include "so2conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --------------------------------------------------------------------------
 * Element embedding
 *
 *   out[i, 0, :] = scale * table[ids[i], :],  out[i, 1.., :] = 0
 *
 * ids int64 [n]; table [n_rows, channels] of table_dtype; out [n, n_comp,
 * channels] of out_dtype, node i at out + i * ld_out elements (ld_out >=
 * n_comp * channels, so it can be a slice of wider rows; what lies between
 * the rows is left as it was).  n_comp = (lmax+1)^2 makes the convolution's
 * input features; n_comp = 1 is a plain lookup.
 *
 * An id equal to pad_id gives a zero row and takes no gradient (INT64_MIN:
 * no such id).  Any other id outside [0, n_rows) does the same and records
 * SO2_ERR_INDEX.
 *
 * Backward: grad_table [n_rows, channels] f32 = scale * the sum of grad_out's
 * component-0 rows of each id (rows no id names get 0).  grad_out has
 * out_dtype, node i at grad_out + i * ld_grad (ld_grad >= channels); only its
 * first `channels` elements are read.  The tokens are sorted by id and each
 * id's rows are added in an order that depends on the sizes and the ids alone.
 *
 * Limits: 1 <= n_rows < 2^31 - 1, 1 <= channels <= 65,536, 1 <= n_comp <=
 * 1,024, 0 <= n <= 2^30, n * n_comp * channels <= 2^38; elements aligned.
 * grad_table must not overlap the inputs.
 * -------------------------------------------------------------------------- */
typedef struct {
  int64_t n_rows;
  int32_t channels, n_comp;
  float scale;
  int32_t table_dtype, out_dtype; /* so2_dtype */
  int64_t pad_id;
} so2conv_embed_desc;

/* Bytes of workspace of the call (which: SO2_WS_FORWARD or SO2_WS_BACKWARD;
 * 0 on an unsupported descriptor); 256-byte aligned, uninitialised. */
size_t so2conv_embed_workspace_size(const so2conv_embed_desc *desc, int64_t n, int which);

so2_status so2conv_embed_forward(const so2conv_embed_desc *desc, int64_t n, const int64_t *ids,
                                 const void *table, void *out, int64_t ld_out, void *ws,
                                 size_t ws_bytes, so2_stream_t stream);

so2_status so2conv_embed_backward(const so2conv_embed_desc *desc, int64_t n, const int64_t *ids,
                                  const void *grad_out, int64_t ld_grad, float *grad_table,
                                  void *ws, size_t ws_bytes, so2_stream_t stream);

/* --------------------------------------------------------------------------
 * Routing to experts
 *
 *   s = softmax(logits) or sigmoid(logits)            per row, f32
 *   c = s + bias                                      selects, nothing else
 *   groups: a group's rank is the sum of its group_top largest c; the best
 *           top_groups groups stay
 *   chosen: the top_k largest c of those groups
 *   weights[t, j] = scale * s[chosen_j]               (/ sum of the chosen s
 *                                                      with renormalise)
 *
 * logits [n_tokens, n_experts] of dtype; bias f32 [n_experts] or NULL;
 * weights f32 and index int32 [n_tokens, top_k], in order of falling c;
 * counts int32 [n_experts] or NULL: how often each expert was chosen.  Ties
 * go to the lowest index.  Without a bias experts are ranked by their logits;
 * with one, and between groups of group_top = 2, by c in 64 bits, so that the
 * choice does not depend on an f32 rounding.
 * With top_k = n_experts nothing is selected: slot j is expert j.
 *
 * A logit of -inf, or a c of -inf, takes the expert out; slots that are left
 * over hold index -1 and weight 0, and a row without any expert holds nothing
 * else.  A logit of the type's lowest value is an ordinary, very small one.
 * NaN ranks below every number; weights follow the formula, where softmax with
 * renormalise is the softmax of the chosen logits (so it does not see logits
 * that were not chosen, and chosen scores that vanish in f32 keep their
 * ratios).  Chosen sigmoid scores that are all 0 in f32 renormalise to 0.
 *
 * Backward of <grad_weights, weights> for the choice made: grad_logits f32
 * [n_tokens, n_experts].  An index outside [0, n_experts) is an unused slot:
 * its grad_weights is not used.  The bias takes no gradient.
 *
 * Limits: 1 <= top_k <= n_experts <= 1,024; n_groups divides n_experts;
 * 1 <= group_top <= 2 (<= experts in a group); top_k <= top_groups experts in
 * the groups that stay; 0 <= n_tokens <= 2^30; scale finite and not 0.
 * -------------------------------------------------------------------------- */
enum { SO2_SCORE_SOFTMAX = 0, SO2_SCORE_SIGMOID = 1 };

typedef struct {
  int32_t n_experts, top_k, n_groups, top_groups, group_top;
  int32_t score;       /* SO2_SCORE_* */
  int32_t renormalise; /* 0 or 1 */
  float scale;
  int32_t dtype; /* so2_dtype of the logits */
} so2conv_route_desc;

so2_status so2conv_route_forward(const so2conv_route_desc *desc, int64_t n_tokens,
                                 const void *logits, const float *bias, float *weights,
                                 int32_t *index, int32_t *counts, so2_stream_t stream);

so2_status so2conv_route_backward(const so2conv_route_desc *desc, int64_t n_tokens,
                                  const void *logits, const int32_t *index,
                                  const float *grad_weights, float *grad_logits,
                                  so2_stream_t stream);

/* --------------------------------------------------------------------------
 * Mixing of experts' weights
 *
 *   out[t, :] = sum_j weights[t, j] * experts[index[t, j], :]
 *
 * experts [n_experts, n_weights] of expert_dtype, each row one convolution's
 * packed weights (n_weights = so2conv_num_weights) or any other parameters;
 * weights f32 and index int32 [n_systems, top_k] as so2conv_route_forward
 * writes them; out [n_systems, n_weights] of out_dtype, ready to be a
 * convolution's `w`.  index NULL: every expert in order (top_k = n_experts).
 * An index of -1 is an unused slot: its weight is not used.  The same expert
 * may be named twice.  Another index outside [0, n_experts) is skipped and
 * recorded as SO2_ERR_INDEX.
 *
 * Sums are f32 (fused multiply-adds, or tensor-core products of three bf16
 * parts of each operand, which keep 2^-24 of magnitudes down to 2^-109); NaN
 * and infinities in an expert or in grad_out reach what the formula says.
 *
 * Backward: with grad_out f32 [n_systems, n_weights] (a convolution's grad_w
 * per system),
 *   grad_experts[e, :] = sum over (t, j) naming e of weights[t, j] grad_out[t, :]
 *   grad_weights[t, j] = <grad_out[t, :], experts[index[t, j], :]>, 0 in
 *                        unused slots
 * both f32; NULL skips one.  An expert that no slot names gets 0.
 *
 * Limits: 1 <= top_k <= n_experts <= 4,096, 1 <= n_weights <= 2^32, 0 <=
 * n_systems <= 65,535, n_systems * top_k <= 2^22; elements aligned.
 * -------------------------------------------------------------------------- */
typedef struct {
  int32_t n_experts, top_k;
  int64_t n_weights;
  int32_t expert_dtype, out_dtype; /* so2_dtype */
} so2conv_mix_desc;

size_t so2conv_mix_workspace_size(const so2conv_mix_desc *desc, int64_t n_systems, int which);

so2_status so2conv_mix_experts_forward(const so2conv_mix_desc *desc, int64_t n_systems,
                                       const void *experts, const float *weights,
                                       const int32_t *index, void *out, void *ws,
                                       size_t ws_bytes, so2_stream_t stream);

so2_status so2conv_mix_experts_backward(const so2conv_mix_desc *desc, int64_t n_systems,
                                        const void *experts, const float *weights,
                                        const int32_t *index, const float *grad_out,
                                        float *grad_experts, float *grad_weights, void *ws,
                                        size_t ws_bytes, so2_stream_t stream);

/* --------------------------------------------------------------------------
 * Dropout
 *
 *   out = keep ? x / (1 - p) : 0,  + residual if given
 *
 * x, residual and out [n, n_comp, channels] of dtype, contiguous; out may be
 * x or residual itself.  The mask is never stored: keep is drawn from the
 * counter-based generator Philox-4x32-10 (Salmon, Moraes, Dror and Shaw,
 * "Parallel random numbers: as easy as 1, 2, 3", 2011) with rng[0] as its key
 * and (m / 4, rng[1]) as its 128-bit counter; word m % 4 keeps the unit m if
 * it is >= p 2^32.  rng is two 64-bit numbers in device memory, read when the
 * kernel runs, so a captured graph draws anew when they change between
 * replays.  Give each call of a step its own rng[1].
 *
 * unit: SO2_DROP_ELEMENT, m = flat index of the element;
 *       SO2_DROP_CHANNEL, m = i * channels + c, one draw for all components of
 *       a channel, which keeps the features equivariant;
 *       SO2_DROP_ROW, m = rows[i] (its 64 bits taken as unsigned; NULL: i), one
 *       draw for a node, or for all nodes of a system when rows names systems.
 * A dropped x is not used, so NaN there does not spread.  p = 1 drops all.
 *
 * Limits: 0 <= p <= 1, 1 <= channels <= 65,536, 1 <= n_comp <= 1,024, 0 <= n
 * <= 2^30, n * n_comp * channels <= 2^38, elements aligned.
 * -------------------------------------------------------------------------- */
enum { SO2_DROP_ELEMENT = 0, SO2_DROP_CHANNEL = 1, SO2_DROP_ROW = 2 };

typedef struct {
  int32_t channels, n_comp;
  int32_t unit; /* SO2_DROP_* */
  float p;
  int32_t dtype; /* so2_dtype */
} so2conv_dropout_desc;

so2_status so2conv_dropout(const so2conv_dropout_desc *desc, int64_t n, const void *x,
                           const void *residual, const int64_t *rows, const uint64_t *rng,
                           void *out, so2_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SO2MODEL_H */
