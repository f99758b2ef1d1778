/*
 * moe_experts.h - C ABI of the operators around the experts (libcrs_moe.so):
 * routing scores to expert ids and weights, with its gradient; the experts'
 * product on microscaled 4-bit (MX FP4) and on 8-bit integer operands, with the
 * quantisers that make them; and the gradients of combine and dispatch. They join
 * onto include/moe.h: moe_route writes the expert_ids and expert_scales that
 * moe_dispatch and moe_combine take, moe_expert_product reads the rows, scales and
 * counts that moe_dispatch leaves in quant_mode 4 with MOE_Y_FP4_E2M1,
 * moe_expert_product_int8 those of quant_mode 2, and a training step goes
 * moe_combine_backward, the experts' own gradient, moe_dispatch_backward and
 * moe_route_backward.
 *
 * The conventions of include/moe.h hold: array pointers are device pointers of
 * the caller, nothing is allocated or kept, `stream` is a cudaStream_t, calls
 * only enqueue work, argument errors return before anything is launched, and
 * the same inputs give the same bytes.
 */
#ifndef CRS_MOE_EXPERTS_H
#define CRS_MOE_EXPERTS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types beyond moe_dtype_t: fp32 logits and quantiser inputs, and MX
 * FP4 output rows of moe_expert_product. */
enum { MOE_F32 = 3, MOE_MXFP4 = 4 };

/* ------------------------------------------------------------------ routing */

enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2_SUM = 1 };

typedef struct {
  int32_t tokens;        /* T >= 0 */
  int32_t expert_num;    /* E in [1, 1024] */
  int32_t topk;          /* K in [1, 32], K <= topk_group * (E / group_num) */
  int32_t group_num;     /* G >= 1, E % G == 0: expert e is in group e / (E / G); 1 = no groups */
  int32_t topk_group;    /* groups that a token may choose from, [1, G] */
  int32_t group_score;   /* MOE_GROUP_*: a group's value is its largest key, or the sum of its two largest */
  int32_t score_func;    /* MOE_SCORE_* */
  int32_t renormalize;   /* 1: the weights of a token are divided by their sum; 0: not */
  int32_t logits_dtype;  /* MOE_F32, MOE_F16 or MOE_BF16 */
  float scaling;         /* finite factor on the weights */
  int64_t logits_stride; /* elements from one token's logits to the next one's, >= E */
} moe_router_config_t;

/* Chooses topk experts for every token.
 *
 *   score  s_e = softmax(logits)_e or sigmoid(logits_e), fp32. An expert whose
 *          logit is -inf or NaN is masked out: it scores 0 and is left out of
 *          the softmax. (+inf logits share the softmax among themselves.)
 *   key    s_e + bias_e with a bias (s_e alone for MOE_GROUP_TOP2_SUM without
 *          one); the logit itself otherwise, which orders as the score does.
 *          A masked expert's key, and a NaN key, count as -inf.
 *   groups with G > 1, the topk_group groups of largest value stay open; in
 *          MOE_GROUP_TOP2_SUM a second key of -inf adds nothing.
 *   picks  the K largest keys of the open groups in descending order; equal
 *          keys and equal groups go to the lower index, so masked experts are
 *          picked last, and the ids of a token are always distinct and valid.
 *   weight w_k = scaling * s_k / (renormalize ? sum_j s_j : 1), zeros where
 *          that sum is 0 (a token whose picks are all masked, or all have sigmoid
 *          scores below those of fp32's exponential: logits under -88).
 *
 *   logits        [T] rows of E elements, logits_stride apart, aligned to the element
 *   bias          NULL or [E] fp32; it moves the choice, not the weights
 *   expert_ids    [T][K] int32 (moe_dispatch's expert_ids, with T = W * bs)
 *   expert_scales [T][K] fp32  (moe_dispatch's and moe_combine's expert_scales)
 * Weights are computed in fp32 with expf and IEEE division. Scores in keys come from
 * faster functions: within 2^-21 of the formula's, and within 2^-16 of their own size
 * down to 2^-126 (smaller ones may count as 0); experts of equal logit and bias have
 * equal keys. Experts whose keys are nearer than that may be chosen either way.
 * A token's sums run in an order that depends on the batch's size and alignment (in
 * large batches two tokens share a warp): the last bits of its softmax weights, and
 * choices as near as that, may differ from those of another batch. */
moe_status_t moe_route(const moe_router_config_t* rc, const void* logits, const float* bias, int32_t* expert_ids,
                       float* expert_scales, void* stream);

/* The gradient of moe_route's weights with respect to the logits, the choice
 * held fixed (the bias gets none). With g_k = scaling * grad_scales_k and
 * r_k = s_k / sum_j s_j over the token's picks:
 *   softmax, renormalised      d_k = r_k * (g_k - sum_j g_j r_j)
 *   sigmoid, renormalised      d_k = r_k * (g_k - sum_j g_j r_j) * (1 - s_k)
 *   sigmoid, not renormalised  d_k = g_k * s_k * (1 - s_k)
 * at the chosen experts, zero elsewhere, and
 *   softmax, not renormalised  d_e = s_e * (g_e - sum_j g_j s_j), g_e = 0 where e
 *                              was not chosen, at every expert.
 * It is taken in fp32 (zeros where a renormalised token's scores sum to 0).
 * Masked experts get zero, and what grad_scales holds at masked picks (infinities
 * and NaN included) is not used. expert_ids as moe_route gave them; an id outside
 * [0, E) is passed over, ids repeated in a token give unspecified values.
 * group_num, topk_group and group_score are checked as in moe_route and not
 * used otherwise.
 *   grad_scales [T][K] fp32; grad_logits [T] rows of E elements of logits_dtype,
 *   grad_stride (>= E) apart; it must not overlap logits. */
moe_status_t moe_route_backward(const moe_router_config_t* rc, const void* logits, const int32_t* expert_ids,
                                const float* grad_scales, void* grad_logits, int64_t grad_stride, void* stream);

/* ------------------------------------------------- MX FP4 quantisation and product */

/* Where the E8M0 scale of block b (32 elements) of row r goes. */
enum {
  MOE_SF_ROWS = 0,  /* [experts][rows][B], B = ceil(cols / 32), as moe_dispatch writes dynamic_scales */
  MOE_SF_TILED = 1, /* [experts][ceil(rows / 128)][ceil(B / 4)][512]: tiles of 128 rows x 4 blocks, the
                       byte of (r, b) at (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4 of its tile (the order
                       in which the tensor cores take scales); bytes beyond the edges are 0 */
};

/* Bytes of the scale array of an [experts][rows][cols] tensor; 0 for sizes
 * that moe_mx_quantize refuses. */
uint64_t moe_mx_scale_bytes(int32_t experts, int64_t rows, int32_t cols, int32_t sf_layout);

/* Quantises `experts` matrices of `rows` x `cols` elements to OCP MX FP4 E2M1,
 * with moe_dispatch's quant_mode 4 arithmetic: blocks of 32 elements along a
 * row share X = 2^(floor(log2 amax) - 2) clamped to [2^-127, 2^127], stored as
 * the byte log2 X + 127; code = x / X to the nearest E2M1 value, ties to even,
 * saturating at 6. A block of zeros gets byte 0 and zero codes. Two codes a
 * byte, the even element in the low nibble. Infinities saturate; a NaN is
 * passed over in amax and its code is unspecified (the format has no NaN).
 *
 *   x          x_dtype MOE_F32, MOE_F16 or MOE_BF16, aligned to the element; row r
 *              of matrix e begins at e * expert_stride + r * row_stride elements
 *              (row_stride >= cols, expert_stride >= 0)
 *   cols       even, [2, 2^30]; the last block of a row may be short
 *   codes      [experts][rows][cols / 2]
 *   scales     moe_mx_scale_bytes(experts, rows, cols, sf_layout) bytes
 * experts >= 0, rows >= 0, experts * rows < 2^31. */
moe_status_t moe_mx_quantize(const void* x, int32_t x_dtype, int32_t experts, int64_t rows, int32_t cols,
                             int64_t row_stride, int64_t expert_stride, int32_t sf_layout, uint8_t* codes,
                             uint8_t* scales, void* stream);

enum {
  MOE_EPI_NONE = 0,   /* y[r][n] = z[r][n] */
  MOE_EPI_SWIGLU = 1, /* y[r][i] = silu(z[r][2i]) * z[r][2i + 1], n even: the weight rows of
                         gate and up take turns */
};

/* The experts' product on dispatched rows: for every row r of rank d that
 * ep_recv_count gives to local expert le (expert e = d * L + le),
 *   z[r][j] = sum over i of x[r][i] * w[e][j][i]
 * with x and w the MX FP4 values, on the tensor cores' block-scaled path with
 * fp32 accumulation, then the epilogue in fp32, rounded once to y_dtype. silu takes
 * the fast exponential and reciprocal: within 2^-16 of its size for gates above -87.
 *
 *   cfg           the dispatch's configuration: W, bs, topk, E, wait_timeout_us and
 *                 the workspace size are taken from it; h, types and modes are not
 *   k             elements of a row: a multiple of 32, at most 2^30 (cfg->h for rows of moe_dispatch,
 *                 the intermediate size for rows of this function's MOE_MXFP4 output)
 *   x             [W][A][k / 2] codes (A from moe_get_workspace_size), 16-byte aligned
 *   x_scales      [W][A][k / 32] E8M0 bytes, 4-byte aligned
 *   ep_recv_count [W][L*W] as moe_dispatch wrote it; of an expert's W running counts only the last, at
 *                 its rows' end, is read
 *   w             [E][n][k / 2] codes, 16-byte aligned
 *   w_scales      MOE_SF_TILED scales of w (moe_mx_quantize with experts = E, rows = n,
 *                 cols = k), 16-byte aligned
 *   y             [W][A][c], c = n, or n / 2 with MOE_EPI_SWIGLU: MOE_F16 or MOE_BF16
 *                 elements, or MOE_MXFP4 codes (c / 2 bytes a row, c even; the block's scale
 *                 and codes are taken from the fp32 results); 16-byte aligned
 *   y_scales      [W][A][ceil(c / 32)] E8M0 bytes for MOE_MXFP4, else NULL
 *   ws            the workspace that the dispatch used (it holds the status word)
 * Rows at or beyond ep_recv_count[d][L*W-1] are left untouched. An expert whose
 * count at its rows' begin or end is negative, decreasing or above A is reported
 * as MOE_ERR_BAD_ASSIST, and its rows are passed over (all rows, where the counts
 * left overlap to more 128-row tiles than counts of dispatch can have); a wait that
 * ran out as MOE_ERR_TIMEOUT. */
moe_status_t moe_expert_product(const moe_config_t* cfg, const void* x, const uint8_t* x_scales,
                                const int32_t* ep_recv_count, const void* w, const uint8_t* w_scales, int32_t n,
                                int32_t k, int32_t epilogue, int32_t y_dtype, void* y, uint8_t* y_scales, void* ws,
                                size_t ws_bytes, void* stream);

/* ---------------------------------------------------- int8 quantisation and product */

/* Quantises rows to 8-bit integers with a scale each, with moe_dispatch's
 * quant_mode 2 arithmetic: scale = amax|x| / 127 and code = clamp(rne(x / scale),
 * -127, 127), both IEEE divisions in fp32; a row of zeros gets scale 0 and zero
 * codes. An infinity gives its row an infinite scale and zero codes; a NaN is passed
 * over in amax and its code is unspecified (the format has no NaN).
 * For weights [E][n][k] that is a scale for each output channel, as
 * moe_expert_product_int8 takes them; with `counts`, the rows that the ranks
 * received, such as the SwiGLU output of one product on its way to the next.
 *
 *   x       x_dtype MOE_F32, MOE_F16 or MOE_BF16, aligned to the element; row r of
 *           matrix m begins at m * mat_stride + r * row_stride elements (row_stride >=
 *           cols, mat_stride >= 0)
 *   cols    [1, 2^30]; mats >= 0, rows >= 0, mats * rows < 2^31
 *   counts  NULL, or [mats][counts_len] int32 with mats <= 1024: of matrix m only the
 *           rows below counts[m][counts_len - 1] (taken into [0, rows]) are read and
 *           written: moe_dispatch's ep_recv_count with mats = W and counts_len = L*W
 *   codes   [mats][rows][cols] int8
 *   scales  [mats][rows] fp32 */
moe_status_t moe_int8_quantize(const void* x, int32_t x_dtype, int32_t mats, int64_t rows, int32_t cols,
                               int64_t row_stride, int64_t mat_stride, const int32_t* counts, int32_t counts_len,
                               int8_t* codes, float* scales, void* stream);

/* The experts' product on dispatched int8 rows, with a scale for each row and each
 * output channel: for every row r of rank d that ep_recv_count gives to local
 * expert le (expert e = d * L + le),
 *   z[r][j] = x_scales[r] * w_scales[e][j] * (sum over i of x[r][i] * w[e][j][i])
 * then the epilogue (MOE_EPI_*) in fp32, rounded once to y_dtype; silu as in
 * moe_expert_product. The integers' sum is exact where no partial sum is beyond 2^24
 * (any with k <= 1024). Past that, with k a multiple of 16, the tensor cores may cut what
 * 16 products bring instead of rounding it: an error of up to 2^-23 of the running sum
 * each time, k / 16 * 2^-23 in all (2^-10 for the longest rows, more than half a step of
 * MOE_F16; a sum that grows to 2^29 over k = 131040 was 1.3e-4 of it off). With any
 * other k the sum is an exact 32-bit integer, rounded once.
 *
 *   cfg           the dispatch's configuration: W, bs, topk, E, wait_timeout_us and
 *                 the workspace size are taken from it; h, types and modes are not
 *   k             elements of a row, [1, 131071]; multiples of 16 are some 7 times as fast as others
 *   x             [W][A][k] int8 (A from moe_get_workspace_size), 16-byte aligned
 *   x_scales      [W][A] fp32 as moe_dispatch (quant_mode 2) or moe_int8_quantize wrote
 *                 them, or NULL for 1 everywhere (static scales, folded into w_scales)
 *   ep_recv_count [W][L*W] as moe_dispatch wrote it; of an expert's W running counts only the last, at
 *                 its rows' end, is read
 *   w             [E][n][k] int8, 16-byte aligned; w_scales [E][n] fp32
 *   y             [W][A][c], c = n, or n / 2 with MOE_EPI_SWIGLU: MOE_F16 or MOE_BF16
 *                 elements, 16-byte aligned
 *   ws            the workspace that the dispatch used (it holds the status word)
 * Rows at or beyond ep_recv_count[d][L*W-1] are left untouched; counts that dispatch
 * cannot have written are treated as in moe_expert_product. */
moe_status_t moe_expert_product_int8(const moe_config_t* cfg, const int8_t* x, const float* x_scales,
                                     const int32_t* ep_recv_count, const int8_t* w, const float* w_scales, int32_t n,
                                     int32_t k, int32_t epilogue, int32_t y_dtype, void* y, void* ws, size_t ws_bytes,
                                     void* stream);

/* ------------------------------------------------- gradients of combine and dispatch */

/* The gradient of moe_combine, from grad_out, the gradient of x_out. With g =
 * grad_out[s][t] and w_k = expert_scales[s][t][k]:
 *   routed pick  grad_expert_out[its row] = w_k * g        grad_scales = <g, its row of expert_out>
 *   copy expert  adds w_k to the factor of grad_x[s][t]    grad_scales = <g, x[s][t]>
 *   zero expert or inactive pick                           grad_scales = 0
 *   grad_x[s][t] = (sum of its copies' w_k, k ascending) * g, zeros without a copy
 * in fp32, each rounded once to x_dtype (grad_scales stays fp32). Rows that belong
 * to no pick are left untouched, what tensors hold at picks and tokens that have no
 * part (infinities and NaN included) is not read, and the sums' order is fixed.
 *
 *   cfg         the combine's configuration: quant_mode 0, x_dtype MOE_F16 or MOE_BF16, else
 *               MOE_ERR_UNSUPPORTED; combine_mode plays no part
 *   grad_out    [W][bs][h]
 *   expert_out, x (with copy experts): as given to moe_combine; needed iff grad_scales is wanted
 *   assist_info, ep_recv_count, expert_ids, expert_scales, active_mask: as given to moe_combine
 *   grad_expert_out [W][A][h], grad_scales [W][bs][K] fp32, grad_x [W][bs][h]: any of them, but not all,
 *               may be NULL; none may overlap an input
 *   ws          a workspace of cfg, best the dispatch's, whose pick -> row map is then used (for many tokens of short rows
 *               several times as fast); otherwise each pick's row is looked for among those that ep_recv_count gives to its
 *               expert and source rank (one by one where they are not in dispatch's order), or (moe_dispatch_backward of
 *               many short rows) the map rebuilt as moe_combine does. A pick that no row names, a count above the capacity
 *               and a bad id are reported as there
 * Row arrays are 16-byte aligned. grad_scales is what moe_route_backward takes. */
moe_status_t moe_combine_backward(const moe_config_t* cfg, const void* grad_out, const void* expert_out,
                                  const int32_t* assist_info, const int32_t* ep_recv_count, const int32_t* expert_ids,
                                  const float* expert_scales, const uint8_t* active_mask, const void* x,
                                  void* grad_expert_out, float* grad_scales, void* grad_x, void* ws, size_t ws_bytes,
                                  void* stream);

/* The gradient of moe_dispatch without quantisation (with it: straight through, by a
 * configuration of quant_mode 0), from grad_expand_x, the gradient of expand_x:
 *   grad_x[s][t] = residual[s][t] + sum over its routed picks, k ascending, of the pick's row of grad_expand_x
 * in fp32, rounded once to x_dtype; a token with no row keeps its residual, or gets
 * zeros. And of expand_scales:
 *   grad_scales[s][t][k] = grad_expand_scales[the pick's row], 0 for picks that have none.
 *
 *   cfg, ws, assist_info, ep_recv_count, expert_ids, active_mask: as in moe_combine_backward
 *   grad_expand_x [W][A][h]
 *   residual      NULL or [W][bs][h]: the gradient that x has from elsewhere (moe_combine_backward's
 *                 grad_x, the way past the layer); it may be grad_x itself
 *   grad_expand_scales NULL or [W][A] fp32; NULL iff grad_scales is
 *   grad_x        [W][bs][h]; grad_scales [W][bs][K] fp32 */
moe_status_t moe_dispatch_backward(const moe_config_t* cfg, const void* grad_expand_x, const int32_t* assist_info,
                                   const int32_t* ep_recv_count, const int32_t* expert_ids, const uint8_t* active_mask,
                                   const void* residual, const float* grad_expand_scales, void* grad_x,
                                   float* grad_scales, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CRS_MOE_EXPERTS_H */
