/*
 * mxrouting.h -- C ABI of the path around the routed experts: routing, the plan of
 * the token rows, their dispatch (as they are, or quantized on the way) and their
 * combination, forward and backward.  Same library, status codes, conventions and
 * scale layouts as mxfp8moe.h (device pointers owned by the caller, nothing
 * allocated, nothing synchronized, work enqueued on `stream`, argument errors
 * returned before any launch).  Every call can be captured into a graph.
 */
#ifndef MXROUTING_H
#define MXROUTING_H

#include "mxfp4moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MX_MAX_TOP_K 16

/* ----------------------------------------------------------------------------
 * mx_moe_route -- the experts of each token and their weights.
 *   logits [T, E] of `logits_type`; bias [E] fp32 or NULL.
 *   key_te = score(l_te) + bias_e, score as MX_SCORE_*: the logit itself
 *   (MX_SCORE_SOFTMAX), softmax over all experts or 1 / (1 + e^-l).  Without a bias, and
 *   with one that is the same finite value for all, experts rank by their logits, which
 *   order as their scores do.
 *   groups > 1: expert e is of group e / (E / groups); a group is worth the sum of its
 *   two largest keys (MX_GROUP_TOP2; of the one, where only one of its experts can be
 *   selected) or its largest (MX_GROUP_MAX), and only the experts of the top_groups best
 *   groups can be selected.  A bias is part of the keys here even where it is the same
 *   for all: a group with one expert left has it once, others twice.
 *   S_t = the top_k largest keys.  Keys, and sums of keys, rank as exact values do: those
 *   whose order 32 bits leave open are computed in 64.  Ties go to the lowest index; NaN
 *   ranks above everything; an expert whose logit or bias is -inf is never selected.
 *   weights: of MX_SCORE_SOFTMAX softmax of the logits over S_t; of the others their
 *   scores, divided by the sum over S_t where `renormalize` is set; times `scale`.
 *   experts [T, top_k] int32 and weights [T, top_k] fp32 in the order of the keys,
 *   largest first.  A token with fewer than top_k experts to select has -1 and 0 in
 *   the places left.
 *   dense [T, E] fp32 or NULL: the weights by expert, -inf for what is not selected (what
 *   mx_moe_tokens takes with MX_SCORE_GIVEN); with it experts and weights may be NULL.
 *   1 <= E <= MXFP8_MAX_GROUPS, 1 <= top_k <= MX_MAX_TOP_K, groups divides E and is at most
 *   32, top_k <= top_groups * E / groups.  Pointers aligned to their elements.
 * mx_moe_route_bwd -- dlogits [T, E] (of logits_type) from dweights [T, top_k] fp32 for
 *   the selection that mx_moe_route made (which has no gradient, nor has the bias).
 * ------------------------------------------------------------------------- */
enum { MX_LOGITS_FP32 = 0, MX_LOGITS_BF16 = 1, MX_LOGITS_FP16 = 2 };
enum { MX_GROUP_TOP2 = 0, MX_GROUP_MAX = 1 };

mxfp8_status_t mx_moe_route(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t top_k, int32_t score,
                            const float* bias, int32_t groups, int32_t top_groups, int32_t group_score,
                            int32_t renormalize, float scale, int32_t* experts, float* weights, float* dense,
                            mxfp8_stream_t stream);
mxfp8_status_t mx_moe_route_bwd(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t top_k,
                                int32_t score, int32_t renormalize, float scale, const int32_t* experts,
                                const float* dweights, void* dlogits, mxfp8_stream_t stream);

/* ----------------------------------------------------------------------------
 * mx_moe_plan -- rows grouped by expert for the experts [T, top_k] of T tokens
 *   (int32, or int64 where index_bytes is 8; a value outside 0 .. E - 1 takes no row).
 *   Row order: by expert, within an expert by t * top_k + j.  Group sizes are padded to
 *   multiples of `multiple`.
 *   offs [E]: cumulative end rows (of one expert: all rows);  counts [E]: rows that hold a
 *   token;
 *   slot [rows]: t * top_k + j of the row, -1 for padding and for rows past offs[E - 1];
 *   place [T, top_k]: the row, -1 where there is none.
 *   rows >= mx_moe_plan_rows(...), which always suffices: the largest multiple of
 *   `multiple` in T * top_k + min(E, T * top_k) * (multiple - 1).
 *   workspace: mx_moe_plan_workspace bytes (0: none needed), 16-byte aligned, the call's
 *   own until it has finished.
 * ------------------------------------------------------------------------- */
int64_t mx_moe_plan_rows(int64_t T, int32_t top_k, int32_t E, int32_t multiple);
size_t mx_moe_plan_workspace(int64_t T, int32_t top_k, int32_t E);
mxfp8_status_t mx_moe_plan(const void* experts, int32_t index_bytes, int64_t T, int32_t top_k, int32_t E,
                           int32_t multiple, int64_t rows, int32_t* offs, int32_t* counts, int32_t* slot, int32_t* place,
                           void* workspace, size_t workspace_bytes, mxfp8_stream_t stream);

/* ----------------------------------------------------------------------------
 * Rows.  slot [rows] and place [T, top_k] as mx_moe_plan writes them: place[t, j] = r where
 * slot[r] = t * top_k + j, and only there (kernels read the one or the other); entries out
 * of range are taken as -1.  D % 8 == 0; matrices 16-byte aligned.
 * mx_moe_gather -- out[r] = x[slot[r] / top_k], 0 where slot[r] is -1; bf16.
 * mx_moe_combine -- out[t] = sum over j of w[t, j] y[place[t, j]] (w NULL: of ones), fp32
 *   sums in the order of j, one rounding to bf16; y [rows, D], out [T, D] bf16.
 * mx_moe_combine_bwd -- dy[r] = w[slot[r]] dout[slot[r] / top_k], 0 where slot[r] is -1
 *   (dy NULL: not computed); dw[t, j] = <dout[t], y[place[t, j]]> in fp32, 0 where the
 *   place is -1 (dw NULL: not computed, y may be NULL then).
 * ------------------------------------------------------------------------- */
mxfp8_status_t mx_moe_gather(const void* x_bf16, const int32_t* slot, const int32_t* place, int64_t rows, int64_t T,
                             int32_t top_k, int64_t D, void* out_bf16, mxfp8_stream_t stream);
mxfp8_status_t mx_moe_combine(const void* y_bf16, const int32_t* place, const float* w, int64_t rows, int64_t T,
                              int32_t top_k, int64_t D, void* out_bf16, mxfp8_stream_t stream);
mxfp8_status_t mx_moe_combine_bwd(const void* dout_bf16, const void* y_bf16, const int32_t* slot, const int32_t* place,
                                  const float* w, int64_t rows, int64_t T, int32_t top_k, int64_t D, void* dy_bf16,
                                  float* dw, mxfp8_stream_t stream);

/* ----------------------------------------------------------------------------
 * mxfp8_gather_quantize -- mxfp8_quantize_2d(rows, dirs, blocked, offs) of the rows that
 *   mx_moe_gather gives, or with w [T, top_k] of bf16(w * row), without writing them.
 *   dirs: MXFP8_ROW and / or MXFP8_COL; D % 32 == 0; for MXFP8_COL rows and group sizes
 *   are multiples of 32.  Buffers as for mxfp8_quantize_2d with M = rows.
 * mxfp4_gather_quantize -- mxfp4_quantize_2d(rows, blocked, offs) of the same rows.
 * Groups padded to 128 rows are counted in 32 bits: rows + 127 G < 2^31.
 * ------------------------------------------------------------------------- */
mxfp8_status_t mxfp8_gather_quantize(const void* x_bf16, const int32_t* slot, const int32_t* place, const float* w,
                                     int64_t rows, int64_t T, int32_t top_k, int64_t D, unsigned dirs, const int32_t* offs,
                                     int32_t G, void* q_row, void* s_row, void* q_col, void* s_col, int32_t* dev_status,
                                     mxfp8_stream_t stream);
mxfp8_status_t mxfp4_gather_quantize(const void* x_bf16, const int32_t* slot, const int32_t* place, int64_t rows, int64_t T,
                                     int32_t top_k, int64_t D, const int32_t* offs, int32_t G, void* q, void* s,
                                     mxfp8_stream_t stream);

/* ----------------------------------------------------------------------------
 * mxfp8_dequantize -- the values that one copy of mxfp8_quantize_2d stands for, in bf16:
 *   dir MXFP8_ROW: q [M, K], s along K;  MXFP8_COL: q [K, M], s along M.  Scales compact,
 *   or blocked with the row groups of offs (NULL: one group of M rows).  out has q's
 *   shape.  Values are exact but for those below bf16's smallest subnormal, which round;
 *   a block whose scale is 0xFF is NaN; rows (columns) outside every group are 0.
 *   K % 32 == 0, for MXFP8_COL M % 32 == 0; pointers 16-byte aligned; with offs M + 127 G < 2^31.
 * ------------------------------------------------------------------------- */
mxfp8_status_t mxfp8_dequantize(const void* q, const void* s, int64_t M, int64_t K, unsigned dir, int scale_layout,
                                const int32_t* offs, int32_t G, void* out_bf16, mxfp8_stream_t stream);

/* ----------------------------------------------------------------------------
 * mxfp8_swiglu_bwd_quantize_mxfp8 -- mxfp8_swiglu_bwd_quantize with h1 and h3 kept in 8
 *   bits: h1_q, h3_q [M, H] codes and h1_s, h3_s [M, H/32] compact scales, as
 *   mxfp8_quantize_2d(MXFP8_ROW, MXFP8_SCALES_COMPACT) writes them.  The outputs are those
 *   of mxfp8_swiglu_bwd_quantize for the bf16 values that mxfp8_dequantize gives.
 * ------------------------------------------------------------------------- */
mxfp8_status_t mxfp8_swiglu_bwd_quantize_mxfp8(const void* dh_bf16, const void* h1_q, const void* h1_s, const void* h3_q,
                                               const void* h3_s, int64_t M, int64_t H, const int32_t* offs, int32_t G,
                                               void* dh1_q, void* dh1_s, void* dh1T_q, void* dh1T_s, void* dh3_q,
                                               void* dh3_s, void* dh3T_q, void* dh3T_s, int32_t* dev_status,
                                               mxfp8_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MXROUTING_H */
