/*
 * mxfp4moe.h -- C ABI of the 4-bit side of the routed-expert library and of the
 * routed layer for a few tokens: MXFP4 quantization and grouped products, and a
 * whole routed SwiGLU layer (top-k, gate, up, SwiGLU, down, weighted sum) for 1 to
 * 64 tokens over MXFP8 or MXFP4 expert weights.  Same library, status codes,
 * conventions and scale layouts as mxfp8moe.h (device pointers owned by the caller,
 * nothing allocated, nothing synchronized, work enqueued on `stream`, argument
 * errors returned before any launch).
 *
 * MXFP4 (OCP Microscaling v1.0): E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives), one E8M0 scale per 32 elements.  e = floor(log2(amax)) - 2
 * clamped at -127, scale byte s = e + 127, element x * 2^-e rounded to nearest
 * even and saturated to +-6.  An all-zero block gets s = 0.  A block holding Inf or
 * NaN gets s = 0xFF (NaN) and every code 7 with the element's sign.
 * Codes are packed two to a byte along the row: element 2i in the low half of byte
 * i, element 2i + 1 in the high half.
 */
#ifndef MXFP4MOE_H
#define MXFP4MOE_H

#include "mxfp8moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------------------------
 * mxfp4_quantize_2d -- x[M, K] bf16 -> q [M, K/2], scales along K.
 *   s: compact [M, K/32], or blocked with row groups from `offs` (offs NULL: one
 *   group of M rows), sized by mxfp8_scale_bytes(M, K, G, layout); the blocked
 *   layout's padding bytes are written as 0.  With offs only the rows inside a
 *   group are written (all of them, for offsets that end at M).
 *   K % 32 == 0, M >= 0; x, q, s 16-byte aligned.
 * mxfp4_swiglu_quantize -- the same for h = silu(h1) * h3 of two bf16 matrices
 *   [M, K], silu(x) = x / (1 + e^-x), computed and quantized in fp32 (h is not
 *   rounded to bf16 on the way).
 * mxfp4_quantize_2d_mxfp8_cols -- both copies that a product with an MXFP4 forward and an
 *   MXFP8 weight gradient needs, from one read of x: q, s as mxfp4_quantize_2d
 *   writes them (blocked), and qT [K, M], sT as mxfp8_quantize_2d writes its
 *   column-wise copy (blocked).  M % 32 == 0; group sizes multiples of 32.
 * mxfp4_quantize_3d_experts -- w[G, N, K] bf16 -> q [G, N, K/2]; scales per expert,
 *   compact [N, K/32] or blocked (ceil(N/128)*128*ceil(K/128)*4 bytes each).
 * mxfp4_quantize_3d_experts_mxfp8_cols -- the same with blocked scales, and the MXFP8
 *   copy along N for the input gradient: qT [G, K, N], sT as mxfp8_quantize_3d_experts
 *   writes its column-wise copy.  N % 32 == 0.
 * mxfp4_dequantize -- the values codes and scales stand for, in bf16 (exact):
 *   out [batch, M, K] from q [batch, M, K/2]; scales compact, or blocked per matrix
 *   (batch > 1 or offs NULL) or blocked with row groups (batch == 1).
 * ------------------------------------------------------------------------- */
mxfp8_status_t mxfp4_quantize_2d(const void* x_bf16, int64_t M, int64_t K, int scale_layout, const int32_t* offs,
                                 int32_t G, void* q, void* s, mxfp8_stream_t stream);
mxfp8_status_t mxfp4_swiglu_quantize(const void* h1_bf16, const void* h3_bf16, int64_t M, int64_t K, int scale_layout,
                                     const int32_t* offs, int32_t G, void* q, void* s, mxfp8_stream_t stream);
mxfp8_status_t mxfp4_quantize_2d_mxfp8_cols(const void* x_bf16, int64_t M, int64_t K, const int32_t* offs, int32_t G,
                                            void* q, void* s, void* qT, void* sT, int32_t* dev_status,
                                            mxfp8_stream_t stream);
mxfp8_status_t mxfp4_quantize_3d_experts_mxfp8_cols(const void* w_bf16, int32_t G, int64_t N, int64_t K, void* q,
                                                    void* s, void* qT, void* sT, int32_t* dev_status,
                                                    mxfp8_stream_t stream);
mxfp8_status_t mxfp4_quantize_3d_experts(const void* w_bf16, int32_t G, int64_t N, int64_t K, int scale_layout,
                                         void* q, void* s, mxfp8_stream_t stream);
mxfp8_status_t mxfp4_dequantize(const void* q, const void* s, int32_t batch, int64_t M, int64_t K, int scale_layout,
                                const int32_t* offs, int32_t G, void* out_bf16, mxfp8_stream_t stream);

/* ----------------------------------------------------------------------------
 * mxfp4_grouped_mm_fwd -- out[m, n] = sum_k A[m,k] W[g][n,k] for the rows m of
 *   group g, fp32 accumulation, bf16 out rounded to nearest even.
 *   a_q [M, K/2], a_s blocked row groups (offs); w_q [G, N, K/2], w_s blocked per
 *   expert; out [M, N].  K % 32 == 0, N % 32 == 0, 1 <= G <= MXFP8_MAX_GROUPS,
 *   every pointer 16-byte aligned, group sizes of any length, M may be 0.  Rows
 *   past the last group's end are not written.
 * ------------------------------------------------------------------------- */
mxfp8_status_t mxfp4_grouped_mm_fwd(const void* a_q, const void* a_s, const void* w_q, const void* w_s,
                                    const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, void* out_bf16,
                                    int32_t* dev_status, mxfp8_stream_t stream);

/* ----------------------------------------------------------------------------
 * mx_moe_tokens -- a routed SwiGLU layer for T = 1 .. 64 tokens in one launch:
 *   S_t  = the top_k largest of router_logits[t] (NaN ranks above everything, ties go to
 *          the lowest expert, -inf is never selected);
 *   w_te = MX_SCORE_SOFTMAX: softmax over S_t; MX_SCORE_SOFTMAX_ALL: softmax over all
 *          experts; MX_SCORE_SIGMOID: 1 / (1 + e^-logit); MX_SCORE_GIVEN: the entry itself
 *          (a matrix of weights with -inf for what is not selected, as mx_moe_route writes it);
 *   h_te = silu(xq_t Wg_e^T) * (xq_t Wu_e^T) in fp32;
 *   y_t  = bf16( sum over e in S_t of w_te MX(h_te) Wd_e^T ), fp32 sums, one rounding.
 * xq = MX(x_t) and MX(h) are quantized along D and H to the weights' format: bits = 8
 * (E4M3, codes [E, H, D] / [E, D, H]) or 4 (E2M1, two codes to a byte).  Weight scales
 * blocked per expert, as mxfp8_quantize_3d_experts / mxfp4_quantize_3d_experts write
 * them.  x [T, D] bf16, router_logits [T, E] fp32, y [T, D] bf16.  A token whose logits
 * are all -inf gets y = 0.  Only the experts that some token selected are read.
 *   D % 32 == 0, H % 32 == 0, E <= 256, top_k <= min(E, 16); pointers 16-byte aligned
 *   (the logits 4).  T == 0 does nothing.
 *   workspace: mx_moe_tokens_workspace(max_tokens, ...) bytes for T <= max_tokens, the
 *   first 256 zero before the first call; it is the launch's own until the launch has
 *   finished (one per stream).  Every launch leaves it ready for the next.
 *   The launch is cooperative (its CTAs wait for one another, each wait bounded:
 *   MXFP8_ERR_TIMEOUT in dev_status); it can be captured into a graph.
 * mx_moe_tokens_workspace returns 0 for arguments mx_moe_tokens would refuse.
 * ------------------------------------------------------------------------- */
enum { MX_SCORE_SOFTMAX = 0, MX_SCORE_SOFTMAX_ALL = 1, MX_SCORE_SIGMOID = 2, MX_SCORE_GIVEN = 16 };

size_t mx_moe_tokens_workspace(int32_t max_tokens, int32_t E, int64_t D, int64_t H, int32_t top_k, int32_t bits);
mxfp8_status_t mx_moe_tokens(const void* x_bf16, const float* router_logits, int32_t T, int32_t E, int64_t D,
                             int64_t H, int32_t top_k, int32_t score, int32_t bits, const void* gate_q,
                             const void* gate_s, const void* up_q, const void* up_s, const void* down_q,
                             const void* down_s, void* workspace, size_t workspace_bytes, void* y_bf16,
                             int32_t* dev_status, mxfp8_stream_t stream);

/* ----------------------------------------------------------------------------
 * mx_debug_moe_tokens -- mx_moe_tokens with the limit of its waits given (0 ns ..
 *   10 s; mx_moe_tokens: 2 s).  With 0, CTAs that wait for one another give up at
 *   once: *dev_status becomes MXFP8_ERR_TIMEOUT, y is incomplete, and the
 *   workspace is ready for the next launch.  It exists so that giving up can be
 *   exercised without a fault or a hang.
 * ------------------------------------------------------------------------- */
mxfp8_status_t mx_debug_moe_tokens(const void* x_bf16, const float* router_logits, int32_t T, int32_t E, int64_t D,
                                   int64_t H, int32_t top_k, int32_t score, int32_t bits, const void* gate_q,
                                   const void* gate_s, const void* up_q, const void* up_s, const void* down_q,
                                   const void* down_s, void* workspace, size_t workspace_bytes, void* y_bf16,
                                   int32_t* dev_status, uint64_t limit_ns, mxfp8_stream_t stream);

/* ----------------------------------------------------------------------------
 * mx_debug_moe_tokens_cut -- how mx_moe_tokens divides one half of the layer (0:
 *   gate and up, 1: down) among `ctas` CTAs, one a multiprocessor, when T tokens
 *   have selected `active` experts: 128 or 64 where every CTA has whole tiles of so
 *   many weight rows, 1 where CTAs share tiles, 0 for arguments out of range.  Host
 *   only; it tells tests which way a size goes.
 * ------------------------------------------------------------------------- */
int32_t mx_debug_moe_tokens_cut(int32_t half, int32_t T, int32_t active, int64_t D, int64_t H, int32_t bits,
                                int32_t ctas);

#ifdef __cplusplus
}
#endif
#endif /* MXFP4MOE_H */
