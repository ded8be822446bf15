/*
 * libroutedmoe, dense path in 8 bits: what a decoder does around the routed-MoE layer and its
 * attention.  The residual's addition with a root-mean-square norm, rows quantised to 8 bits,
 * products with block-scaled 8-bit weights (one weight, or one for each group of rows), and the
 * log probabilities by which drafted tokens are accepted.
 *
 * The pages keep the dense layers and the vocabulary in FP8 with a scale for 128 x 128 of a weight
 * ("How I forked vLLM and made Qwen3.8-Flash-Next decode 1.6x faster on one GPU", sections 2 and 3);
 * the norm is the one that follows the layer's residual ("TokenSpeed: Qwen3.8-Flash-Next
 * optimisations", section "Residual update and normalization fusion").
 *
 * Rows in 8 bits.  codes [rows][k] E4M3 (row stride in bytes), scales FP32, one for a row and 128
 * consecutive channels (the last block may be shorter): the scale of row r and block b lies at
 * scales[r * scale_row + b * scale_block].  A block of values v is held as
 *     s = max|v| / 448 (rounded to FP32),   code = E4M3(v / s)   (the exact quotient, to nearest even)
 * with codes 0 where s is 0.  A block with an infinity or a NaN has a NaN scale, so that what is
 * computed from that row is NaN.
 *
 * Weights.  codes [n][k] E4M3, rows consecutive (k bytes apart); scales FP32
 * [ceil(n / 128)][ceil(k / 128)], one for 128 x 128 of the codes.  With groups, one such weight
 * after the other.
 *
 * Conventions are those of moe.h: device pointers owned by the caller, asynchronous calls that can
 * be captured in a CUDA graph, host-detected errors returned before anything is enqueued, nothing
 * kept between calls, and no workspace: calls on different streams do not meet.  Outputs do not
 * overlap inputs or each other unless a call says so, and an output's rows lie apart.  The products OR device-detected conditions into the
 * caller's status word (moe_dense_read_status).
 */
#ifndef ROUTED_MOE_DENSE_H
#define ROUTED_MOE_DENSE_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Status bits of a product. */
#define MOE_DENSE_BAD_OFFSETS 0x1u /* a group's offsets decrease or leave [0, rows]: they are cut to that
                                      range, a group begins where those before it have ended at the
                                      earliest, and one that would end before it begins has no rows */
#define MOE_DENSE_TIMEOUT 0x2u     /* a bounded wait gave up: the product's results are not valid */

/* Element types. */
#define MOE_DENSE_FP32 0
#define MOE_DENSE_BF16 1
#define MOE_DENSE_FP16 2

/* For every row of d values:
 *     h = x + residual, rounded to `dtype` (h = x without a residual)
 *     n = h / sqrt(mean(h^2) + eps) * w,   w = weight, or 1 + weight with one_plus
 * and residual_out = h, normed = n rounded to `dtype`, codes and scales = n (not rounded) in 8 bits.
 * outer * inner rows: row r of x lies at (r / inner) * x_outer + (r % inner) * x_inner elements, of
 * normed likewise (heads of a fused projection's rows); residual, residual_out and the codes have
 * one stride.  residual, residual_out (needs residual), normed and codes (with scales) may be null,
 * but something is written.  residual_out may be x or residual; normed may be x or residual; with the same strides.
 * Sums and statistics in FP32; a row whose mean square (with eps) FP32 does not hold as a normal value is
 * summed times a power of two.  In a row with an infinity what is finite becomes 0 and the infinity NaN.
 * Any d >= 1; rows of 16-byte aligned starts and lengths are faster.
 * dtype, weight_dtype: MOE_DENSE_*. */
MOE_API int moe_rms_norm(int outer, int inner, int d, int dtype, const void* x, int64_t x_outer, int64_t x_inner,
                         const void* residual, int64_t residual_stride, const void* weight, int weight_dtype,
                         int one_plus, float eps, void* residual_out, int64_t residual_out_stride, void* normed,
                         int64_t normed_outer, int64_t normed_inner, uint8_t* codes, int64_t code_stride,
                         float* scales, int64_t scale_row, int64_t scale_block, moe_stream_t stream);

/* rows of d values in 8 bits; gated: x has 2 d values a row, gate then up, and what is quantised is
 * gate / (1 + exp(-gate)) * up (FP32; a gate below -87.3, where exp(gate) is no normal value, counts as 0). */
MOE_API int moe_quantize_rows(int rows, int d, int gated, int dtype, const void* x, int64_t x_stride,
                              uint8_t* codes, int64_t code_stride, float* scales, int64_t scale_row,
                              int64_t scale_block, moe_stream_t stream);

/* out[t][c] = sum over blocks b of scales[t][b] * w_scales[c / 128][b] *
 *             (sum over the block's channels k of codes[t][k] * w_codes[c][k]),
 * sums in FP32, rounded once to out_dtype.  k a multiple of 16; codes, w_codes 16-byte aligned, code_stride
 * a multiple of 16 (of one row it says nothing); out rows out_stride elements apart, channels consecutive.
 *
 * groups > 0: w_codes [groups][n][k] (w_scales likewise), and rows offsets[g] .. offsets[g + 1] - 1
 * meet weight g (offsets on the device, [groups + 1], non-decreasing, within [0, rows]; empty groups
 * are allowed).  Rows of no group are left as they were.  groups <= 1024.
 * groups = 0: one weight, offsets null.
 * status: one word on the device. */
MOE_API int moe_fp8_matmul(int rows, int n, int k, int groups, const uint8_t* codes, int64_t code_stride,
                           const float* scales, int64_t scale_row, int64_t scale_block, const uint8_t* w_codes,
                           const float* w_scales, const int32_t* offsets, void* out, int64_t out_stride,
                           int out_dtype, uint32_t* status, moe_stream_t stream);

/* For every row of `vocab` logits, x = scale * logits (FP32):
 *     lse = log(sum exp(x)),  logprobs[j] = x[tokens[j]] - lse,  entropy = lse - sum exp(x - lse) x
 * and the `top` best tokens by logit (equal logits: the lower id first; -0 equals 0), with their log probabilities.
 * tokens [rows][n_tokens] int32 (row stride token_stride); logprobs [rows][n_tokens], lse [rows],
 * entropy [rows], top_ids and top_logprobs [rows][top], all contiguous; any output may be null, both
 * of the last two are null where top is 0.  n_tokens <= 1024, top <= 32, top <= vocab, 2^-80 <= scale <= 2^80.
 * A logit of -infinity has probability 0 and log probability -infinity; so has a token outside
 * [0, vocab).  A row of nothing else has lse -infinity, log probabilities -infinity and entropy 0.
 * A row with a NaN or +infinity (also where scale * logit is that in FP32) has NaN for them; its alternatives are ordered as if the NaNs were
 * -infinity. */
MOE_API int moe_token_logprobs(int rows, int vocab, int dtype, const void* logits, int64_t row_stride, float scale,
                               const int32_t* tokens, int n_tokens, int64_t token_stride, int top, float* logprobs,
                               float* lse, float* entropy, int32_t* top_ids, float* top_logprobs,
                               moe_stream_t stream);

/* The product's status word: read on `stream`, with `clear` non-zero exchanged for 0 in the same step, and waited for.  It has the
 * bits of the products that are ordered before this call on `stream`, and of others that ran by then; a bit that a product of
 * another stream sets meanwhile is in this result or stays for the next.  MOE_OK if no bit is set, MOE_ERR_DEVICE if any is. */
MOE_API int moe_dense_read_status(uint32_t* status, int clear, uint32_t* status_bits, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ROUTED_MOE_DENSE_H */
