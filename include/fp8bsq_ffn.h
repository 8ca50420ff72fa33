/*
 * fp8bsq_ffn.h -- C ABI of the feed-forward operators on the block-scaled
 * formats of fp8bsq.h, for AMD Instinct MI355X (gfx950): the gated
 * feed-forward block and its backward pass, 4-bit weights with the
 * matrix-vector product that reads them, gradient clipping by the global norm,
 * and the same block behind a router: tokens sorted by expert and back, and the
 * experts' products.  They live in libfp8bsq_ffn.so, which uses libfp8bsq.so.
 *
 * The conventions of fp8bsq.h hold here too: device pointers owned by the
 * caller, dense row-major tensors, work queued on `hip_stream` without
 * synchronizing, no allocation, fp8bsq_status codes, every argument checked
 * before any HIP call, empty outputs answered with FP8BSQ_OK before any pointer
 * is looked at, finite inputs (NaN and Inf give unspecified but memory-safe
 * outputs unless an entry point says otherwise).  Additions:
 *
 *  - A workspace is device memory of at least the size that the entry point's
 *    ..._workspace function gives for the same sizes with the same device
 *    current, 256-byte aligned, with no initial contents required, in use until
 *    the queued work has finished.  A smaller one is FP8BSQ_ESCRATCH.  Calls that
 *    share one workspace must not overlap.
 *  - That size follows from how a product is planned for the device's compute
 *    units, for which the runtime is asked: a workspace's size is the one argument
 *    whose check makes HIP calls (it queues nothing).
 *  - The ..._workspace functions answer 0 for sizes that the call refuses; the
 *    call says FP8BSQ_ERANGE or FP8BSQ_ESHAPE then, before it looks at the
 *    workspace.
 *  - fp8bsq_strerror (libfp8bsq.so) describes the status codes.
 */
#ifndef FP8BSQ_FFN_H
#define FP8BSQ_FFN_H

#include <stddef.h>
#include <stdint.h>

#include "fp8bsq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp8_gated_ffn -- the gated half of a feed-forward block:
 *     (a, a_s) = fp8_act_quant(x, scale_fmt)
 *     g = a . w_gate^T,  u = a . w_up^T     (fp8_block_gemm's product, in FP32)
 *     h = silu(g) * u,   silu(g) = g / (1 + exp(-g))
 * with both products, the activation and the product in one kernel.
 *
 *   x            [m, k] activations, dtype x_dtype (FP8BSQ_F32 or FP8BSQ_BF16),
 *                16-byte aligned.
 *   w_gate, w_up [f, k] E4M3 codes, 16-byte aligned, with their
 *   .._s         [ceil(f / 128), k / 128] FP32 block scales, 4-byte aligned.
 *   h            [m, f] out, dtype out_dtype, aligned to its elements.
 *   g, u         [m, f] out, of the same dtype, or both NULL: the values the
 *                backward pass takes.
 *   m, f, k      m, f >= 0; k >= 128, k % 128 == 0 (else FP8BSQ_ESHAPE; k = 0 is
 *                FP8BSQ_EINVAL); m <= 65535 * 16, f, k <= 2^21 (else
 *                FP8BSQ_ERANGE).  m or f = 0: nothing to do.
 *
 * g and u meet fp8_block_gemm's error bound; they are rounded once, from the
 * FP32 values that h is formed from.
 */
FP8BSQ_API int fp8_gated_ffn(const void *x, int x_dtype, int scale_fmt, const uint8_t *w_gate,
                  const float *w_gate_s, const uint8_t *w_up, const float *w_up_s, void *h, void *g,
                  void *u, int out_dtype, int64_t m, int64_t f, int64_t k, void *workspace,
                  size_t workspace_bytes, void *hip_stream);
FP8BSQ_API size_t fp8_gated_ffn_workspace(int64_t m, int64_t f, int64_t k);

/*
 * fp8_gated_ffn_backward -- gradients of fp8_gated_ffn, its quantization taken
 * as the identity:
 *     dg = dh u silu'(g),   du = dh silu(g),   silu'(g) = s (1 + g (1 - s)), s = 1 / (1 + exp(-g))
 *     dx      = Q(dg) . W_gate + Q(du) . W_up      Q over 128 features
 *     dw_gate = Q(dg)^T . Q(x),  dw_up = Q(du)^T . Q(x)    Q over 128 tokens
 * W are the weights the codes stand for.  Q rounds to E4M3 with one scale per
 * 128 consecutive values along the contraction, the smallest power of two s
 * with max |v| <= 448 s (max |v| taken as at least 2^-100); the last block of
 * tokens is filled up with zeros.  Products are accumulated in FP32.
 *
 *   dh, g, u     [m, f], x [m, k]: all of dtype in_dtype, 16-byte aligned.
 *   w_..         as for fp8_gated_ffn.
 *   dx           [m, k] out, or NULL: not computed (w_.. are not read and may
 *                then be NULL).
 *   dw_gate, dw_up  [f, k] out, or both NULL: not computed (x is not read and
 *                may then be NULL).
 *                Outputs have dtype out_dtype and are 16-byte aligned.
 *   m, f, k      m, f, k >= 0, f and k multiples of 128 (else FP8BSQ_ESHAPE);
 *                ranges as for fp8_gated_ffn.
 *                f = 0 or k = 0 is FP8BSQ_EINVAL.  m = 0: dw_gate and dw_up are
 *                set to zero, and nothing else is read or written.
 */
FP8BSQ_API int fp8_gated_ffn_backward(const void *dh, const void *x, const void *g, const void *u,
                           int in_dtype, const uint8_t *w_gate, const float *w_gate_s,
                           const uint8_t *w_up, const float *w_up_s, void *dx, void *dw_gate,
                           void *dw_up, int out_dtype, int64_t m, int64_t f, int64_t k,
                           void *workspace, size_t workspace_bytes, void *hip_stream);
FP8BSQ_API size_t fp8_gated_ffn_backward_workspace(int64_t m, int64_t f, int64_t k);

/*
 * fp4_weight_quant -- 4-bit weights: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * a sign bit) with one power-of-two scale per 32 consecutive weights of a row.
 *
 *   w        [n, k], dtype w_dtype, 16-byte aligned; n, k >= 0, k % 32 == 0
 *            (else FP8BSQ_ESHAPE); either 0: nothing to do.
 *   q        [n, k / 2] out, 4-byte aligned: byte j holds the code of weight 2 j
 *            in its low half and of weight 2 j + 1 in its high half.
 *   s        [n, k / 32] out: E8M0 bytes e, the scale being 2^(e - 127), the
 *            smallest power of two with max |w| <= 6 * scale (max |w| taken as
 *            at least 2^-100).
 *   code = E2M1(w / scale), round to nearest even, the sign kept on zero.
 */
FP8BSQ_API int fp4_weight_quant(const void *w, int w_dtype, int64_t n, int64_t k, uint8_t *q, uint8_t *s,
                     void *hip_stream);

/*
 * fp4_gemv -- y = x . W^T (+ bias) with a 4-bit weight: one matrix-vector
 * product per row of x.  Made for few rows (the decode step); any number works.
 *
 *   x        [m, k] activations, dtype x_dtype, 16-byte aligned.
 *   q, s     as fp4_weight_quant writes them; q 16-byte aligned; scale bytes
 *            0..252.  With 253 (which the quantizer writes for weights above
 *            6 * 2^125 only) codes of 4 and 6 are beyond the weights' bf16, with
 *            254 those from 2 on: such a row's results are infinite or NaN.
 *   bias     [n] of y's dtype, or NULL.
 *   y        [m, n] out, dtype y_dtype, aligned to its elements.
 *   m, n, k  m, n >= 0; k >= 32, k % 32 == 0 (else FP8BSQ_ESHAPE; k = 0 is
 *            FP8BSQ_EINVAL); m <= 65535 * 16, n <= 144 * (2^22 - 1), k <= 2^27 (else
 *            FP8BSQ_ERANGE).
 *
 * Every product x * w is exact, of fp32 x down to |x| = 2^-110; below, x loses
 * what lies under 2^-133.  Sums are FP32.
 */
FP8BSQ_API int fp4_gemv(const void *x, int x_dtype, const uint8_t *q, const uint8_t *s, const void *bias,
             void *y, int y_dtype, int64_t m, int64_t n, int64_t k, void *hip_stream);

/*
 * fp8bsq_clip_grad_norm -- norm = sqrt(sum over all tensors of sum g^2), and
 * out = g * min(1, max_norm / (norm + eps)).
 *
 *   grads, outs, numels, dtypes   HOST arrays of `count` entries, read during
 *            the call: device pointers (aligned to their elements, NULL allowed
 *            where numel is 0), element counts >= 0, FP8BSQ_F32 or FP8BSQ_BF16.
 *            outs = NULL: the norm only.  outs[i] has grads[i]'s dtype and is
 *            grads[i] itself (clipped in place, then apart from all other
 *            grads) or does not overlap any grad; outs do not overlap.  This is
 *            not checked.
 *   max_norm, eps   >= 0; the factor is 1 where max_norm >= norm + eps, so also
 *            for an infinite max_norm, and for max_norm = norm + eps = 0.
 *   norm     device float out, 4-byte aligned.
 *
 * Squares are summed in FP64 in a fixed order: equal calls give equal bits, and
 * no square of a finite gradient overflows.  A NaN among the gradients makes
 * the norm and all outputs NaN; an infinite norm above max_norm gives the factor
 * 0 (and NaN where a gradient is infinite).
 */
FP8BSQ_API int fp8bsq_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *numels,
                          const int32_t *dtypes, int64_t count, float max_norm, float eps, float *norm,
                          void *workspace, size_t workspace_bytes, void *hip_stream);
FP8BSQ_API size_t fp8bsq_clip_grad_norm_workspace(int64_t count);

/*
 * The expert operators.  `tokens` tokens choose `top_k` experts each; choice
 * c = t * top_k + j is token t's j-th.  The n = tokens * top_k choices, sorted by
 * expert, have a row each:
 *
 *   offsets  [num_experts + 1] int32: expert e's rows are offsets[e] .. offsets[e + 1] - 1.
 *   rows     [n] int32: choice c's row r; ~r (negative) for a choice that takes no
 *            part, its row then being one of those behind, from offsets[num_experts] on.
 *
 * Sizes: tokens >= 0, top_k >= 1, n < 2^31, 1 <= num_experts <= 1024, and the
 * rows' lengths as the entry points say; else FP8BSQ_ERANGE (negative sizes,
 * top_k = 0 and num_experts = 0: FP8BSQ_EINVAL).  What offsets and rows hold is not
 * checked; other contents than fp8bsq_expert_sort's give unspecified but
 * memory-safe outputs.
 */

/*
 * fp8bsq_expert_sort -- the stable sort of the choices by expert.
 *
 *   experts  [n] expert numbers, int32 or int64 (index_bytes 4 or 8), aligned to
 *            their size.  A number outside 0 .. num_experts - 1 takes no part: a
 *            padded token's, or an expert's of another rank.
 *   offsets, rows, choices   out, 4-byte aligned: the above, and [n] int32 the
 *            choice of each row (the inverse of rows, also behind).
 *            Within an expert, and behind, rows follow the order of the choices.
 *   n = 0    offsets are set to zero.
 *   workspace   may be NULL where its size is 0.
 */
FP8BSQ_API int fp8bsq_expert_sort(const void *experts, int index_bytes, int64_t n, int64_t num_experts, int32_t *offsets,
                       int32_t *rows, int32_t *choices, void *workspace, size_t workspace_bytes, void *hip_stream);
FP8BSQ_API size_t fp8bsq_expert_sort_workspace(int64_t n, int64_t num_experts);

/*
 * fp8bsq_expert_dispatch -- y[rows[c]] = x[c / top_k], and zeros in the rows behind.
 *
 *   x        [tokens, h], y [n, h] out, both of `dtype`, aligned to their elements.
 *   h        0 <= h <= 2^21.
 *
 * Its gradient is fp8bsq_expert_combine with weights NULL.
 */
FP8BSQ_API int fp8bsq_expert_dispatch(const void *x, int dtype, const int32_t *rows, int64_t tokens, int64_t top_k, int64_t h,
                           void *y, void *hip_stream);

/*
 * fp8_expert_dispatch_quant -- fp8_act_quant of that, each token quantized once.
 *
 *   x        [tokens, h], dtype x_dtype, 16-byte aligned; h % 128 == 0 (else
 *            FP8BSQ_ESHAPE), 0 <= h <= 2^21.
 *   y, s     [n, h] E4M3 codes out, 16-byte aligned, and [n, h / 128] FP32 scales
 *            out, 4-byte aligned; the rows behind are those of rows of zeros.
 */
FP8BSQ_API int fp8_expert_dispatch_quant(const void *x, int x_dtype, int scale_fmt, const int32_t *rows, int64_t tokens,
                              int64_t top_k, int64_t h, uint8_t *y, float *s, void *hip_stream);

/*
 * fp8bsq_expert_combine -- out[t] = sum over j of weights[t, j] y[rows[t, j]], in
 * FP32 and j's order; choices that take no part are left out, and what y holds in
 * the rows behind is not read.
 *
 *   y        [n, h], out [tokens, h] out, both of `dtype`, aligned to their
 *            elements.  No other tensor overlaps out.
 *   weights  [tokens, top_k], dtype w_dtype, aligned to its elements, or NULL: ones.
 *   h        0 <= h <= 2^21.
 */
FP8BSQ_API int fp8bsq_expert_combine(const void *y, int dtype, const int32_t *rows, const void *weights, int w_dtype,
                          int64_t tokens, int64_t top_k, int64_t h, void *out, void *hip_stream);

/*
 * fp8bsq_expert_combine_backward --
 *     dy[rows[t, j]] = weights[t, j] dout[t]             (rows behind: zero)
 *     dweights[t, j] = sum of dout[t] * y[rows[t, j]]    (taking no part: zero)
 *
 *   dout     [tokens, h], y [n, h], dy [n, h] out, of `dtype`; 0 <= h <= 2^21.  All are
 *            aligned to their elements, and dy overlaps no other tensor.
 *   dy       or NULL: not computed.
 *   dweights [tokens, top_k] out, dtype w_dtype, or NULL: not computed (y is not
 *            read and may then be NULL).  Sums are FP32, in a fixed order.
 */
FP8BSQ_API int fp8bsq_expert_combine_backward(const void *dout, const void *y, int dtype, const int32_t *rows,
                                   const void *weights, int w_dtype, int64_t tokens, int64_t top_k, int64_t h, void *dy,
                                   void *dweights, void *hip_stream);

/*
 * fp8_expert_gemm -- c[r] = a[r] . b[e]^T for expert e's rows r, fp8_block_gemm's
 * product; the rows behind are zero.
 *
 *   a, a_s   [rows, k] E4M3 codes, 16-byte aligned, and [rows, k / 128] FP32
 *            scales, 4-byte aligned; the rows behind are not read.
 *   offsets  as fp8bsq_expert_sort writes them.
 *   b, b_s   [num_experts, n, k] E4M3 codes, 16-byte aligned, and
 *            [num_experts, ceil(n / 128), k / 128] FP32 scales, 4-byte aligned.
 *   c        [rows, n] out, dtype c_dtype, aligned to its elements.
 *   sizes    rows, n >= 0; k >= 128, k % 128 == 0 (else FP8BSQ_ESHAPE; k = 0 is
 *            FP8BSQ_EINVAL); rows <= 65535 * 16, n, k <= 2^21, num_experts as above
 *            (else FP8BSQ_ERANGE).  rows or n = 0: nothing to do.
 *
 * Results meet fp8_block_gemm's error bound.  Equal calls give equal bits.  The order in
 * which a row's K blocks are added goes by rows, num_experts, n and k: up to k = 512 it
 * is always the same, and from k = 640 on a row's last bits can change with the number
 * of rows that come along.
 */
FP8BSQ_API int fp8_expert_gemm(const uint8_t *a, const float *a_s, const int32_t *offsets, const uint8_t *b,
                    const float *b_s, void *c, int c_dtype, int64_t rows, int64_t num_experts, int64_t n, int64_t k,
                    void *hip_stream);

/*
 * fp8_expert_gated_ffn -- h[r] = silu(g) * u, g = a[r] . w_gate[e]^T and
 * u = a[r] . w_up[e]^T: fp8_gated_ffn of each expert's rows, already quantized.
 *
 *   w_gate, w_up, .._s   [num_experts, f, k] and [num_experts, ceil(f / 128), k / 128].
 *   h        [rows, f] out, dtype out_dtype, aligned to its elements; the rows
 *            behind are zero.
 *   others, sizes        as for fp8_expert_gemm.
 */
FP8BSQ_API int fp8_expert_gated_ffn(const uint8_t *a, const float *a_s, const int32_t *offsets, const uint8_t *w_gate,
                         const float *w_gate_s, const uint8_t *w_up, const float *w_up_s, void *h, int out_dtype,
                         int64_t rows, int64_t num_experts, int64_t f, int64_t k, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BSQ_FFN_H */
