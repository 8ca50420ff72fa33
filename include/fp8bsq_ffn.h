/*
 * fp8bsq_ffn.h -- C ABI of the feed-forward operators on the block-scaled
 * formats of fp8bsq.h, for AMD Instinct MI355X (gfx950): the gated
 * feed-forward block and its backward pass, 4-bit weights with the
 * matrix-vector product that reads them, and gradient clipping by the global
 * norm.  They live in libfp8bsq_ffn.so, which uses libfp8bsq.so.
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

#ifdef __cplusplus
}
#endif

#endif /* FP8BSQ_FFN_H */
