// Internal launchers of the feed-forward operators.  Arguments are already
// validated by the C ABI layer (ffn_abi.cpp); each returns the HIP error of its
// launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8bsq {

// h = silu(g) * u with g, u [m, f] the block-scaled products of the codes a
// [m, k] (scales a_s; a_s_pow2: all powers of two) and the weights wg, wu
// [f, k].  g_out, u_out: both null, or both receive g and u.
hipError_t launch_gated_gemm(const uint8_t *a, const float *a_s, const uint8_t *wg, const float *wg_s,
                             const uint8_t *wu, const float *wu_s, void *h, void *g_out, void *u_out,
                             bool a_s_pow2, bool out_bf16, int64_t m, int64_t f, int64_t k,
                             hipStream_t stream);

// Columns of the quantized-along-tokens operands: m rounded up to whole blocks.
inline int64_t tokens_padded(int64_t m) { return (m + 127) / 128 * 128; }
// Bytes of one operand's token-block exponents: a 4-byte word per row and four
// token blocks.
inline int64_t token_exp_bytes(int64_t rows, int64_t m) { return (tokens_padded(m) / 128 + 3) / 4 * rows * 4; }

// From dh, g, u [m, f]: dg and du, quantized twice.  Along the features: codes
// rq [m, 2 f] (dg, then du) with scales rs [m, 2 f / 128].  Along the tokens,
// transposed: codes cq [2 f, tokens_padded(m)] with exponents ce.  Either pair
// may be null.
hipError_t launch_ffn_grad_quant(const void *dh, const void *g, const void *u, bool in_bf16, int64_t m,
                                 int64_t f, uint8_t *rq, float *rs, uint8_t *cq, uint8_t *ce,
                                 hipStream_t stream);

// x [m, k] quantized along the tokens, transposed: cq [k, tokens_padded(m)], ce.
hipError_t launch_token_quant(const void *x, bool x_bf16, int64_t m, int64_t k, uint8_t *cq, uint8_t *ce,
                              hipStream_t stream);

// Both weights' codes and scales transposed side by side: wt [k, 2 f],
// wt_s [k / 128, 2 f / 128].
hipError_t launch_weights_transpose(const uint8_t *wg, const float *wg_s, const uint8_t *wu,
                                    const float *wu_s, int64_t f, int64_t k, uint8_t *wt, float *wt_s,
                                    hipStream_t stream);

// dw [2 f, k] = dgu^T x from the token-quantized operands; rows below f go to
// dwg, the others to dwu.
hipError_t launch_weight_grad(const uint8_t *dq, const uint8_t *de, const uint8_t *xq, const uint8_t *xe,
                              void *dwg, void *dwu, bool out_bf16, int64_t m, int64_t f, int64_t k,
                              hipStream_t stream);

// w [n, k] -> codes q [n, k / 2] and E8M0 scales s [n, k / 32].
hipError_t launch_fp4_weight_quant(const void *w, bool w_bf16, int64_t n, int64_t k, uint8_t *q, uint8_t *s,
                                   hipStream_t stream);

// y [m, n] = x [m, k] . W^T (+ bias[n] of y's dtype, if not null).
hipError_t launch_fp4_gemv(const void *x, bool x_bf16, const uint8_t *q, const uint8_t *s, const void *bias,
                           void *y, bool y_bf16, int64_t m, int64_t n, int64_t k, hipStream_t stream);

// Global norm over `count` tensors and, with outs, the clipped tensors.
size_t clip_workspace_bytes(int64_t count);
hipError_t launch_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *numel,
                                 const int32_t *dtypes, int64_t count, float max_norm, float eps,
                                 float *norm, void *workspace, hipStream_t stream);

}  // namespace fp8bsq
