// Internal launchers of the feed-forward operators.  Arguments are already
// validated by the C ABI layer (ffn_abi.cpp); each returns the HIP error of its
// launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8bsq {

// Where the pieces of a feed-forward call's workspace start, each 256-byte
// aligned, and its size.
struct FfnSpace {
  size_t bytes = 0;
  size_t a = 0, a_s = 0;          // columns operand of the (input) product, its scales
  size_t cq = 0, cs = 0;          // backward: (dg | du)^T quantized along the tokens
  size_t xq = 0, xs = 0;          // backward: x^T quantized along the tokens
  size_t partials = 0;            // of a split product
  size_t add(int64_t n) {
    const size_t at = bytes;
    bytes += ((size_t)n + 255) / 256 * 256;
    return at;
  }
};

// Tokens rounded up to whole blocks of 128, and rows to the widest tile (what a
// scale row's stride allows for).
inline int64_t tokens_padded(int64_t m) { return (m + 127) / 128 * 128; }
inline int64_t rows_padded(int64_t rows) { return (rows + 255) / 256 * 256; }

// h = silu(g) * u; g_out, u_out: both null, or both receive g and u.
// workspace: gated_space(m, f, k).bytes.
FfnSpace gated_space(int64_t m, int64_t f, int64_t k);
hipError_t launch_gated_ffn(const void *x, bool x_bf16, bool ue8m0, const uint8_t *wg, const float *wg_s,
                            const uint8_t *wu, const float *wu_s, void *h, void *g_out, void *u_out, bool out_bf16,
                            int64_t m, int64_t f, int64_t k, void *workspace, hipStream_t stream);

// dx, or dwg and dwu, may be null; with m = 0 only the weights' (zero)
// gradients are written.  workspace: backward_space(m, f, k).bytes.
FfnSpace backward_space(int64_t m, int64_t f, int64_t k);
hipError_t launch_gated_ffn_backward(const void *dh, const void *x, const void *g, const void *u, bool in_bf16,
                                     const uint8_t *wg, const float *wg_s, const uint8_t *wu, const float *wu_s,
                                     void *dx, void *dwg, void *dwu, bool out_bf16, int64_t m, int64_t f, int64_t k,
                                     void *workspace, hipStream_t stream);

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
