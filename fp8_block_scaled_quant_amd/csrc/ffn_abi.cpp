// C ABI of the feed-forward operators: argument validation, workspace layout
// and dispatch.  Every check runs before anything is queued; the one of a
// workspace's size asks the runtime for the current device's compute units, by
// which the products are planned.
#include <stddef.h>
#include <stdint.h>

#include "ffn_launch.h"
#include "fp8bsq_ffn.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;
// A launch has fewer than 2^32 threads along an axis, and more are dropped without
// an error: the matrix-vector product's workgroups have up to 1024 for 144 rows of a
// weight of so many.
constexpr int64_t kMaxGemvN = 144 * (((int64_t)1 << 22) - 1);
constexpr int64_t kMaxRows = (int64_t)65535 * 16;     // grid.y limit of the smallest row tile
constexpr int64_t kMaxFeatures = (int64_t)1 << 21;    // features and K of the feed-forward block
constexpr int64_t kMaxGemvK = (int64_t)1 << 27;       // 16 rows of codes within 32-bit offsets

bool aligned(const void *p, uintptr_t bytes) { return ((uintptr_t)p % bytes) == 0; }
bool known_dtype(int d) { return d == FP8BSQ_F32 || d == FP8BSQ_BF16; }
uintptr_t size_of(int dtype) { return dtype == FP8BSQ_F32 ? 4 : 2; }
int launch_status(hipError_t e) { return e == hipSuccess ? FP8BSQ_OK : FP8BSQ_ELAUNCH; }

// Rows reach the tile kernels by 32-bit offsets from their tile.
bool ffn_sizes_ok(int64_t m, int64_t f, int64_t k) {
  return m > 0 && f > 0 && k > 0 && k % 128 == 0 && m <= kMaxRows && f <= kMaxFeatures && k <= kMaxFeatures;
}

}  // namespace

extern "C" {

size_t fp8_gated_ffn_workspace(int64_t m, int64_t f, int64_t k) {
  return ffn_sizes_ok(m, f, k) ? fp8bsq::gated_space(m, f, k).bytes : 0;
}

int fp8_gated_ffn(const void *x, int x_dtype, int scale_fmt, const uint8_t *w_gate, const float *w_gate_s,
                  const uint8_t *w_up, const float *w_up_s, void *h, void *g, void *u, int out_dtype, int64_t m,
                  int64_t f, int64_t k, void *workspace, size_t workspace_bytes, void *hip_stream) {
  if (m < 0 || f < 0 || k <= 0) return FP8BSQ_EINVAL;
  if (!known_dtype(x_dtype) || !known_dtype(out_dtype)) return FP8BSQ_EINVAL;
  if (scale_fmt != FP8BSQ_SCALE_NONE && scale_fmt != FP8BSQ_SCALE_UE8M0) return FP8BSQ_EINVAL;
  if (k % 128 != 0) return FP8BSQ_ESHAPE;
  if (m == 0 || f == 0) return FP8BSQ_OK;
  if (!x || !w_gate || !w_gate_s || !w_up || !w_up_s || !h || !g != !u) return FP8BSQ_EINVAL;
  // no workspace holds such sizes: its size was answered with 0
  if (!ffn_sizes_ok(m, f, k)) return FP8BSQ_ERANGE;
  if (!workspace) return FP8BSQ_EINVAL;
  const uintptr_t out = size_of(out_dtype);
  if (!aligned(x, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_gate_s, 4) ||
      !aligned(w_up_s, 4) || !aligned(h, out) || !aligned(g, out) || !aligned(u, out) || !aligned(workspace, 256))
    return FP8BSQ_EALIGN;
  if (workspace_bytes < fp8bsq::gated_space(m, f, k).bytes) return FP8BSQ_ESCRATCH;
  return launch_status(fp8bsq::launch_gated_ffn(x, x_dtype == FP8BSQ_BF16, scale_fmt == FP8BSQ_SCALE_UE8M0, w_gate,
                                                w_gate_s, w_up, w_up_s, h, g, u, out_dtype == FP8BSQ_BF16, m, f, k,
                                                workspace, (hipStream_t)hip_stream));
}

size_t fp8_gated_ffn_backward_workspace(int64_t m, int64_t f, int64_t k) {
  return ffn_sizes_ok(m, f, k) && f % 128 == 0 ? fp8bsq::backward_space(m, f, k).bytes : 0;
}

int fp8_gated_ffn_backward(const void *dh, const void *x, const void *g, const void *u, int in_dtype,
                           const uint8_t *w_gate, const float *w_gate_s, const uint8_t *w_up,
                           const float *w_up_s, void *dx, void *dw_gate, void *dw_up, int out_dtype, int64_t m,
                           int64_t f, int64_t k, void *workspace, size_t workspace_bytes, void *hip_stream) {
  if (m < 0 || f <= 0 || k <= 0) return FP8BSQ_EINVAL;
  if (!known_dtype(in_dtype) || !known_dtype(out_dtype)) return FP8BSQ_EINVAL;
  if (f % 128 != 0 || k % 128 != 0) return FP8BSQ_ESHAPE;
  if (!dw_gate != !dw_up) return FP8BSQ_EINVAL;
  const hipStream_t st = (hipStream_t)hip_stream;
  const bool in_bf16 = in_dtype == FP8BSQ_BF16, out_bf16 = out_dtype == FP8BSQ_BF16;
  if (m == 0) {
    if (!dw_gate) return FP8BSQ_OK;
    if (!aligned(dw_gate, 16) || !aligned(dw_up, 16)) return FP8BSQ_EALIGN;
    if (!ffn_sizes_ok(1, f, k)) return FP8BSQ_ERANGE;
    // no tokens: the product over an empty contraction
    return launch_status(fp8bsq::launch_gated_ffn_backward(nullptr, nullptr, nullptr, nullptr, in_bf16, nullptr,
                                                           nullptr, nullptr, nullptr, nullptr, dw_gate, dw_up,
                                                           out_bf16, 0, f, k, nullptr, st));
  }
  if (!dx && !dw_gate) return FP8BSQ_OK;
  if (!dh || !g || !u || (dx && (!w_gate || !w_gate_s || !w_up || !w_up_s)) || (dw_gate && !x)) return FP8BSQ_EINVAL;
  if (!ffn_sizes_ok(m, f, k)) return FP8BSQ_ERANGE;
  if (!workspace) return FP8BSQ_EINVAL;
  if (!aligned(dh, 16) || !aligned(g, 16) || !aligned(u, 16) || !aligned(x, 16) || !aligned(w_gate, 16) ||
      !aligned(w_up, 16) || !aligned(w_gate_s, 4) || !aligned(w_up_s, 4) || !aligned(dx, 16) ||
      !aligned(dw_gate, 16) || !aligned(dw_up, 16) || !aligned(workspace, 256))
    return FP8BSQ_EALIGN;
  if (workspace_bytes < fp8bsq::backward_space(m, f, k).bytes) return FP8BSQ_ESCRATCH;
  return launch_status(fp8bsq::launch_gated_ffn_backward(dh, x, g, u, in_bf16, w_gate, w_gate_s, w_up, w_up_s, dx,
                                                         dw_gate, dw_up, out_bf16, m, f, k, workspace, st));
}

int fp4_weight_quant(const void *w, int w_dtype, int64_t n, int64_t k, uint8_t *q, uint8_t *s, void *hip_stream) {
  if (n < 0 || k < 0) return FP8BSQ_EINVAL;
  if (!known_dtype(w_dtype)) return FP8BSQ_EINVAL;
  if (k % 32 != 0) return FP8BSQ_ESHAPE;
  if (n == 0 || k == 0) return FP8BSQ_OK;
  if (!w || !q || !s) return FP8BSQ_EINVAL;
  if (!aligned(w, 16) || !aligned(q, 4)) return FP8BSQ_EALIGN;
  if (n >= kMaxDim || k >= kMaxDim || n * (k / 32) >= (int64_t)1 << 37) return FP8BSQ_ERANGE;
  return launch_status(
      fp8bsq::launch_fp4_weight_quant(w, w_dtype == FP8BSQ_BF16, n, k, q, s, (hipStream_t)hip_stream));
}

int fp4_gemv(const void *x, int x_dtype, const uint8_t *q, const uint8_t *s, const void *bias, void *y,
             int y_dtype, int64_t m, int64_t n, int64_t k, void *hip_stream) {
  if (m < 0 || n < 0 || k <= 0) return FP8BSQ_EINVAL;
  if (!known_dtype(x_dtype) || !known_dtype(y_dtype)) return FP8BSQ_EINVAL;
  if (k % 32 != 0) return FP8BSQ_ESHAPE;
  if (m == 0 || n == 0) return FP8BSQ_OK;
  if (!x || !q || !s || !y) return FP8BSQ_EINVAL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(bias, size_of(y_dtype)) || !aligned(y, size_of(y_dtype)))
    return FP8BSQ_EALIGN;
  if (m > kMaxRows || n > kMaxGemvN || k > kMaxGemvK) return FP8BSQ_ERANGE;
  return launch_status(fp8bsq::launch_fp4_gemv(x, x_dtype == FP8BSQ_BF16, q, s, bias, y, y_dtype == FP8BSQ_BF16, m,
                                               n, k, (hipStream_t)hip_stream));
}

size_t fp8bsq_clip_grad_norm_workspace(int64_t count) { return count < 0 ? 0 : fp8bsq::clip_workspace_bytes(count); }

int fp8bsq_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *numels,
                          const int32_t *dtypes, int64_t count, float max_norm, float eps, float *norm,
                          void *workspace, size_t workspace_bytes, void *hip_stream) {
  if (count < 0 || !(max_norm >= 0.0f) || !(eps >= 0.0f)) return FP8BSQ_EINVAL;
  if (!norm || !workspace || (count > 0 && (!grads || !numels || !dtypes))) return FP8BSQ_EINVAL;
  for (int64_t i = 0; i < count; ++i) {
    if (numels[i] < 0 || !known_dtype(dtypes[i])) return FP8BSQ_EINVAL;
    if (numels[i] > 0 && (!grads[i] || (outs && !outs[i]))) return FP8BSQ_EINVAL;
    const uintptr_t size = size_of(dtypes[i]);
    if (!aligned(grads[i], size) || (outs && !aligned(outs[i], size))) return FP8BSQ_EALIGN;
    if (numels[i] >= (int64_t)1 << 48) return FP8BSQ_ERANGE;
  }
  if (!aligned(norm, 4) || !aligned(workspace, 256)) return FP8BSQ_EALIGN;
  if (count > kMaxDim / 1024) return FP8BSQ_ERANGE;
  if (workspace_bytes < fp8bsq::clip_workspace_bytes(count)) return FP8BSQ_ESCRATCH;
  return launch_status(fp8bsq::launch_clip_grad_norm(grads, outs, numels, dtypes, count, max_norm, eps, norm,
                                                     workspace, (hipStream_t)hip_stream));
}

}  // extern "C"
