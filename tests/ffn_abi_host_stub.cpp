// Host-only stand-ins for the feed-forward operators' launchers (ffn_launch.h),
// so that their C ABI layer (ffn_abi.cpp) can be built with g++ under
// AddressSanitizer and UndefinedBehaviorSanitizer and run without a GPU.
//
// Each launcher records its name and arguments and returns hipSuccess, or the
// error set by _fp8bsq_stub_fail_next.  The clip launcher reads its host arrays to
// their last entry.  The accessors start with an underscore so the export check
// of the ABI tests leaves them out.
#include <string.h>

#include "ffn_launch.h"

namespace {

struct Record {
  char name[64];
  int64_t ints[16];
  const void *ptrs[20];
  int nints, nptrs;
};

Record g_last;
int g_calls = 0;
hipError_t g_fail = hipSuccess;

struct Rec {
  explicit Rec(const char *name) {
    memset(&g_last, 0, sizeof(g_last));
    strncpy(g_last.name, name, sizeof(g_last.name) - 1);
    ++g_calls;
  }
  template <typename... T>
  Rec &i(T... v) {
    ((g_last.ints[g_last.nints++] = (int64_t)v), ...);
    return *this;
  }
  template <typename... T>
  Rec &p(T... v) {
    ((g_last.ptrs[g_last.nptrs++] = (const void *)v), ...);
    return *this;
  }
};

hipError_t result() {
  const hipError_t e = g_fail;
  g_fail = hipSuccess;
  return e;
}

fp8bsq::FfnSpace space(int64_t m, int64_t f, int64_t k) {   // a value the test can recognize
  fp8bsq::FfnSpace s;
  s.bytes = (size_t)(m * 1000000 + f * 1000 + k);
  return s;
}

}  // namespace

namespace fp8bsq {

FfnSpace gated_space(int64_t m, int64_t f, int64_t k) { return space(m, f, k); }
FfnSpace backward_space(int64_t m, int64_t f, int64_t k) { return space(m, 2 * f, k); }
size_t clip_workspace_bytes(int64_t count) { return 8192 * (size_t)(1 + count / 256); }

hipError_t launch_gated_ffn(const void *x, bool x_bf16, bool ue8m0, const uint8_t *wg, const float *wg_s,
                            const uint8_t *wu, const float *wu_s, void *h, void *g_out, void *u_out, bool out_bf16,
                            int64_t m, int64_t f, int64_t k, void *workspace, hipStream_t stream) {
  Rec("gated_ffn").i(x_bf16, ue8m0, out_bf16, m, f, k).p(x, wg, wg_s, wu, wu_s, h, g_out, u_out, workspace, stream);
  return result();
}

hipError_t launch_gated_ffn_backward(const void *dh, const void *x, const void *g, const void *u, bool in_bf16,
                                     const uint8_t *wg, const float *wg_s, const uint8_t *wu, const float *wu_s,
                                     void *dx, void *dwg, void *dwu, bool out_bf16, int64_t m, int64_t f, int64_t k,
                                     void *workspace, hipStream_t stream) {
  Rec("gated_ffn_backward").i(in_bf16, out_bf16, m, f, k)
      .p(dh, x, g, u, wg, wg_s, wu, wu_s, dx, dwg, dwu, workspace, stream);
  return result();
}

hipError_t launch_fp4_weight_quant(const void *w, bool w_bf16, int64_t n, int64_t k, uint8_t *q, uint8_t *s,
                                   hipStream_t stream) {
  Rec("fp4_weight_quant").i(w_bf16, n, k).p(w, q, s, stream);
  return result();
}

hipError_t launch_fp4_gemv(const void *x, bool x_bf16, const uint8_t *q, const uint8_t *s, const void *bias,
                           void *y, bool y_bf16, int64_t m, int64_t n, int64_t k, hipStream_t stream) {
  Rec("fp4_gemv").i(x_bf16, y_bf16, m, n, k).p(x, q, s, bias, y, stream);
  return result();
}

hipError_t launch_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *numel,
                                 const int32_t *dtypes, int64_t count, float max_norm, float eps,
                                 float *norm, void *workspace, hipStream_t stream) {
  int64_t sum = 0, bf16 = 0, addresses = 0;
  for (int64_t i = 0; i < count; ++i) {
    sum += numel[i];
    bf16 += dtypes[i];
    addresses += (int64_t)(uintptr_t)grads[i] + (outs ? (int64_t)(uintptr_t)outs[i] : 0);
  }
  Rec("clip_grad_norm").i(count, sum, bf16, addresses, (int64_t)max_norm, (int64_t)eps, outs != nullptr)
      .p(norm, workspace, stream);
  return result();
}

}  // namespace fp8bsq

extern "C" {

// Name, integer and pointer arguments of the last launcher call; returns the
// number of launcher calls so far.
__attribute__((visibility("default"))) int _fp8bsq_stub_last(char *name, int name_len, int64_t *ints,
                                                             const void **ptrs) {
  strncpy(name, g_last.name, (size_t)name_len - 1);
  name[name_len - 1] = 0;
  memcpy(ints, g_last.ints, sizeof(g_last.ints));
  memcpy(ptrs, g_last.ptrs, sizeof(g_last.ptrs));
  return g_calls;
}

// The next launcher call returns hipErrorLaunchFailure.
__attribute__((visibility("default"))) void _fp8bsq_stub_fail_next(void) { g_fail = hipErrorLaunchFailure; }

}  // extern "C"
