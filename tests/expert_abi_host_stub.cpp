// Host-only stand-ins for the expert operators' launchers (expert_launch.h), beside
// those of ffn_abi_host_stub.cpp, whose record they share.
#include "ffn_abi_host_stub.cpp"

#include "expert_launch.h"

namespace fp8bsq {

size_t expert_sort_bytes(int64_t n, int64_t num_experts) { return n > 100 ? (size_t)(n * 1000 + num_experts) : 0; }

hipError_t launch_expert_sort(const void *experts, bool wide, int64_t n, int64_t num_experts, int32_t *offsets,
                              int32_t *rows, int32_t *choices, void *workspace, hipStream_t stream) {
  Rec("expert_sort").i(wide, n, num_experts).p(experts, offsets, rows, choices, workspace, stream);
  return result();
}

hipError_t launch_expert_dispatch(const void *x, bool bf16, const int32_t *rows, int64_t tokens, int64_t top_k,
                                  int64_t h, void *y, hipStream_t stream) {
  Rec("expert_dispatch").i(bf16, tokens, top_k, h).p(x, rows, y, stream);
  return result();
}

hipError_t launch_expert_dispatch_quant(const void *x, bool bf16, bool ue8m0, const int32_t *rows, int64_t tokens,
                                        int64_t top_k, int64_t h, uint8_t *y, float *s, hipStream_t stream) {
  Rec("expert_dispatch_quant").i(bf16, ue8m0, tokens, top_k, h).p(x, rows, y, s, stream);
  return result();
}

hipError_t launch_expert_combine(const void *y, bool bf16, const int32_t *rows, const void *weights, bool w_bf16,
                                 int64_t tokens, int64_t top_k, int64_t h, void *out, hipStream_t stream) {
  Rec("expert_combine").i(bf16, w_bf16, tokens, top_k, h).p(y, rows, weights, out, stream);
  return result();
}

hipError_t launch_expert_combine_backward(const void *dout, const void *y, bool bf16, const int32_t *rows,
                                          const void *weights, bool w_bf16, int64_t tokens, int64_t top_k, int64_t h,
                                          void *dy, void *dweights, hipStream_t stream) {
  Rec("expert_combine_backward").i(bf16, w_bf16, tokens, top_k, h).p(dout, y, rows, weights, dy, dweights, stream);
  return result();
}

hipError_t launch_expert_product(const uint8_t *a, const float *a_s, const int32_t *offsets, const uint8_t *w0,
                                 const float *w0_s, const uint8_t *w1, const float *w1_s, void *out, bool out_bf16,
                                 int64_t rows, int64_t experts, int64_t f, int64_t k, hipStream_t stream) {
  Rec("expert_product").i(out_bf16, rows, experts, f, k).p(a, a_s, offsets, w0, w0_s, w1, w1_s, out, stream);
  return result();
}

}  // namespace fp8bsq
