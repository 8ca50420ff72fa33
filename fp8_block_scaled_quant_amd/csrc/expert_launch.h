// Internal launchers of the expert operators.  Arguments are already validated by
// the C ABI layer (ffn_abi.cpp); each returns the HIP error of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8bsq {

constexpr int64_t kMaxExperts = 1024;   // tables of all experts are kept in LDS

// experts: n int32, or (wide) int64 numbers.
size_t expert_sort_bytes(int64_t n, int64_t num_experts);
hipError_t launch_expert_sort(const void *experts, bool wide, int64_t n, int64_t num_experts, int32_t *offsets,
                              int32_t *rows, int32_t *choices, void *workspace, hipStream_t stream);

// y [tokens * top_k, h] in x's type.
hipError_t launch_expert_dispatch(const void *x, bool bf16, const int32_t *rows, int64_t tokens, int64_t top_k,
                                  int64_t h, void *y, hipStream_t stream);

// y codes, s scales [tokens * top_k, h / 128].
hipError_t launch_expert_dispatch_quant(const void *x, bool bf16, bool ue8m0, const int32_t *rows, int64_t tokens,
                                        int64_t top_k, int64_t h, uint8_t *y, float *s, hipStream_t stream);

// weights may be null: ones.
hipError_t launch_expert_combine(const void *y, bool bf16, const int32_t *rows, const void *weights, bool w_bf16,
                                 int64_t tokens, int64_t top_k, int64_t h, void *out, hipStream_t stream);

// dy or dweights may be null; y is read for dweights only.
hipError_t launch_expert_combine_backward(const void *dout, const void *y, bool bf16, const int32_t *rows,
                                          const void *weights, bool w_bf16, int64_t tokens, int64_t top_k, int64_t h,
                                          void *dy, void *dweights, hipStream_t stream);

// out [rows, f]: a times each expert's w0^T, or with w1 silu of that times a w1^T.
hipError_t launch_expert_product(const uint8_t *a, const float *a_s, const int32_t *offsets, const uint8_t *w0,
                                 const float *w0_s, const uint8_t *w1, const float *w1_s, void *out, bool out_bf16,
                                 int64_t rows, int64_t experts, int64_t f, int64_t k, hipStream_t stream);

}  // namespace fp8bsq
