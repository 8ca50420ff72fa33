// Products of the experts' rows with their own block-scaled E4M3 weights, for
// gfx950: out[r] = a[r] W[e]^T for offsets[e] <= r < offsets[e + 1], or with two
// weights silu(a[r] Wg[e]^T) * (a[r] Wu[e]^T).  Each 128-wide K block's partial is
// multiplied by a_s[r, kb] * w_s[e, j / 128, kb] and added in FP32.
#include "e4m3_tiles.h"
#include "expert_launch.h"

namespace fp8bsq {
namespace {

struct ProductArgs {
  const uint8_t *a;
  const float *a_s;
  const int32_t *offsets;
  const uint8_t *w0, *w1;   // [expert][f][k]; w1 null where there is one weight
  const float *w0_s, *w1_s;
  void *out;
  int64_t rows, f, k;
  int experts, nkb;
  bool out_bf16;
};

// A wave per 16 features; a workgroup's four waves go through the expert's rows
// 16 at a time.  The last expert's workgroups clear the rows behind.
template <bool kGated>
__global__ __launch_bounds__(256) void product_simple_kernel(const ProductArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, fr = lane & 15, fq = lane >> 4;
  const int e = blockIdx.y;
  const int64_t f0 = ((int64_t)blockIdx.x * 4 + wave) * 16;
  if (f0 >= p.f) return;
  const int64_t feature = min(f0 + fr, p.f - 1);
  const int64_t begin = min(max((int64_t)p.offsets[e], (int64_t)0), p.rows);
  const int64_t end = min(max((int64_t)p.offsets[e + 1], begin), p.rows);
  const int64_t grid_rows = (p.f + kBlock - 1) / kBlock;
  const float *s0 = p.w0_s + ((int64_t)e * grid_rows + f0 / kBlock) * p.nkb;
  const float *s1 = kGated ? p.w1_s + ((int64_t)e * grid_rows + f0 / kBlock) * p.nkb : nullptr;
  for (int64_t r0 = begin; r0 < end; r0 += 16) {
    const int64_t row = min(r0 + fr, end - 1);
    f32x4 g = {0.f, 0.f, 0.f, 0.f}, u = g;
    for (int kb = 0; kb < p.nkb; ++kb) {
      const i32x8 a = load_frag(p.a + row * p.k + kb * kBlock + 32 * fq);
      const float sa = p.a_s[row * p.nkb + kb];
      const int64_t at = ((int64_t)e * p.f + feature) * p.k + kb * kBlock + 32 * fq;
      const f32x4 v0 = mfma_e4m3_16x16x128(load_frag(p.w0 + at), a, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = __builtin_fmaf(v0[i], sa * s0[kb], g[i]);
      if (kGated) {
        const f32x4 v1 = mfma_e4m3_16x16x128(load_frag(p.w1 + at), a, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __builtin_fmaf(v1[i], sa * s1[kb], u[i]);
      }
    }
    if (r0 + fr < end) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t col = f0 + 4 * fq + i;
        if (col < p.f) store_out(p.out, p.out_bf16, row * p.f + col, kGated ? gated(g[i], u[i]) : g[i]);
      }
    }
  }
  if (e == p.experts - 1)
    for (int64_t row = end + fr; row < p.rows; row += 16)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (f0 + 4 * fq + i < p.f) store_out(p.out, p.out_bf16, row * p.f + f0 + 4 * fq + i, 0.0f);
}

}  // namespace

hipError_t launch_expert_product(const uint8_t *a, const float *a_s, const int32_t *offsets, const uint8_t *w0,
                                 const float *w0_s, const uint8_t *w1, const float *w1_s, void *out, bool out_bf16,
                                 int64_t rows, int64_t experts, int64_t f, int64_t k, hipStream_t stream) {
  const ProductArgs p = {a, a_s, offsets, w0, w1, w0_s, w1_s, out, rows, f, k, (int)experts, (int)(k / kBlock), out_bf16};
  const dim3 grid((unsigned)((f + 63) / 64), (unsigned)experts), block(256);
  if (w1)
    hipLaunchKernelGGL(product_simple_kernel<true>, grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL(product_simple_kernel<false>, grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace fp8bsq
