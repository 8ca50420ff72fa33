// Gated feed-forward block for gfx950, forward: h = silu(g) * u with
// g = Q(x) Wg^T and u = Q(x) Wu^T on E4M3 codes and block scales.
//
// One K block of 128 gives, per 16 x 16 output tile and projection, one E4M3
// MFMA whose partial is multiplied by a_s[i, kb] * w_s[j / 128, kb] and added
// in FP32, as in the block-scaled GEMM.  Gate and up accumulators of one
// output element sit in the same lane, so silu(g) * u is formed in registers
// and only h (and, for training, g and u) reaches memory.
#include "ffn_launch.h"
#include "mfma_tile.h"

namespace fp8bsq {
namespace {

// silu(g) * u; the exponential overflows to infinity for g below -88, where
// the sigmoid is 0 to fp32's precision.
__device__ __forceinline__ float gated(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// 256 threads = 2 x 2 waves, each wave 32 x 32 outputs of both projections,
// fragments read straight from global memory.  The 64-column workgroup tile
// never straddles a 128-row weight block.
template <bool kBf16Out>
__global__ __launch_bounds__(256) void gated_simple_kernel(
    const uint8_t *__restrict__ a, const float *__restrict__ a_s, const uint8_t *__restrict__ wg,
    const float *__restrict__ wg_s, const uint8_t *__restrict__ wu, const float *__restrict__ wu_s,
    void *__restrict__ h, void *__restrict__ g_out, void *__restrict__ u_out, int64_t m, int64_t f, int64_t k) {
  const int nkb = (int)(k / kBlock);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t m0 = (int64_t)blockIdx.y * 64 + (wave >> 1) * 32;
  const int64_t n0 = (int64_t)blockIdx.x * 64 + (wave & 1) * 32;
  const int64_t b_row = ((int64_t)blockIdx.x * 64) / kBlock;
  const int lr = lane & 15, lk = (lane >> 4) * 32, lq = (lane >> 4) * 4;

  f32x4 acc[2][2][2];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[w][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const i32x8 zero8 = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int kb = 0; kb < nkb; ++kb) {
    i32x8 af[2], bfr[2][2];
    float sa[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = m0 + 16 * i + lr;
      af[i] = row < m ? load_frag(a + row * k + (int64_t)kb * kBlock + lk) : zero8;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t orow = m0 + 16 * i + lq + r;
        sa[i][r] = orow < m ? a_s[orow * nkb + kb] : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t col = n0 + 16 * j + lr;
      const int64_t off = col * k + (int64_t)kb * kBlock + lk;
      bfr[0][j] = col < f ? load_frag(wg + off) : zero8;
      bfr[1][j] = col < f ? load_frag(wu + off) : zero8;
    }
    const float sb[2] = {wg_s[b_row * nkb + kb], wu_s[b_row * nkb + kb]};
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f32x4 p = mfma_e4m3_16x16x128(af[i], bfr[w][j], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[w][i][j][r] = __builtin_fmaf(p[r], sa[i][r] * sb[w], acc[w][i][j][r]);
        }
  }

#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t col = n0 + 16 * j + lr;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t row = m0 + 16 * i + lq + r;
        if (row < m && col < f) {
          const float g = acc[0][i][j][r], u = acc[1][i][j][r];
          store_out(h, kBf16Out, row * f + col, gated(g, u));
          if (g_out) {
            store_out(g_out, kBf16Out, row * f + col, g);
            store_out(u_out, kBf16Out, row * f + col, u);
          }
        }
      }
    }
}

}  // namespace

hipError_t launch_gated_gemm(const uint8_t *a, const float *a_s, const uint8_t *wg, const float *wg_s,
                             const uint8_t *wu, const float *wu_s, void *h, void *g_out, void *u_out,
                             bool out_bf16, int64_t m, int64_t f, int64_t k, hipStream_t stream) {
  const dim3 grid((unsigned)((f + 63) / 64), (unsigned)((m + 63) / 64)), block(256);
  if (out_bf16)
    hipLaunchKernelGGL(gated_simple_kernel<true>, grid, block, 0, stream, a, a_s, wg, wg_s, wu, wu_s, h, g_out,
                       u_out, m, f, k);
  else
    hipLaunchKernelGGL(gated_simple_kernel<false>, grid, block, 0, stream, a, a_s, wg, wg_s, wu, wu_s, h, g_out,
                       u_out, m, f, k);
  return hipGetLastError();
}

}  // namespace fp8bsq
