// 4-bit weights for gfx950: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign),
// two to a byte, and one E8M0 scale byte per 32 weights of a row.
#include "ffn_launch.h"
#include "mfma_tile.h"
#include "pow2_scale.h"

namespace fp8bsq {
namespace {

constexpr int kGroup = 32;

// ---------------------------------------------------------------------------
// Quantizer: per group, s = smallest power of two with amax <= 6 s, codes =
// E2M1(w / s), round to nearest even.  w / s is exact (a power of two), so the
// conversion instruction's rounding is the only one.  Groups of the whole
// weight form one sequence (k is a multiple of 32); four lanes own a group,
// eight weights each.
// ---------------------------------------------------------------------------
template <bool kBf16>
__global__ __launch_bounds__(256) void fp4_weight_quant_kernel(const void *__restrict__ w, int64_t ngroups,
                                                               uint32_t *__restrict__ q, uint8_t *__restrict__ s) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // eight weights
  const bool live = i < 4 * ngroups;
  float v[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) v[c] = 0.0f;
  if (live) {
    if (kBf16) {
      const u32x4 d = ((const u32x4 *)w)[i];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[2 * c] = __uint_as_float(d[c] << 16);
        v[2 * c + 1] = __uint_as_float(d[c] & 0xFFFF0000u);
      }
    } else {
      const f32x4 lo = ((const f32x4 *)w)[2 * i], hi = ((const f32x4 *)w)[2 * i + 1];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = lo[c];
        v[4 + c] = hi[c];
      }
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) top = max(top, abs_bits(v[c]));
  const uint32_t e = e2m1_scale_byte(quad_max_u32(top));
  const float inv = pow2_inverse(e);
  uint32_t codes = 0;
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[0] * inv, v[1] * inv, 1.0f, 0);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2] * inv, v[3] * inv, 1.0f, 1);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[4] * inv, v[5] * inv, 1.0f, 2);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[6] * inv, v[7] * inv, 1.0f, 3);
  if (live) {
    q[i] = codes;
    if ((i & 3) == 0) s[i >> 2] = (uint8_t)e;
  }
}

// ---------------------------------------------------------------------------
// y = x W^T.  An E2M1 code times its power-of-two scale is exact in bf16, and
// one instruction turns two codes and the scale into two bf16, so the group
// scales cost nothing in the product and one FP32 accumulator runs through K.
//
// MFMA 16x16x32 with the weights as the 16-row operand and up to 16 rows of x
// as columns.  The order of K inside the operands is free as long as both
// agree: lane l takes weight row l % 16 and the whole group 4 step + l / 16 --
// 16 bytes of codes and one scale -- and feeds it to four MFMAs, eight codes
// each; x's lane reads the same eight k.  The four waves of a workgroup split
// the steps of 128 k and add their sums in LDS.
//
// fp32 x is split exactly into three bf16 (3 x 8 significand bits), one MFMA
// each.
// ---------------------------------------------------------------------------
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ bf16x8 fp4_to_bf16(uint32_t codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) {   // two fp32's upper 16 bits
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

constexpr int kGemvWaves = 4;

template <bool kBf16X, bool kBf16Out>
__global__ __launch_bounds__(64 * kGemvWaves) void fp4_gemv_kernel(
    const void *__restrict__ x, const uint8_t *__restrict__ q, const uint8_t *__restrict__ s,
    const void *__restrict__ bias, void *__restrict__ y, int64_t m, int64_t n, int64_t k) {
  __shared__ f32x4 sums[kGemvWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = lane & 15, lq = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16;
  const int ng = (int)(k / kGroup);
  const int64_t row = min(n0 + lr, n - 1);
  const uint8_t *qrow = q + row * (k / 2), *srow = s + row * ng;
  const bool xlive = m0 + lr < m;
  const int64_t xrow = (m0 + (xlive ? lr : 0)) * k;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int step = wave; 4 * step < ng; step += kGemvWaves) {
    const int grp = 4 * step + lq;
    const bool live = grp < ng;
    u32x4 codes = {0, 0, 0, 0};
    float scale = 1.0f;
    if (live) {
      codes = *(const u32x4 *)(qrow + (int64_t)grp * 16);
      scale = pow2_scale(srow[grp]);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const bf16x8 w = fp4_to_bf16(codes[t], scale);
      const int64_t at = xrow + (int64_t)grp * kGroup + 8 * t;
      if (kBf16X) {
        u32x4 xv = {0, 0, 0, 0};
        if (live && xlive) xv = *(const u32x4 *)((const uint16_t *)x + at);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, xv), acc, 0, 0, 0);
      } else {
        f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
        if (live && xlive) {
          lo = *(const f32x4 *)((const float *)x + at);
          hi = *(const f32x4 *)((const float *)x + at + 4);
        }
        float r[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          u32x4 p;
#pragma unroll
          for (int c = 0; c < 4; ++c) p[c] = high_halves(__float_as_uint(r[2 * c]), __float_as_uint(r[2 * c + 1]));
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, p), acc, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < 8; ++c) r[c] -= __uint_as_float(__float_as_uint(r[c]) & 0xFFFF0000u);
        }
      }
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave != 0 || !xlive) return;
#pragma unroll
  for (int w = 1; w < kGemvWaves; ++w) acc += sums[w][lane];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t col = n0 + 4 * lq + e;
    if (col < n) store_out(y, kBf16Out, (m0 + lr) * n + col, acc[e] + bias_at(bias, kBf16Out, col));
  }
}

}  // namespace

hipError_t launch_fp4_weight_quant(const void *w, bool w_bf16, int64_t n, int64_t k, uint8_t *q, uint8_t *s,
                                   hipStream_t stream) {
  const int64_t ngroups = n * (k / kGroup);
  const dim3 grid((unsigned)((4 * ngroups + 255) / 256)), block(256);
  if (w_bf16)
    hipLaunchKernelGGL(fp4_weight_quant_kernel<true>, grid, block, 0, stream, w, ngroups, (uint32_t *)q, s);
  else
    hipLaunchKernelGGL(fp4_weight_quant_kernel<false>, grid, block, 0, stream, w, ngroups, (uint32_t *)q, s);
  return hipGetLastError();
}

hipError_t launch_fp4_gemv(const void *x, bool x_bf16, const uint8_t *q, const uint8_t *s, const void *bias,
                           void *y, bool y_bf16, int64_t m, int64_t n, int64_t k, hipStream_t stream) {
  const dim3 grid((unsigned)((n + 15) / 16), (unsigned)((m + 15) / 16)), block(64 * kGemvWaves);
#define FP8BSQ_GEMV(XB, YB) \
  hipLaunchKernelGGL((fp4_gemv_kernel<XB, YB>), grid, block, 0, stream, x, q, s, bias, y, m, n, k)
  if (x_bf16) {
    if (y_bf16) FP8BSQ_GEMV(true, true); else FP8BSQ_GEMV(true, false);
  } else {
    if (y_bf16) FP8BSQ_GEMV(false, true); else FP8BSQ_GEMV(false, false);
  }
#undef FP8BSQ_GEMV
  return hipGetLastError();
}

}  // namespace fp8bsq
