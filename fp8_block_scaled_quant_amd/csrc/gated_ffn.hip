// Gated feed-forward block for gfx950, forward: h = silu(g) * u with
// g = Q(x) Wg^T and u = Q(x) Wu^T on E4M3 codes and block scales.
//
// One K block of 128 gives, per 16 x 16 output tile and projection, one E4M3
// MFMA whose partial is multiplied by a_s[i, kb] * w_s[j / 128, kb] and added
// in FP32, as in the block-scaled GEMM.  Gate and up accumulators of one
// output element sit in the same lane, so silu(g) * u is formed in registers
// and only h (and, for training, g and u) reaches memory.
#include "device_cus.h"
#include "e4m3_tiles.h"
#include "ffn_launch.h"
#include "quant_common.h"

namespace fp8bsq {
namespace {

// act_quant's arithmetic with the scales laid out [K block][row], as the tile
// kernels' transfers read them.  Sixteen lanes own a 1 x 128 block, 8 values
// each; a workgroup takes 16 rows and up to four consecutive K blocks of them,
// so a row is read in 1 KB runs (bf16) and 16 rows' scales are written together.
constexpr int kQuantRows = 16, kQuantKb = 4;

template <bool kBf16, bool kUe8m0>
__global__ __launch_bounds__(256) void ffn_act_quant_kernel(const void *__restrict__ x, int64_t m, int nkb,
                                                            uint8_t *__restrict__ a, float *__restrict__ a_s,
                                                            int64_t stride) {
  const int sub = threadIdx.x & 15;
  const int64_t row = (int64_t)blockIdx.x * kQuantRows + (threadIdx.x >> 4);
  if (row >= m) return;   // whole 16-lane groups
  const int kb0 = blockIdx.y * kQuantKb, n = min(kQuantKb, nkb - kb0);
  const int64_t blk0 = row * nkb + kb0;
  u32x4 v[kQuantKb][kBf16 ? 1 : 2];
#pragma unroll
  for (int i = 0; i < kQuantKb; ++i)
    if (i < n) {
      if (kBf16) {
        v[i][0] = ((const u32x4 *)x)[(blk0 + i) * 16 + sub];
      } else {
        v[i][0] = ((const u32x4 *)x)[(blk0 + i) * 32 + 2 * sub];
        v[i][kBf16 ? 0 : 1] = ((const u32x4 *)x)[(blk0 + i) * 32 + 2 * sub + 1];
      }
    }
#pragma unroll
  for (int i = 0; i < kQuantKb; ++i) {
    if (i >= n) break;
    float s, r;
    u32x2 codes;
    if (kBf16) {
      u16x2 m2 = {0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(u16x2, v[i][0][j] & 0x7FFF7FFFu));
      block_scale_fast(row_max_u32((uint32_t)(m2.x > m2.y ? m2.x : m2.y) << 16), kUe8m0, s, r);
      codes = encode_chunk_bf16(v[i][0], s, r);
    } else {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(v[i][0][j] & 0x7FFFFFFFu, v[i][kBf16 ? 0 : 1][j] & 0x7FFFFFFFu));
      block_scale(row_max_u32(top), kUe8m0, s, r);
      codes = u32x2{encode_chunk_f32(v[i][0], s), encode_chunk_f32(v[i][kBf16 ? 0 : 1], s)};
    }
    *(u32x2 *)(a + (blk0 + i) * kBlock + 8 * sub) = codes;
    if (sub == 0) a_s[(kb0 + i) * stride + row] = s;
  }
}

TilePlan gated_plan(int64_t m, int64_t f, int64_t k) {
  return tile_plan(m, f, kBigTile / 2, (int)(k / kBlock), current_device_cus());
}

}  // namespace

FfnSpace gated_space(int64_t m, int64_t f, int64_t k) {
  const TilePlan plan = gated_plan(m, f, k);
  FfnSpace s;
  s.a = s.add(m * k);
  s.a_s = s.add((k / kBlock) * rows_padded(m) * 4);
  s.partials = s.add((int64_t)plan.partial_bytes);
  return s;
}

hipError_t launch_gated_ffn(const void *x, bool x_bf16, bool ue8m0, const uint8_t *wg, const float *wg_s,
                            const uint8_t *wu, const float *wu_s, void *h, void *g_out, void *u_out, bool out_bf16,
                            int64_t m, int64_t f, int64_t k, void *workspace, hipStream_t stream) {
  const TilePlan plan = gated_plan(m, f, k);
  const FfnSpace ws = gated_space(m, f, k);
  uint8_t *base = (uint8_t *)workspace;
  TileArgs p = {};
  p.a = base + ws.a;
  p.a_s = (const float *)(base + ws.a_s);
  p.partials = (float *)(base + ws.partials);
  p.b0 = wg;
  p.b1 = wu;
  p.b0_s = wg_s;
  p.b1_s = wu_s;
  p.out0 = h;
  p.out1 = g_out;
  p.out2 = u_out;
  p.rows_a = m;
  p.rows_b = f;
  p.lda = p.ldb = k;
  p.a_stride = rows_padded(m);
  p.nkb = (int)(k / kBlock);
  const uintptr_t mask = out_bf16 ? 7 : 15;
  p.vec = f % 4 == 0 && (((uintptr_t)h | (uintptr_t)g_out | (uintptr_t)u_out) & mask) == 0;

  const dim3 grid((unsigned)((m + kQuantRows - 1) / kQuantRows), (unsigned)((p.nkb + kQuantKb - 1) / kQuantKb));
#define FP8BSQ_QUANT(BF, UE)                                                                                   \
  hipLaunchKernelGGL((ffn_act_quant_kernel<BF, UE>), grid, dim3(256), 0, stream, x, m, p.nkb, base + ws.a,     \
                     (float *)(base + ws.a_s), p.a_stride)
  if (x_bf16) {
    if (ue8m0) FP8BSQ_QUANT(true, true); else FP8BSQ_QUANT(true, false);
  } else {
    if (ue8m0) FP8BSQ_QUANT(false, true); else FP8BSQ_QUANT(false, false);
  }
#undef FP8BSQ_QUANT
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int cus = current_device_cus();
  return ue8m0 ? launch_tiles<TileMode::kGated, true>(plan, p, out_bf16, cus, stream)
               : launch_tiles<TileMode::kGated, false>(plan, p, out_bf16, cus, stream);
}

}  // namespace fp8bsq
