// Gated feed-forward block for gfx950, backward pass.
//
// With s = sigmoid(g), silu(g) = g s and silu'(g) = s (1 + g (1 - s)):
//     dg = dh u silu'(g),   du = dh silu(g)
//     dx  = Q(dg) Wg + Q(du) Wu           (contraction over the 2 f features)
//     dWg = Q(dg)^T Q(x),  dWu = Q(du)^T Q(x)   (contraction over the tokens)
// Q rounds to E4M3 with one power-of-two scale per 128 values along the
// product's contraction axis (gradients take a power of two so that their
// scale goes into the MX-scaled MFMA; unlike act_quant there is no floor of
// 1e-4 on amax, which gradients lie below).  128 x 128 weight blocks stay
// 128 x 128 blocks when transposed, so Wg and Wu enter dx exactly.
//
// The products are the tile kernels' kInput and kWeight modes; the quantizers
// below write dg and du (and x) in the layouts these read, straight from dh, g
// and u: dg and du exist in registers only.
#include "device_cus.h"
#include "e4m3_tiles.h"
#include "ffn_launch.h"
#include "pow2_scale.h"
#include "quant_common.h"

namespace fp8bsq {
namespace {

// ---------------------------------------------------------------------------
// Quantizers.  A workgroup of 256 threads owns a 128 x 128 tile; lane l of
// wave w holds rows 8 (4 w + l / 16) .. + 7 and columns 8 (l % 16) .. + 7, so
// loads cover 256-byte row segments, a row's amax is a DPP reduction over 16
// lanes, and a column's eight rows pack into one 8-byte piece of the
// transposed tile, which goes through LDS to whole-line stores.
// ---------------------------------------------------------------------------

template <bool kBf16>
__device__ __forceinline__ void load8(const void *p, int64_t idx, bool live, float (&v)[8]) {
  if (!live) {
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = 0.0f;
  } else if (kBf16) {
    const u32x4 w = *(const u32x4 *)((const uint16_t *)p + idx);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[2 * c] = __uint_as_float(w[c] << 16);
      v[2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
    }
  } else {
    const f32x4 lo = *(const f32x4 *)((const float *)p + idx), hi = *(const f32x4 *)((const float *)p + idx + 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[c] = lo[c];
      v[4 + c] = hi[c];
    }
  }
}

// E4M3 codes of four values already divided by their scale.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return cvt_pk_e4m3<true>(c, d, cvt_pk_e4m3<false>(a, b, 0u));
}

struct TokenTile {
  uint8_t codes[128 * 128];      // [column][token], 8-byte pieces swizzled by the column
  uint32_t colmax[4][128];       // per wave
};

// Quantize a tile's values v [8 rows][8 columns] along the rows (tokens) and
// write it transposed: codes to out [row0 + column][mpad] at token m0, the
// scales to scales[row0 + column].  Every thread of the workgroup takes part.
__device__ __forceinline__ void store_tokens(const float (&v)[8][8], TokenTile &sm, uint8_t *__restrict__ out,
                                             float *__restrict__ scales, int64_t row0, int64_t m0, int64_t mpad) {
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63, grp = lane >> 4, sub = lane & 15;
  uint32_t top[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    top[c] = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) top[c] = max(top[c], abs_bits(v[r][c]));
    top[c] = max(top[c], (uint32_t)__shfl_xor((int)top[c], 16));
    top[c] = max(top[c], (uint32_t)__shfl_xor((int)top[c], 32));
  }
  if (grp == 0)
#pragma unroll
    for (int c = 0; c < 8; ++c) sm.colmax[wave][8 * sub + c] = top[c];
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int col = 8 * sub + c;
    const uint32_t e = e4m3_scale_byte(max(max(sm.colmax[0][col], sm.colmax[1][col]),
                                           max(sm.colmax[2][col], sm.colmax[3][col])));
    const float inv = pow2_inverse(e);
    u32x2 q;
    q.x = codes4(v[0][c] * inv, v[1][c] * inv, v[2][c] * inv, v[3][c] * inv);
    q.y = codes4(v[4][c] * inv, v[5][c] * inv, v[6][c] * inv, v[7][c] * inv);
    *(u32x2 *)&sm.codes[col * 128 + (((4 * wave + grp) ^ sub) << 3)] = q;
    if (wave == 0 && grp == 0) scales[row0 + col] = pow2_scale(e);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int idx = i * 256 + t, col = idx >> 3, j = idx & 7, s = (col >> 3) & 15;
    const u32x2 lo = *(const u32x2 *)&sm.codes[col * 128 + (((2 * j) ^ s) << 3)];
    const u32x2 hi = *(const u32x2 *)&sm.codes[col * 128 + (((2 * j + 1) ^ s) << 3)];
    *(u32x4 *)(out + (row0 + col) * mpad + m0 + 16 * j) = u32x4{lo.x, lo.y, hi.x, hi.y};
  }
  __syncthreads();   // the tile may be reused
}

// Quantize each row's 128 columns: codes to out + row * ld, scale to scales[row].
__device__ __forceinline__ void store_rows(const float (&v)[8][8], uint8_t *__restrict__ out, int64_t ld,
                                           float *__restrict__ scales, int64_t row0, int64_t m) {
  const int sub = threadIdx.x & 15;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) top = max(top, abs_bits(v[r][c]));
    const uint32_t e = e4m3_scale_byte(row_max_u32(top));
    const float inv = pow2_inverse(e);
    if (row0 + r < m) {
      u32x2 q;
      q.x = codes4(v[r][0] * inv, v[r][1] * inv, v[r][2] * inv, v[r][3] * inv);
      q.y = codes4(v[r][4] * inv, v[r][5] * inv, v[r][6] * inv, v[r][7] * inv);
      *(u32x2 *)(out + (row0 + r) * ld + 8 * sub) = q;
      if (sub == 0) scales[row0 + r] = pow2_scale(e);
    }
  }
}

template <bool kBf16>
__global__ __launch_bounds__(256) void ffn_grad_quant_kernel(
    const void *__restrict__ dh, const void *__restrict__ g, const void *__restrict__ u, int64_t m, int64_t f,
    int64_t mpad, uint8_t *__restrict__ rq, float *__restrict__ rs, int64_t rs_stride, uint8_t *__restrict__ cq,
    float *__restrict__ cs, int64_t cs_stride) {
  __shared__ TokenTile sm;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t f0 = (int64_t)blockIdx.x * kBlock, m0 = (int64_t)blockIdx.y * kBlock;
  const int64_t row0 = m0 + 8 * (4 * wave + (lane >> 4)), col0 = f0 + 8 * (lane & 15);
  float dg[8][8], du[8][8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const bool live = row0 + r < m;
    const int64_t idx = (row0 + r) * f + col0;
    float hv[8], gv[8], uv[8];
    load8<kBf16>(dh, idx, live, hv);
    load8<kBf16>(g, idx, live, gv);
    load8<kBf16>(u, idx, live, uv);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float s = 1.0f / (1.0f + __expf(-gv[c]));
      du[r][c] = hv[c] * (gv[c] * s);
      dg[r][c] = hv[c] * uv[c] * (s * __builtin_fmaf(gv[c], 1.0f - s, 1.0f));
    }
  }
  if (rq) {
    const int64_t nfb = f / kBlock;
    float *s = rs + blockIdx.x * rs_stride;
    store_rows(dg, rq + f0, 2 * f, s, row0, m);
    store_rows(du, rq + f + f0, 2 * f, s + nfb * rs_stride, row0, m);
  }
  if (cq) {
    float *s = cs + blockIdx.y * cs_stride;
    store_tokens(dg, sm, cq, s, f0, m0, mpad);
    store_tokens(du, sm, cq, s, f + f0, m0, mpad);
  }
}

template <bool kBf16>
__global__ __launch_bounds__(256) void token_quant_kernel(const void *__restrict__ x, int64_t m, int64_t k,
                                                          int64_t mpad, uint8_t *__restrict__ cq,
                                                          float *__restrict__ cs) {
  __shared__ TokenTile sm;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k0 = (int64_t)blockIdx.x * kBlock, m0 = (int64_t)blockIdx.y * kBlock;
  const int64_t row0 = m0 + 8 * (4 * wave + (lane >> 4)), col0 = k0 + 8 * (lane & 15);
  float v[8][8];
#pragma unroll
  for (int r = 0; r < 8; ++r) load8<kBf16>(x, (row0 + r) * k + col0, row0 + r < m, v[r]);
  store_tokens(v, sm, cq, cs + blockIdx.y * k, k0, m0, mpad);
}

TilePlan input_plan(int64_t m, int64_t f, int64_t k) {
  return tile_plan(m, k, kBigTile, (int)(2 * f / kBlock), current_device_cus());
}
TilePlan weight_plan(int64_t m, int64_t f, int64_t k) {
  return tile_plan(2 * f, k, kBigTile, (int)(tokens_padded(m) / kBlock), current_device_cus());
}

}  // namespace

FfnSpace backward_space(int64_t m, int64_t f, int64_t k) {
  const TilePlan in = input_plan(m, f, k), wt = weight_plan(m, f, k);
  const int64_t mpad = tokens_padded(m);
  FfnSpace s;
  s.a = s.add(m * 2 * f);
  s.a_s = s.add((2 * f / kBlock) * rows_padded(m) * 4);
  s.cq = s.add(2 * f * mpad);
  s.cs = s.add((mpad / kBlock) * rows_padded(2 * f) * 4);
  s.xq = s.add(k * mpad);
  s.xs = s.add((mpad / kBlock) * k * 4);
  // one after the other on the stream, the two products share the partials
  s.partials = s.add((int64_t)(in.partial_bytes > wt.partial_bytes ? in.partial_bytes : wt.partial_bytes));
  return s;
}

hipError_t launch_gated_ffn_backward(const void *dh, const void *x, const void *g, const void *u, bool in_bf16,
                                     const uint8_t *wg, const float *wg_s, const uint8_t *wu, const float *wu_s,
                                     void *dx, void *dwg, void *dwu, bool out_bf16, int64_t m, int64_t f, int64_t k,
                                     void *workspace, hipStream_t stream) {
  const TilePlan in = input_plan(m, f, k), wt = weight_plan(m, f, k);
  const FfnSpace ws = backward_space(m, f, k);
  const int64_t mpad = tokens_padded(m);
  const int cus = current_device_cus();
  uint8_t *base = (uint8_t *)workspace;
  float *partials = (float *)(base + ws.partials);
  hipError_t e = hipSuccess;
  if (m > 0) {
    const dim3 grid((unsigned)(f / kBlock), (unsigned)(mpad / kBlock));
#define FP8BSQ_GRAD_QUANT(BF)                                                                                   \
  hipLaunchKernelGGL(ffn_grad_quant_kernel<BF>, grid, dim3(256), 0, stream, dh, g, u, m, f, mpad,               \
                     dx ? base + ws.a : nullptr, (float *)(base + ws.a_s), rows_padded(m),                      \
                     dwg ? base + ws.cq : nullptr, (float *)(base + ws.cs), rows_padded(2 * f))
    if (in_bf16) FP8BSQ_GRAD_QUANT(true); else FP8BSQ_GRAD_QUANT(false);
#undef FP8BSQ_GRAD_QUANT
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (dwg) {
      const dim3 xgrid((unsigned)(k / kBlock), (unsigned)(mpad / kBlock));
      if (in_bf16)
        hipLaunchKernelGGL(token_quant_kernel<true>, xgrid, dim3(256), 0, stream, x, m, k, mpad, base + ws.xq,
                           (float *)(base + ws.xs));
      else
        hipLaunchKernelGGL(token_quant_kernel<false>, xgrid, dim3(256), 0, stream, x, m, k, mpad, base + ws.xq,
                           (float *)(base + ws.xs));
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (dx && m > 0) {
    TileArgs p = {};
    p.a = base + ws.a;
    p.a_s = (const float *)(base + ws.a_s);
    p.b0 = wg;
    p.b1 = wu;
    p.b0_s = wg_s;
    p.b1_s = wu_s;
    p.out0 = dx;
    p.partials = partials;
    p.rows_a = m;
    p.rows_b = k;
    p.lda = 2 * f;
    p.ldb = k;
    p.a_stride = rows_padded(m);
    p.nkb = (int)(2 * f / kBlock);
    p.half = (int)(f / kBlock);
    e = launch_tiles<TileMode::kInput, true>(in, p, out_bf16, cus, stream);
    if (e != hipSuccess) return e;
  }
  if (dwg) {
    TileArgs p = {};
    p.a = base + ws.cq;
    p.a_s = (const float *)(base + ws.cs);
    p.b0 = base + ws.xq;
    p.b0_s = (const float *)(base + ws.xs);
    p.out0 = dwg;
    p.out1 = dwu;
    p.partials = partials;
    p.rows_a = 2 * f;
    p.rows_b = k;
    p.lda = p.ldb = mpad;
    p.a_stride = rows_padded(2 * f);
    p.b_stride = k;
    p.nkb = (int)(mpad / kBlock);
    e = launch_tiles<TileMode::kWeight, true>(wt, p, out_bf16, cus, stream);
  }
  return e;
}

}  // namespace fp8bsq
