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
// dx is the block-scaled GEMM of [dg | du] (m x 2 f) and [Wg^T | Wu^T]
// (k x 2 f).  dW is a product with power-of-two scales on both operands: both
// go into the MFMA, which then accumulates over the whole contraction.
#include "ffn_launch.h"
#include "mfma_tile.h"
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
// exponent bytes to exps (byte mb % 4 of word [mb / 4][row]).  Every thread of
// the workgroup takes part.
__device__ __forceinline__ void store_tokens(const float (&v)[8][8], TokenTile &sm, uint8_t *__restrict__ out,
                                             uint8_t *__restrict__ exps, int64_t row0, int64_t rows,
                                             int64_t m0, int64_t mpad) {
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
    if (wave == 0 && grp == 0) {
      const int64_t mb = m0 / kBlock;
      exps[((mb >> 2) * rows + row0 + col) * 4 + (mb & 3)] = (uint8_t)e;
    }
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

// Quantize each row's 128 columns: codes to out + row * ld, scale to scales.
__device__ __forceinline__ void store_rows(const float (&v)[8][8], uint8_t *__restrict__ out, int64_t ld,
                                           float *__restrict__ scales, int64_t lds, int64_t row0, int64_t m) {
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
      if (sub == 0) scales[(row0 + r) * lds] = pow2_scale(e);
    }
  }
}

template <bool kBf16>
__global__ __launch_bounds__(256) void ffn_grad_quant_kernel(
    const void *__restrict__ dh, const void *__restrict__ g, const void *__restrict__ u, int64_t m, int64_t f,
    int64_t mpad, uint8_t *__restrict__ rq, float *__restrict__ rs, uint8_t *__restrict__ cq,
    uint8_t *__restrict__ ce) {
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
    store_rows(dg, rq + f0, 2 * f, rs + f0 / kBlock, 2 * nfb, row0, m);
    store_rows(du, rq + f + f0, 2 * f, rs + nfb + f0 / kBlock, 2 * nfb, row0, m);
  }
  if (cq) {
    store_tokens(dg, sm, cq, ce, f0, 2 * f, m0, mpad);
    store_tokens(du, sm, cq, ce, f + f0, 2 * f, m0, mpad);
  }
}

template <bool kBf16>
__global__ __launch_bounds__(256) void token_quant_kernel(const void *__restrict__ x, int64_t m, int64_t k,
                                                          int64_t mpad, uint8_t *__restrict__ cq,
                                                          uint8_t *__restrict__ ce) {
  __shared__ TokenTile sm;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k0 = (int64_t)blockIdx.x * kBlock, m0 = (int64_t)blockIdx.y * kBlock;
  const int64_t row0 = m0 + 8 * (4 * wave + (lane >> 4)), col0 = k0 + 8 * (lane & 15);
  float v[8][8];
#pragma unroll
  for (int r = 0; r < 8; ++r) load8<kBf16>(x, (row0 + r) * k + col0, row0 + r < m, v[r]);
  store_tokens(v, sm, cq, ce, k0, k, m0, mpad);
}

// ---------------------------------------------------------------------------
// Transposed weight codes: a workgroup turns one 128 x 128 block, each thread
// an 8 x 8 patch by byte permutes, through LDS to whole-line stores.
// ---------------------------------------------------------------------------

// Four rows of four bytes -> four columns of four bytes.
__device__ __forceinline__ void transpose4x4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&o)[4]) {
  const uint32_t t0 = __builtin_amdgcn_perm(b, a, 0x05010400u), t1 = __builtin_amdgcn_perm(d, c, 0x05010400u);
  const uint32_t t2 = __builtin_amdgcn_perm(b, a, 0x07030602u), t3 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  o[0] = __builtin_amdgcn_perm(t1, t0, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(t1, t0, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(t3, t2, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(t3, t2, 0x07060302u);
}

__global__ __launch_bounds__(256) void weights_transpose_kernel(
    const uint8_t *__restrict__ wg, const float *__restrict__ wg_s, const uint8_t *__restrict__ wu,
    const float *__restrict__ wu_s, int64_t f, int64_t k, uint8_t *__restrict__ wt, float *__restrict__ wt_s) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * 128];
  const int t = threadIdx.x, grp = t >> 4, sub = t & 15;
  const int64_t k0 = (int64_t)blockIdx.x * kBlock, f0 = (int64_t)blockIdx.y * kBlock;
  const bool up = blockIdx.z != 0;
  const uint8_t *w = up ? wu : wg;
  u32x2 row[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) row[r] = *(const u32x2 *)(w + (f0 + 8 * grp + r) * k + k0 + 8 * sub);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t lo[4], hi[4];
    transpose4x4(row[0][half], row[1][half], row[2][half], row[3][half], lo);
    transpose4x4(row[4][half], row[5][half], row[6][half], row[7][half], hi);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *(u32x2 *)&tile[(8 * sub + 4 * half + c) * 128 + ((grp ^ sub) << 3)] = u32x2{lo[c], hi[c]};
  }
  __syncthreads();
  const int64_t at = (up ? f : 0) + f0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int idx = i * 256 + t, col = idx >> 3, j = idx & 7, s = (col >> 3) & 15;
    const u32x2 lo = *(const u32x2 *)&tile[col * 128 + (((2 * j) ^ s) << 3)];
    const u32x2 hi = *(const u32x2 *)&tile[col * 128 + (((2 * j + 1) ^ s) << 3)];
    *(u32x4 *)(wt + (k0 + col) * (2 * f) + at + 16 * j) = u32x4{lo.x, lo.y, hi.x, hi.y};
  }
  if (t == 0)
    wt_s[blockIdx.x * (2 * f / kBlock) + at / kBlock] = (up ? wu_s : wg_s)[blockIdx.y * (k / kBlock) + blockIdx.x];
}

// ---------------------------------------------------------------------------
// dW: 256 threads = 2 x 2 waves, each wave a 32 x 32 output tile, fragments
// straight from global memory; f and k are multiples of 128, so no edges.
// ---------------------------------------------------------------------------
template <bool kBf16Out>
__global__ __launch_bounds__(256) void weight_grad_simple_kernel(
    const uint8_t *__restrict__ dq, const uint32_t *__restrict__ de, const uint8_t *__restrict__ xq,
    const uint32_t *__restrict__ xe, void *__restrict__ dwg, void *__restrict__ dwu, int64_t mpad, int64_t f,
    int64_t k) {
  const int nmb = (int)(mpad / kBlock);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t r0 = (int64_t)blockIdx.y * 64 + (wave >> 1) * 32, c0 = (int64_t)blockIdx.x * 64 + (wave & 1) * 32;
  const int lr = lane & 15, lk = (lane >> 4) * 32, lq = (lane >> 4) * 4;
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int mb = 0; mb < nmb; ++mb) {
    i32x8 af[2], bf[2];
    int ea[2], eb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t ra = r0 + 16 * i + lr, rb = c0 + 16 * i + lr;
      af[i] = load_frag(dq + ra * mpad + (int64_t)mb * kBlock + lk);
      bf[i] = load_frag(xq + rb * mpad + (int64_t)mb * kBlock + lk);
      ea[i] = (int)((de[(mb >> 2) * (2 * f) + ra] >> (8 * (mb & 3))) & 0xFFu);
      eb[i] = (int)((xe[(mb >> 2) * k + rb] >> (8 * (mb & 3))) & 0xFFu);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af[i], bf[j], acc[i][j], 0, 0, 0, ea[i], 0,
                                                                     eb[j]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t row = r0 + 16 * i + lq + e, col = c0 + 16 * j + lr;
        if (row < f)
          store_out(dwg, kBf16Out, row * k + col, acc[i][j][e]);
        else
          store_out(dwu, kBf16Out, (row - f) * k + col, acc[i][j][e]);
      }
}

}  // namespace

hipError_t launch_ffn_grad_quant(const void *dh, const void *g, const void *u, bool in_bf16, int64_t m,
                                 int64_t f, uint8_t *rq, float *rs, uint8_t *cq, uint8_t *ce,
                                 hipStream_t stream) {
  const int64_t mpad = tokens_padded(m);
  const dim3 grid((unsigned)(f / kBlock), (unsigned)(mpad / kBlock)), block(256);
  if (in_bf16)
    hipLaunchKernelGGL(ffn_grad_quant_kernel<true>, grid, block, 0, stream, dh, g, u, m, f, mpad, rq, rs, cq, ce);
  else
    hipLaunchKernelGGL(ffn_grad_quant_kernel<false>, grid, block, 0, stream, dh, g, u, m, f, mpad, rq, rs, cq, ce);
  return hipGetLastError();
}

hipError_t launch_token_quant(const void *x, bool x_bf16, int64_t m, int64_t k, uint8_t *cq, uint8_t *ce,
                              hipStream_t stream) {
  const int64_t mpad = tokens_padded(m);
  const dim3 grid((unsigned)(k / kBlock), (unsigned)(mpad / kBlock)), block(256);
  if (x_bf16)
    hipLaunchKernelGGL(token_quant_kernel<true>, grid, block, 0, stream, x, m, k, mpad, cq, ce);
  else
    hipLaunchKernelGGL(token_quant_kernel<false>, grid, block, 0, stream, x, m, k, mpad, cq, ce);
  return hipGetLastError();
}

hipError_t launch_weights_transpose(const uint8_t *wg, const float *wg_s, const uint8_t *wu,
                                    const float *wu_s, int64_t f, int64_t k, uint8_t *wt, float *wt_s,
                                    hipStream_t stream) {
  hipLaunchKernelGGL(weights_transpose_kernel, dim3((unsigned)(k / kBlock), (unsigned)(f / kBlock), 2), dim3(256), 0,
                     stream, wg, wg_s, wu, wu_s, f, k, wt, wt_s);
  return hipGetLastError();
}

hipError_t launch_weight_grad(const uint8_t *dq, const uint8_t *de, const uint8_t *xq, const uint8_t *xe,
                              void *dwg, void *dwu, bool out_bf16, int64_t m, int64_t f, int64_t k,
                              hipStream_t stream) {
  const int64_t mpad = tokens_padded(m);
  const dim3 grid((unsigned)(k / 64), (unsigned)(2 * f / 64)), block(256);
  if (out_bf16)
    hipLaunchKernelGGL(weight_grad_simple_kernel<true>, grid, block, 0, stream, dq, (const uint32_t *)de, xq,
                       (const uint32_t *)xe, dwg, dwu, mpad, f, k);
  else
    hipLaunchKernelGGL(weight_grad_simple_kernel<false>, grid, block, 0, stream, dq, (const uint32_t *)de, xq,
                       (const uint32_t *)xe, dwg, dwu, mpad, f, k);
  return hipGetLastError();
}

}  // namespace fp8bsq
