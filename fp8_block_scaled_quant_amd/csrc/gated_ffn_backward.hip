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
#include "device_cus.h"
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
// dW [2 f, k] = dgu^T x over the tokens.  Power-of-two scales on both operands
// go into the MFMA (one exponent per row and 128 tokens, which is the MFMA's
// whole K), so the matrix core accumulates by itself and no vector instruction
// touches an accumulator before the epilogue.
//
// Workgroup tile 256 x 256, 512 threads = 8 waves, 2 (dgu rows) x 4 (x rows),
// each 128 x 64: acc[8][4] tiles of 16 x 16.  Operands come by direct
// global->LDS transfers into a two-stage ring (token block mb + 1 while mb is
// computed); exponents come from memory straight to registers, one word of four
// token blocks per fragment row, a chunk ahead.  The x rows are the MFMA's row
// operand, so a lane holds four consecutive columns of a dW row.
// ---------------------------------------------------------------------------
constexpr int kDwTile = 256, kDwThreads = 512;

struct DwSmem {
  uint8_t a[2][kDwTile * kBlock];   // dgu rows
  uint8_t b[2][kDwTile * kBlock];   // x rows
};

// Tile of workgroup turn `it`: each XCD (workgroups are dealt to the eight
// round-robin) walks a contiguous share of the tiles, in groups of four dgu
// tiles across x's.
__device__ __forceinline__ void dw_tile_coords(int it, int tiles_r, int tiles_c, int &tr, int &tc) {
  const int ntiles = tiles_r * tiles_c, base = ntiles / 8, rest = ntiles % 8, xcd = it % 8;
  const int tile = xcd * base + min(xcd, rest) + it / 8;
  constexpr int kGroup = 4;
  const int group = tile / (kGroup * tiles_c), first = group * kGroup;
  const int gr = min(tiles_r - first, kGroup), idx = tile - group * kGroup * tiles_c;
  tr = first + idx % gr;
  tc = idx / gr;
}

template <bool kBf16Out>
__global__ __launch_bounds__(kDwThreads) void weight_grad_tile_kernel(
    const uint8_t *__restrict__ dq, const uint32_t *__restrict__ de, const uint8_t *__restrict__ xq,
    const uint32_t *__restrict__ xe, void *__restrict__ dwg, void *__restrict__ dwu, int64_t mpad, int64_t f,
    int64_t k, int tiles_r, int tiles_c) {
  __shared__ __attribute__((aligned(1024))) DwSmem sm;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nmb = (int)(mpad / kBlock), ntiles = tiles_r * tiles_c;
  const int64_t rows = 2 * f;
  const int wr = (wave >> 2) * 128, wc = (wave & 3) * 64;
  const int fr = lane & 15, fq = lane >> 4, dr = lane >> 3, ds = lane & 7;
  const uint32_t lds_a = lds_addr(&sm.a[0][0]), lds_b = lds_addr(&sm.b[0][0]);
  for (int it = blockIdx.x; it < ntiles; it += gridDim.x) {
    int tr, tc;
    dw_tile_coords(it, tiles_r, tiles_c, tr, tc);
    const int64_t r0 = (int64_t)tr * kDwTile, c0 = (int64_t)tc * kDwTile;
    // 8-row groups 4 wave .. + 3 of both operands; rows past the matrix re-read its last
    uint32_t a_off[4], b_off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * (4 * wave + i) + dr;
      const int chunk = (ds ^ swz(row)) << 4;
      a_off[i] = (uint32_t)((min(r0 + row, rows - 1) - r0) * mpad + chunk);
      b_off[i] = (uint32_t)((min(c0 + row, k - 1) - c0) * mpad + chunk);
    }
    const uint8_t *a_base = dq + r0 * mpad, *b_base = xq + c0 * mpad;
    auto issue = [&](int mb, int s) {
      const int64_t at = (int64_t)mb * kBlock;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lds_dma16(a_base + at, a_off[i], lds_a + s * (kDwTile * kBlock) + (4 * wave + i) * 1024);
        lds_dma16(b_base + at, b_off[i], lds_b + s * (kDwTile * kBlock) + (4 * wave + i) * 1024);
      }
    };
    uint32_t ea[8], eb[4], ea_next[8], eb_next[4];
    auto load_exps = [&](int chunk) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ea_next[i] = de[(int64_t)chunk * rows + min(r0 + wr + 16 * i + fr, rows - 1)];
#pragma unroll
      for (int j = 0; j < 4; ++j) eb_next[j] = xe[(int64_t)chunk * k + min(c0 + wc + 16 * j + fr, k - 1)];
    };
    f32x4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (nmb > 0) {
      issue(0, 0);
      load_exps(0);
    }
#pragma nounroll
    for (int mb = 0; mb < nmb; ++mb) {
      const int cur = mb & 1;
      wait_dma_all();
      workgroup_barrier();   // stage cur landed for every wave; stage cur ^ 1 no longer read
      if ((mb & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ea[i] = ea_next[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) eb[j] = eb_next[j];
        if (mb + 4 < nmb) load_exps(mb / 4 + 1);
      }
      if (mb + 1 < nmb) issue(mb + 1, cur ^ 1);
      i32x8 bf[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = wc + 16 * j + fr;
        bf[j] = frag_from_lds(&sm.b[cur][r * kBlock], fq, r);
      }
      const int shift = 8 * (mb & 3);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = wr + 16 * i + fr;
        const i32x8 af = frag_from_lds(&sm.a[cur][r * kBlock], fq, r);
        const int sa = (int)((ea[i] >> shift) & 0xFFu);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[j], af, acc[i][j], 0, 0, 0,
                                                                       (int)((eb[j] >> shift) & 0xFFu), 0, sa);
      }
    }
    workgroup_barrier();   // every wave is done with LDS before the next tile's transfers
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = r0 + wr + 16 * i + fr;
      if (row >= rows) continue;
      void *out = row < f ? dwg : dwu;
      const int64_t at = (row < f ? row : row - f) * k;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t col = c0 + wc + 16 * j + 4 * fq;
        if (col >= k) continue;   // k is a multiple of 128: four columns are in or out together
        const f32x4 v = acc[i][j];
        if (kBf16Out)
          *(u32x2 *)((uint16_t *)out + at + col) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
          *(f32x4 *)((float *)out + at + col) = v;
      }
    }
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
  const int64_t tiles_r = (2 * f + kDwTile - 1) / kDwTile, tiles_c = (k + kDwTile - 1) / kDwTile;
  int cus = current_device_cus();
  if (cus <= 0) cus = 256;
  const dim3 grid((unsigned)(tiles_r * tiles_c < cus ? tiles_r * tiles_c : cus)), block(kDwThreads);
  if (out_bf16)
    hipLaunchKernelGGL(weight_grad_tile_kernel<true>, grid, block, 0, stream, dq, (const uint32_t *)de, xq,
                       (const uint32_t *)xe, dwg, dwu, mpad, f, k, (int)tiles_r, (int)tiles_c);
  else
    hipLaunchKernelGGL(weight_grad_tile_kernel<false>, grid, block, 0, stream, dq, (const uint32_t *)de, xq,
                       (const uint32_t *)xe, dwg, dwu, mpad, f, k, (int)tiles_r, (int)tiles_c);
  return hipGetLastError();
}

}  // namespace fp8bsq
