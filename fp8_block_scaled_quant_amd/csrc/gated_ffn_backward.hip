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
// Quantizers.  A workgroup of 512 threads owns a 128 x 128 tile; lane l of wave
// w holds rows 4 (4 w + l / 16) .. + 3 and columns 8 (l % 16) .. + 7, so loads
// cover 256-byte row segments, a row's amax is a DPP reduction over 16 lanes,
// and a column's four rows pack into one 4-byte piece of the transposed tile,
// which goes through LDS to whole-line stores.
//
// Measured, 4096 x 18432 and x 4096 x 7168: 843 MB in 168 us, 5.0 TB/s, a copy's
// rate; 333 x 1024 and x 896 6 us.  What it took: no branch inside the unrolled
// element loops (199 and 10.5 us with rows tested at their loads), transposed
// stores that meet every bank once (225 us on half the banks), and the column
// scales found once a workgroup (212 us by every thread).
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 512, kQuantWaves = kQuantThreads / 64, kLaneRows = 4;

template <bool kBf16>
__device__ __forceinline__ void load8(const void *p, int64_t idx, float (&v)[8]) {
  if (kBf16) {
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

// The values of rows past the last, loaded from it, are zero.
__device__ __forceinline__ void clear_past(float (&v)[kLaneRows][8], int64_t row0, int64_t m0, int64_t m) {
  if (m0 + kBlock <= m) return;
#pragma unroll
  for (int r = 0; r < kLaneRows; ++r)
#pragma unroll
    for (int c = 0; c < 8; ++c) v[r][c] = row0 + r < m ? v[r][c] : 0.0f;
}

// E4M3 codes of four values already divided by their scale.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return cvt_pk_e4m3<true>(c, d, cvt_pk_e4m3<false>(a, b, 0u));
}

struct TokenTile {
  // [column][token]: 16-byte pieces swizzled by the column's 8, and columns 64
  // on in swapped pairs, so that a wave's stores, 16 columns apart by 8, touch
  // all banks once
  alignas(16) uint8_t codes[128 * 128];
  uint32_t colmax[128][kQuantWaves + 1];   // padded: a lane's eight columns, 8 apart, in different banks
  alignas(16) float inverse[128];
};

// Quantize a tile's values v [4 rows][8 columns] along the rows (tokens) and
// write it transposed: codes to out [row0 + column][mpad] at token m0, the
// scales to scales[row0 + column].  Every thread of the workgroup takes part.
__device__ __forceinline__ void store_tokens(const float (&v)[kLaneRows][8], TokenTile &sm, uint8_t *__restrict__ out,
                                             float *__restrict__ scales, int64_t row0, int64_t m0, int64_t mpad) {
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63, grp = lane >> 4, sub = lane & 15;
  uint32_t top[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    top[c] = max(max(abs_bits(v[0][c]), abs_bits(v[1][c])), max(abs_bits(v[2][c]), abs_bits(v[3][c])));
    // against the lane 16, then 32 away: the swap of a value with itself leaves
    // one of the pair's two in every lane of either result
    const auto far16 = __builtin_amdgcn_permlane16_swap(top[c], top[c], false, false);
    top[c] = max(far16[0], far16[1]);
    const auto far32 = __builtin_amdgcn_permlane32_swap(top[c], top[c], false, false);
    top[c] = max(far32[0], far32[1]);
  }
  if (grp == 0) {
#pragma unroll
    for (int c = 0; c < 8; ++c) sm.colmax[8 * sub + c][wave] = top[c];
  }
  __syncthreads();
  {   // four lanes a column
    const uint32_t *w = &sm.colmax[t >> 2][2 * (t & 3)];
    const uint32_t e = e4m3_scale_byte(quad_max_u32(max(w[0], w[1])));
    if ((t & 3) == 0) {
      sm.inverse[t >> 2] = pow2_inverse(e);
      scales[row0 + (t >> 2)] = pow2_scale(e);
    }
  }
  __syncthreads();
  const f32x4 lo = *(const f32x4 *)&sm.inverse[8 * sub], hi = *(const f32x4 *)&sm.inverse[8 * sub + 4];
  const int piece = wave;   // 16 tokens
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int col = 8 * sub + c;
    const float inv = c < 4 ? lo[c & 3] : hi[c & 3];
    *(uint32_t *)&sm.codes[(col ^ (sub >> 3)) * 128 + ((piece ^ (sub & 7)) << 4) + 4 * grp] =
        codes4(v[0][c] * inv, v[1][c] * inv, v[2][c] * inv, v[3][c] * inv);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 128 * 8 / kQuantThreads; ++i) {
    const int idx = i * kQuantThreads + t, col = idx >> 3, j = idx & 7;
    *(u32x4 *)(out + (row0 + col) * mpad + m0 + 16 * j) =
        *(const u32x4 *)&sm.codes[(col ^ (col >> 6)) * 128 + ((j ^ ((col >> 3) & 7)) << 4)];
  }
  __syncthreads();   // the tile may be reused
}

// Quantize each row's 128 columns: codes to out + row * ld (the lane's eight
// columns), scale to scales[row].
__device__ __forceinline__ void store_rows(const float (&v)[kLaneRows][8], uint8_t *__restrict__ out, int64_t ld,
                                           float *__restrict__ scales, int64_t row0, int64_t m) {
  const int sub = threadIdx.x & 15;
#pragma unroll
  for (int r = 0; r < kLaneRows; ++r) {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) top = max(top, abs_bits(v[r][c]));
    const uint32_t e = e4m3_scale_byte(row_max_u32(top));
    const float inv = pow2_inverse(e);
    if (row0 + r < m) {
      u32x2 q;
      q.x = codes4(v[r][0] * inv, v[r][1] * inv, v[r][2] * inv, v[r][3] * inv);
      q.y = codes4(v[r][4] * inv, v[r][5] * inv, v[r][6] * inv, v[r][7] * inv);
      *(u32x2 *)(out + (row0 + r) * ld) = q;
      if (sub == 0) scales[row0 + r] = pow2_scale(e);
    }
  }
}

struct QuantArgs {
  const void *dh, *g, *u, *x;
  int64_t m, f, k, mpad;
  uint8_t *rq;   // [m][2 f] codes along the features, or null
  float *rs;     // [2 f / 128][rs_stride]
  int64_t rs_stride;
  uint8_t *cq;   // [2 f][mpad] codes along the tokens, or null
  float *cs;     // [mpad / 128][cs_stride]
  int64_t cs_stride;
  uint8_t *xq;   // [k][mpad], with cq
  float *xs;     // [mpad / 128][k]
  int grad_tiles;
};

// Everything that the products read, in one launch: the first workgroups
// quantize a tile of dg and du each, the others a tile of x.  With fewer tiles
// than CUs (kSplit) the tile's four results (dg or du, along the features or the
// tokens) go to a workgroup each (333 x 1024 in one piece: 15 us in the kernel's
// first form, 11 in four, its arithmetic on 24 CUs).
template <bool kBf16, bool kSplit>
__global__ __launch_bounds__(kQuantThreads) void ffn_quant_kernel(const QuantArgs p) {
  __shared__ TokenTile sm;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lane_row = kLaneRows * (4 * wave + (lane >> 4)), lane_col = 8 * (lane & 15);
  const int grads = p.grad_tiles * (kSplit ? 4 : 1);
  if ((int)blockIdx.x >= grads) {
    const int tile = blockIdx.x - grads, across = (int)(p.k / kBlock);
    const int64_t m0 = (int64_t)(tile / across) * kBlock, k0 = (int64_t)(tile % across) * kBlock;
    float v[kLaneRows][8];
#pragma unroll
    for (int r = 0; r < kLaneRows; ++r) load8<kBf16>(p.x, min(m0 + lane_row + r, p.m - 1) * p.k + k0 + lane_col, v[r]);
    clear_past(v, m0 + lane_row, m0, p.m);
    store_tokens(v, sm, p.xq, p.xs + m0 / kBlock * p.k, k0, m0, p.mpad);
    return;
  }
  const int tile = kSplit ? blockIdx.x >> 2 : blockIdx.x, across = (int)(p.f / kBlock);
  const int64_t m0 = (int64_t)(tile / across) * kBlock, f0 = (int64_t)(tile % across) * kBlock;
  const int64_t row0 = m0 + lane_row;
  // the two gradients from dh, g, u: the reciprocal instruction is within one
  // ulp; exp overflows to infinity for g below -88, where the sigmoid is 0 to
  // fp32's precision.  The slope meets u before h: h u may overflow where the
  // slope is 0 (a closed gate), and their product would be NaN
  auto sigmoid = [](float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); };
  auto grad_gate = [](float h, float g, float u, float s) { return h * (u * (s * __builtin_fmaf(g, 1.0f - s, 1.0f))); };
  auto grad_up = [](float h, float g, float s) { return h * (g * s); };
  auto along_rows = [&](const float (&v)[kLaneRows][8], bool gate) {
    store_rows(v, p.rq + (gate ? 0 : p.f) + f0 + lane_col, 2 * p.f,
               p.rs + (f0 + (gate ? 0 : p.f)) / kBlock * p.rs_stride, row0, p.m);
  };
  auto along_tokens = [&](const float (&v)[kLaneRows][8], bool gate) {
    store_tokens(v, sm, p.cq, p.cs + m0 / kBlock * p.cs_stride, (gate ? 0 : p.f) + f0, m0, p.mpad);
  };
  float hv[kLaneRows][8], gv[kLaneRows][8], uv[kLaneRows][8];
  const bool split_gate = (blockIdx.x & 1) == 0, split_rows = (blockIdx.x & 2) == 0;
  if (kSplit && (split_rows ? !p.rq : !p.cq)) return;
#pragma unroll
  for (int r = 0; r < kLaneRows; ++r) {
    const int64_t idx = min(row0 + r, p.m - 1) * p.f + f0 + lane_col;
    load8<kBf16>(p.dh, idx, hv[r]);
    load8<kBf16>(p.g, idx, gv[r]);
    if (!kSplit) load8<kBf16>(p.u, idx, uv[r]);
  }
  if (kSplit) {
    if (split_gate) {
#pragma unroll
      for (int r = 0; r < kLaneRows; ++r) load8<kBf16>(p.u, min(row0 + r, p.m - 1) * p.f + f0 + lane_col, uv[r]);
#pragma unroll
      for (int r = 0; r < kLaneRows; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) hv[r][c] = grad_gate(hv[r][c], gv[r][c], uv[r][c], sigmoid(gv[r][c]));
    } else {
#pragma unroll
      for (int r = 0; r < kLaneRows; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) hv[r][c] = grad_up(hv[r][c], gv[r][c], sigmoid(gv[r][c]));
    }
    clear_past(hv, row0, m0, p.m);
    if (split_rows) along_rows(hv, split_gate); else along_tokens(hv, split_gate);
    return;
  }
#pragma unroll
  for (int r = 0; r < kLaneRows; ++r)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float h = hv[r][c], g = gv[r][c], s = sigmoid(g);
      hv[r][c] = grad_gate(h, g, uv[r][c], s);
      gv[r][c] = grad_up(h, g, s);
    }
  clear_past(hv, row0, m0, p.m);
  clear_past(gv, row0, m0, p.m);
  if (p.rq) {
    along_rows(hv, true);
    along_rows(gv, false);
  }
  if (p.cq) {
    along_tokens(hv, true);
    along_tokens(gv, false);
  }
}

// dx and dW in one launch, where both are too small to fill the GPU: the first
// `first` workgroups are dx's.
template <bool kBf16Out>
__global__ __launch_bounds__(kMidThreads) void mid_pair_kernel(const TileArgs in, const TileArgs wt, int first) {
  __shared__ __attribute__((aligned(1024))) MidSlot ring[kMidSlots];
  if ((int)blockIdx.x < first)
    mid_tile<TileMode::kInput, true, kBf16Out, true>(in, blockIdx.x, first, ring);
  else
    mid_tile<TileMode::kWeight, true, kBf16Out, true>(wt, blockIdx.x - first, gridDim.x - first, ring);
}

template <bool kBf16Out>
__global__ __launch_bounds__(256) void reduce_pair_kernel(const TileArgs in, const TileArgs wt, int first) {
  if ((int)blockIdx.x < first)
    mid_reduce<TileMode::kInput, kBf16Out, true>(in, blockIdx.x);
  else
    mid_reduce<TileMode::kWeight, kBf16Out, true>(wt, blockIdx.x - first);
}

hipError_t launch_mid_pair(const TilePlan &in, TileArgs pi, const TilePlan &wt, TileArgs pw, bool out_bf16,
                           hipStream_t stream) {
  in.fill(pi);
  wt.fill(pw);
  const int first = in.tiles_a * in.tiles_b * in.parts;
  const dim3 grid((unsigned)(first + wt.tiles_a * wt.tiles_b * wt.parts)), block(kMidThreads);
  if (out_bf16)
    hipLaunchKernelGGL(mid_pair_kernel<true>, grid, block, 0, stream, pi, pw, first);
  else
    hipLaunchKernelGGL(mid_pair_kernel<false>, grid, block, 0, stream, pi, pw, first);
  const int rin = in.parts > 1 ? in.tiles_a * in.tiles_b * 4 : 0, rwt = wt.parts > 1 ? wt.tiles_a * wt.tiles_b * 4 : 0;
  if (rin + rwt > 0) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (out_bf16)
      hipLaunchKernelGGL(reduce_pair_kernel<true>, dim3((unsigned)(rin + rwt)), dim3(256), 0, stream, pi, pw, rin);
    else
      hipLaunchKernelGGL(reduce_pair_kernel<false>, dim3((unsigned)(rin + rwt)), dim3(256), 0, stream, pi, pw, rin);
  }
  return hipGetLastError();
}

// dx and dW in one launch of 256 x 256 tiles.  Few of dx's tiles, each long, leave
// a part of the last round idle: the workgroups from `late` on, that have one
// less of them, take `extra` of dW's tiles each first, as long together as one
// of dx's, and all then share the rest.  4096 x 18432 x 7168 with its quantizer:
// 2092 us, 2145 in two launches; 3000 x 4096 x 4096: 251 and 249.
template <bool kBf16Out>
__global__ __launch_bounds__(kBigThreads) void big_pair_kernel(const TileArgs in, const TileArgs wt, int late, int extra) {
  __shared__ __attribute__((aligned(1024))) BigSmem sm;
  const int all = gridDim.x, self = blockIdx.x, few = all - late, shared = few * extra;
  big_tiles<TileMode::kInput, true, kBf16Out, true>(in, sm, self, [=](int it) { return it + all; });
  workgroup_barrier();   // the stages are free
  big_tiles<TileMode::kWeight, true, kBf16Out, true>(wt, sm, self >= late && extra > 0 ? self - late : shared + self,
                                                     [=](int it) {
                                                       if (it >= shared) return it + all;
                                                       return it + few < shared ? it + few : shared + self;
                                                     });
}

hipError_t launch_big_pair(const TilePlan &in, TileArgs pi, const TilePlan &wt, TileArgs pw, bool out_bf16, int cus,
                           hipStream_t stream) {
  if (cus <= 0) cus = 256;
  in.fill(pi);
  wt.fill(pw);
  const int tiles = in.tiles_a * in.tiles_b;
  // positions that are equal modulo 8 share an XCD's L2: keep to that
  const int late = min((tiles % cus + 7) / 8 * 8, cus);
  constexpr double kFixed = kBigRoundUs / kBigBlockUs;
  const int extra = late > 0 && late < cus ? (int)((pi.nkb + kFixed) / (pw.nkb + kFixed) + 0.5) : 0;
  if (out_bf16)
    hipLaunchKernelGGL(big_pair_kernel<true>, dim3(cus), dim3(kBigThreads), 0, stream, pi, pw, late, extra);
  else
    hipLaunchKernelGGL(big_pair_kernel<false>, dim3(cus), dim3(kBigThreads), 0, stream, pi, pw, late, extra);
  return hipGetLastError();
}

TilePlan input_plan(int64_t m, int64_t f, int64_t k) {
  return tile_plan(m, k, kBigTile, (int)(2 * f / kBlock), current_device_cus());
}
TilePlan weight_plan(int64_t m, int64_t f, int64_t k) {
  return tile_plan(2 * f, k, kBigTile, (int)(tokens_padded(m) / kBlock), current_device_cus());
}
// dW's plan beside a dx in 128 x 128 tiles: up to three rounds of those, over few
// tokens, cost less in dx's launch than a launch of 256 x 256 tiles after it.
// Measured (us, one launch and two): 1 x 2048 x 1792 28 and 34, 64 x 1664 x 1664 24
// and 32, 5 x 1536 x 3712 33 and 36, 1000 x 2048 x 2048 56 and 58; with ten
// rounds, 2 x 5120 x 3968, 73 and 60.
TilePlan paired_weight_plan(int64_t m, int64_t f, int64_t k) {
  TilePlan wt = weight_plan(m, f, k);
  const int64_t tiles_a = 2 * f / kMidTile, tiles_b = k / kMidTile;
  const int cus = current_device_cus();
  if (wt.big && tokens_padded(m) <= 8 * kBlock && tiles_a * tiles_b <= 3 * (int64_t)(cus > 0 ? cus : 256)) {
    wt.big = false;
    wt.tiles_a = (int)tiles_a;
    wt.tiles_b = (int)tiles_b;
  }
  return wt;
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
  s.partials = s.add((int64_t)(in.partial_bytes + wt.partial_bytes));
  return s;
}

hipError_t launch_gated_ffn_backward(const void *dh, const void *x, const void *g, const void *u, bool in_bf16,
                                     const uint8_t *wg, const float *wg_s, const uint8_t *wu, const float *wu_s,
                                     void *dx, void *dwg, void *dwu, bool out_bf16, int64_t m, int64_t f, int64_t k,
                                     void *workspace, hipStream_t stream) {
  const bool want_dx = dx && m > 0;
  const TilePlan in = input_plan(m, f, k);
  const TilePlan wt = want_dx && !in.big ? paired_weight_plan(m, f, k) : weight_plan(m, f, k);
  const FfnSpace ws = backward_space(m, f, k);
  const int64_t mpad = tokens_padded(m);
  const int cus = current_device_cus();
  uint8_t *base = (uint8_t *)workspace;
  float *partials = (float *)(base + ws.partials);
  if (m > 0) {
    QuantArgs q = {};
    q.dh = dh;
    q.g = g;
    q.u = u;
    q.x = x;
    q.m = m;
    q.f = f;
    q.k = k;
    q.mpad = mpad;
    q.rq = dx ? base + ws.a : nullptr;
    q.rs = (float *)(base + ws.a_s);
    q.rs_stride = rows_padded(m);
    q.cq = dwg ? base + ws.cq : nullptr;
    q.cs = (float *)(base + ws.cs);
    q.cs_stride = rows_padded(2 * f);
    q.xq = base + ws.xq;
    q.xs = (float *)(base + ws.xs);
    const int64_t grad_tiles = (f / kBlock) * (mpad / kBlock), x_tiles = dwg ? (k / kBlock) * (mpad / kBlock) : 0;
    q.grad_tiles = (int)grad_tiles;
    const bool split = grad_tiles < (cus > 0 ? cus : 256);
    const dim3 grid((unsigned)(grad_tiles * (split ? 4 : 1) + x_tiles));
#define FP8BSQ_FFN_QUANT(BF, SPLIT) \
  hipLaunchKernelGGL((ffn_quant_kernel<BF, SPLIT>), grid, dim3(kQuantThreads), 0, stream, q)
    if (in_bf16) {
      if (split) FP8BSQ_FFN_QUANT(true, true); else FP8BSQ_FFN_QUANT(true, false);
    } else {
      if (split) FP8BSQ_FFN_QUANT(false, true); else FP8BSQ_FFN_QUANT(false, false);
    }
#undef FP8BSQ_FFN_QUANT
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  TileArgs pi = {}, pw = {};
  pi.a = base + ws.a;
  pi.a_s = (const float *)(base + ws.a_s);
  pi.b0 = wg;
  pi.b1 = wu;
  pi.b0_s = wg_s;
  pi.b1_s = wu_s;
  pi.out0 = dx;
  pi.partials = (float *)(base + ws.partials);
  pi.rows_a = m;
  pi.rows_b = k;
  pi.lda = 2 * f;
  pi.ldb = k;
  pi.a_stride = rows_padded(m);
  pi.nkb = (int)(2 * f / kBlock);
  pi.half = (int)(f / kBlock);
  pw.a = base + ws.cq;
  pw.a_s = (const float *)(base + ws.cs);
  pw.b0 = base + ws.xq;
  pw.b0_s = (const float *)(base + ws.xs);
  pw.out0 = dwg;
  pw.out1 = dwu;
  pw.partials = (float *)(base + ws.partials) + in.partial_bytes / sizeof(float);
  pw.rows_a = 2 * f;
  pw.rows_b = k;
  pw.lda = pw.ldb = mpad;
  pw.a_stride = rows_padded(2 * f);
  pw.b_stride = k;
  pw.nkb = (int)(mpad / kBlock);
  if (want_dx && dwg && !in.big && !wt.big) return launch_mid_pair(in, pi, wt, pw, out_bf16, stream);
  if (want_dx && dwg && in.big && wt.big) return launch_big_pair(in, pi, wt, pw, out_bf16, cus, stream);
  if (want_dx) {
    const hipError_t e = out_bf16 ? launch_tiles<TileMode::kInput, true, true, true>(in, pi, cus, stream)
                                  : launch_tiles<TileMode::kInput, true, false, true>(in, pi, cus, stream);
    if (e != hipSuccess) return e;
  }
  if (!dwg) return hipSuccess;
  return out_bf16 ? launch_tiles<TileMode::kWeight, true, true, true>(wt, pw, cus, stream)
                  : launch_tiles<TileMode::kWeight, true, false, true>(wt, pw, cus, stream);
}

}  // namespace fp8bsq
