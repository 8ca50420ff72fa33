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

// One 1 x 128 block on 16 lanes, eight values each: codes and scale.
template <bool kBf16>
__device__ __forceinline__ u32x2 quantize_block(const u32x4 (&v)[kBf16 ? 1 : 2], bool ue8m0, float &s) {
  float r;
  if constexpr (kBf16) {
    u16x2 m2 = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(u16x2, v[0][j] & 0x7FFF7FFFu));
    block_scale_fast(row_max_u32((uint32_t)(m2.x > m2.y ? m2.x : m2.y) << 16), ue8m0, s, r);
    return encode_chunk_bf16(v[0], s, r);
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max(v[0][j] & 0x7FFFFFFFu, v[1][j] & 0x7FFFFFFFu));
    block_scale(row_max_u32(top), ue8m0, s, r);
    return u32x2{encode_chunk_f32(v[0], s), encode_chunk_f32(v[1], s)};
  }
}

template <bool kBf16>
__device__ __forceinline__ void load_block(const void *x, int64_t block, int sub, u32x4 (&v)[kBf16 ? 1 : 2]) {
  if constexpr (kBf16) {
    v[0] = ((const u32x4 *)x)[block * 16 + sub];
  } else {
    v[0] = ((const u32x4 *)x)[block * 32 + 2 * sub];
    v[1] = ((const u32x4 *)x)[block * 32 + 2 * sub + 1];
  }
}

// act_quant's arithmetic with the scales laid out [K block][row], as the tile
// kernels' transfers read them.  Sixteen lanes own a 1 x 128 block, 8 values
// each; a workgroup takes 16 rows and up to four consecutive K blocks of them,
// so a row is read in 1 KB runs (bf16) and 16 rows' scales are written together.
// Bound by memory: 8192 x 7168 bf16 36 us, 4.9 TB/s; small ones by the launch.
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
    if (i < n) load_block<kBf16>(x, blk0 + i, sub, v[i]);
#pragma unroll
  for (int i = 0; i < kQuantKb; ++i) {
    if (i >= n) break;
    float s;
    const u32x2 codes = quantize_block<kBf16>(v[i], kUe8m0, s);
    *(u32x2 *)(a + (blk0 + i) * kBlock + 8 * sub) = codes;
    if (sub == 0) a_s[(kb0 + i) * stride + row] = s;
  }
}

// ---------------------------------------------------------------------------
// Few rows of x (the decode step): bound by the weights' bytes, which stream
// once from HBM.
//
// A compute wave owns eight features: its MFMA rows are the eight gate rows and
// the eight up rows of these, its columns up to 16 rows of x, so one MFMA per K
// block serves both projections, and a lane's gate values sit 32 lanes from
// their up values.  Each wave moves its own 16 weight rows, whole 128-byte
// lines, into its own kDepth-slot LDS ring, and waits for nothing else.  A
// workgroup has `tiles` waves' worth of features times `parts` waves that share
// these and split K (their sums meet in LDS): the launch takes as many tiles as
// give every CU one workgroup, and parts where there are fewer tiles than eight
// a CU.
//
// The other waves of the workgroup's 16 quantize x with act_quant's arithmetic
// into LDS while the first weights are on their way; compute waves that loaded x
// themselves would wait for their own older weight transfers first.  They go in
// K order in up to kPhases pieces, a barrier after each, so that the K loop
// starts on the first piece.
//
// Measured, one row, 18432 x 7168 (264 MB of weights): 48 us, 5.5 TB/s, above a
// 1 GiB copy's 5.1; the first, simple kernel took 110 us.
// ---------------------------------------------------------------------------
constexpr int kDecodeRows = 16, kDecodeWaves = 16, kDecodeFeatures = 8, kPhases = 4;

struct DecodeArgs {
  const void *x;
  const uint8_t *wg, *wu;
  const float *wg_s, *wu_s;
  void *h, *g, *u;
  int64_t f, k;
  int m, nkb, tiles, parts, phases;
  bool ue8m0, out_bf16, vec;
};

template <bool kBf16X, int kDepth>
__global__ __launch_bounds__(64 * kDecodeWaves) void gated_decode_kernel(const DecodeArgs p) {
  // [compute wave][slot][16 rows x 128], codes [K block][row][128], scales
  // [K block][16 rows], partial sums [compute wave][64 lanes][4]
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int compute = p.tiles * p.parts;
  constexpr int kSlotBytes = 16 * kBlock;
  uint8_t *codes = lds + compute * kDepth * kSlotBytes;
  float *scales = (float *)(codes + (int64_t)p.m * p.k);
  f32x4 *sums = (f32x4 *)(scales + p.nkb * kDecodeRows);
  const int per = (p.nkb + p.parts - 1) / p.parts, piece = (per + p.phases - 1) / p.phases;

  if (wave >= compute) {
    // block `idx` of a phase: K block first + idx / (rows * parts) of every part
    const int groups = 4 * (kDecodeWaves - compute), sub = lane & 15, across = p.m * p.parts;
    const int group = (wave - compute) * 4 + (lane >> 4);
    for (int phase = 0; phase < p.phases; ++phase) {
      const int first = phase * piece, n = (min(per, first + piece) - first) * across;
      constexpr int kBatch = 4;
      for (int base = group; base < n; base += kBatch * groups) {
        u32x4 v[kBatch][kBf16X ? 1 : 2];
        int at[kBatch];   // K block * 16 + row, or -1
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int idx = base + i * groups;
          const int j = idx / across, rest = idx - j * across, part = rest / p.m, row = rest - part * p.m;
          const int kb = part * per + first + j;
          at[i] = idx < n && kb < p.nkb ? kb * 16 + row : -1;
          if (at[i] >= 0) load_block<kBf16X>(p.x, (int64_t)row * p.nkb + kb, sub, v[i]);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (at[i] < 0) continue;
          const int kb = at[i] >> 4, row = at[i] & 15;
          float s;
          const u32x2 c = quantize_block<kBf16X>(v[i], p.ue8m0, s);
          *(u32x2 *)(codes + ((int64_t)kb * p.m + row) * kBlock + (((sub >> 1) ^ swz(row)) << 4) + 8 * (sub & 1)) = c;
          if (sub == 0) scales[at[i]] = s;
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      workgroup_barrier();
    }
    if (p.parts > 1) workgroup_barrier();   // the compute waves' sums
    return;
  }

  const int tile = wave / p.parts, part = wave - tile * p.parts;
  const int64_t f0 = ((int64_t)blockIdx.x * p.tiles + tile) * kDecodeFeatures;
  const int64_t fc = min(f0, p.f - 1);   // a tile past the last feature re-reads it
  const int fr = lane & 15, fq = lane >> 4, dr = lane >> 3, ds = lane & 7;
  const uint32_t row_off = (uint32_t)((min(fc + dr, p.f - 1) - fc) * p.k);
  const uint32_t off0 = row_off + ((ds ^ swz(dr)) << 4), off1 = row_off + ((ds ^ swz(8 + dr)) << 4);
  const uint8_t *gate = p.wg + fc * p.k, *up = p.wu + fc * p.k;
  const uint8_t *ring = lds + wave * kDepth * kSlotBytes;
  const uint32_t lds_ring = lds_addr(ring);
  const int kb0 = min(p.nkb, part * per), kb1 = min(p.nkb, kb0 + per);
  auto issue = [&](int kb) {   // past the end: the last block again, so that every block counts the same
    const int64_t at = (int64_t)max(min(kb, kb1 - 1), 0) * kBlock;
    const uint32_t slot = lds_ring + (uint32_t)((kb - kb0) % kDepth) * kSlotBytes;
    lds_dma16(gate + at, off0, slot);
    lds_dma16(up + at, off1, slot + 1024);
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) issue(kb0 + d);
  const float *gs = p.wg_s + fc / kBlock * p.nkb, *us = p.wu_s + fc / kBlock * p.nkb;
  const bool live = fr < p.m;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int phase = 0; phase < p.phases; ++phase) {
    workgroup_barrier();   // this piece's codes are in LDS
    const int end = min(kb1, kb0 + (phase + 1) * piece);
    for (int kb = kb0 + phase * piece; kb < end; ++kb) {
      const float sg = load_uniform(gs, kb), su = load_uniform(us, kb);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * (kDepth - 1)) : "memory");   // block kb landed
      const uint8_t *slot = ring + (kb - kb0) % kDepth * kSlotBytes;
      const i32x8 w = frag_from_lds(slot + fr * kBlock, fq, fr);
      i32x8 a = {0, 0, 0, 0, 0, 0, 0, 0};
      float sa = 0.0f;
      if (live) {
        a = frag_from_lds(codes + ((int64_t)kb * p.m + fr) * kBlock, fq, fr);
        sa = scales[kb * 16 + fr];
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: the slot may be refilled
      issue(kb + kDepth);
      const f32x4 q = mfma_e4m3_16x16x128(w, a, f32x4{0.f, 0.f, 0.f, 0.f});
      const float sc = sa * (fq < 2 ? sg : su);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(q[e], sc, acc[e]);
    }
  }
  wait_dma_all();   // transfers past the end, before the workgroup's LDS is released
  if (p.parts > 1) {
    if (part > 0) sums[wave * 64 + lane] = acc;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    workgroup_barrier();
    if (part > 0) return;
    for (int q = 1; q < p.parts; ++q) acc += sums[(wave + q) * 64 + lane];
  }
  f32x4 upper;
#pragma unroll
  for (int e = 0; e < 4; ++e) upper[e] = __shfl_xor(acc[e], 32);
  const int64_t col = f0 + 4 * fq;
  if (fq >= 2 || !live || col >= p.f) return;
  const int left = (int)min((int64_t)4, p.f - col);
  const int64_t at = fr * p.f + col;
  if (p.out_bf16) {
    if (p.vec) store_gated<true, true>(p.h, p.g, p.u, at, acc, upper, 4);
    else store_gated<true, false>(p.h, p.g, p.u, at, acc, upper, left);
  } else {
    if (p.vec) store_gated<false, true>(p.h, p.g, p.u, at, acc, upper, 4);
    else store_gated<false, false>(p.h, p.g, p.u, at, acc, upper, left);
  }
}

// How the decode kernel is launched; depth 0: it does not take these sizes.
struct DecodePlan {
  int tiles = 0, parts = 0, depth = 0, phases = 1;
  size_t lds = 0;
};

DecodePlan decode_plan(int64_t m, int64_t f, int64_t k) {
  DecodePlan p;
  if (m > kDecodeRows || m * k > 128 * 1024) return p;
  int cus = current_device_cus();
  if (cus <= 0) cus = 256;
  const int nkb = (int)(k / kBlock);
  const int64_t all = (f + kDecodeFeatures - 1) / kDecodeFeatures;
  p.tiles = (int)min((all + cus - 1) / cus, (int64_t)9);
  p.parts = 1;
  while (2 * p.parts * p.tiles <= 8 && 2 * p.parts <= nkb) p.parts *= 2;
  const int compute = p.tiles * p.parts;
  const size_t rest = (size_t)m * k + (size_t)nkb * kDecodeRows * 4 + (p.parts > 1 ? (size_t)compute * 1024 : 0);
  for (int depth : {8, 6, 4, 3, 2}) {
    p.lds = rest + (size_t)compute * depth * 16 * kBlock;
    if (p.lds <= 160 * 1024) {
      p.depth = depth;
      break;
    }
  }
  // one piece while the quantizing waves need no more than two rounds of loads
  p.phases = m * nkb > 8 * 4 * (kDecodeWaves - compute) ? kPhases : 1;
  return p;
}

template <bool kBf16X>
hipError_t launch_decode(const DecodePlan &plan, const DecodeArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.f + plan.tiles * kDecodeFeatures - 1) / (plan.tiles * kDecodeFeatures)));
  const dim3 block(64 * kDecodeWaves);
  switch (plan.depth) {
    case 8: hipLaunchKernelGGL((gated_decode_kernel<kBf16X, 8>), grid, block, plan.lds, stream, a); break;
    case 6: hipLaunchKernelGGL((gated_decode_kernel<kBf16X, 6>), grid, block, plan.lds, stream, a); break;
    case 4: hipLaunchKernelGGL((gated_decode_kernel<kBf16X, 4>), grid, block, plan.lds, stream, a); break;
    case 3: hipLaunchKernelGGL((gated_decode_kernel<kBf16X, 3>), grid, block, plan.lds, stream, a); break;
    default: hipLaunchKernelGGL((gated_decode_kernel<kBf16X, 2>), grid, block, plan.lds, stream, a); break;
  }
  return hipGetLastError();
}

TilePlan gated_plan(int64_t m, int64_t f, int64_t k) {
  return tile_plan(m, f, kBigTile / 2, (int)(k / kBlock), current_device_cus());
}

}  // namespace

FfnSpace gated_space(int64_t m, int64_t f, int64_t k) {
  FfnSpace s;
  if (decode_plan(m, f, k).depth) {   // one kernel, nothing in memory
    s.bytes = 256;
    return s;
  }
  const TilePlan plan = gated_plan(m, f, k);
  s.a = s.add(m * k);
  s.a_s = s.add((k / kBlock) * rows_padded(m) * 4);
  s.partials = s.add((int64_t)plan.partial_bytes);
  return s;
}

hipError_t launch_gated_ffn(const void *x, bool x_bf16, bool ue8m0, const uint8_t *wg, const float *wg_s,
                            const uint8_t *wu, const float *wu_s, void *h, void *g_out, void *u_out, bool out_bf16,
                            int64_t m, int64_t f, int64_t k, void *workspace, hipStream_t stream) {
  const uintptr_t mask = out_bf16 ? 7 : 15;
  const bool vec = f % 4 == 0 && (((uintptr_t)h | (uintptr_t)g_out | (uintptr_t)u_out) & mask) == 0;
  const DecodePlan decode = decode_plan(m, f, k);
  if (decode.depth) {
    DecodeArgs d = {x, wg, wu, wg_s, wu_s, h, g_out, u_out, f, k, (int)m, (int)(k / kBlock), decode.tiles,
                    decode.parts, decode.phases, ue8m0, out_bf16, vec};
    return x_bf16 ? launch_decode<true>(decode, d, stream) : launch_decode<false>(decode, d, stream);
  }
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
#define FP8BSQ_GATED(MX, BF, VEC) launch_tiles<TileMode::kGated, MX, BF, VEC>(plan, p, cus, stream)
#define FP8BSQ_GATED_OUT(MX)                                                    \
  (out_bf16 ? (vec ? FP8BSQ_GATED(MX, true, true) : FP8BSQ_GATED(MX, true, false)) \
            : (vec ? FP8BSQ_GATED(MX, false, true) : FP8BSQ_GATED(MX, false, false)))
  return ue8m0 ? FP8BSQ_GATED_OUT(true) : FP8BSQ_GATED_OUT(false);
#undef FP8BSQ_GATED_OUT
#undef FP8BSQ_GATED
}

}  // namespace fp8bsq
