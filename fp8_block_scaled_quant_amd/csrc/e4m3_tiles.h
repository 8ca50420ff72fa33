// The E4M3 products of the feed-forward block.  They differ in where operand
// rows come from, how partial sums are scaled, and what happens to a finished
// tile:
//
//   kGated   columns: 128 rows of x;      rows: 64 features, gate and up
//   kInput   columns: 128 rows of dg|du;  rows: 128 columns of the weights,
//            read transposed (ds_read_b64_tr_b8), so the weights stay as stored
//   kWeight  columns: 128 rows of (dg|du)^T;  rows: 128 rows of x^T
//
// "Columns" and "rows" are the MFMA's: lane l of a 16 x 16 result holds column
// l % 16 and rows 4 (l / 16) .. + 3, four consecutive outputs of one row of the
// row-major result.
//
// Scales come as [block][row] fp32.  Where the columns' scales are powers of two
// (gradients always, activations under ue8m0) they go into the MFMA as E8M0
// exponents; a weight's 128 x 128 block scale multiplies an MFMA's partial in
// FP32.  kWeight has power-of-two scales on both sides and accumulates in the
// matrix core.
//
// Two kernels: 256 x 256 operand tiles for outputs that fill the GPU with them,
// and 128 x 128 tiles with a deeper ring and a split contraction for others.
#pragma once

#include "mfma_tile.h"

namespace fp8bsq {

enum class TileMode { kGated, kInput, kWeight };

struct TileArgs {
  const uint8_t *a;         // columns operand [rows_a][lda] codes
  const float *a_s;         // its scales [block][a_stride]
  const uint8_t *b0, *b1;   // rows operand: gate and up weight, or x^T and null
  const float *b0_s, *b1_s; // 128 x 128 block scales [.., ..]; kWeight: b0_s = x^T's [block][b_stride]
  void *out0, *out1, *out2; // kGated: h, g, u; kInput: dx; kWeight: dw_gate, dw_up
  float *partials;          // [tile][part][128 x 128] in the lanes' order, parts > 1
  int64_t rows_a, rows_b;   // m, f | m, k | 2 f, k
  int64_t lda, ldb;
  int64_t a_stride, b_stride;
  int nkb;                  // blocks of the contraction
  int half;                 // kInput: blocks of the first weight
  int tiles_a, tiles_b, parts;
};

// Swizzle of a tile read transposed, rows of 128 or 256 bytes: the 16-byte chunk
// c of row r sits at slot c ^ swz_tr(r).  One transposed read touches 32 rows,
// 32 q + 8 t + 0..7 for q = 0..3; they spread over all banks, two to each.
template <int kRowBytes>
__device__ __forceinline__ int swz_tr(int r) {
  return kRowBytes == 128 ? ((r >> 1) & 3) | (((r >> 5) & 1) << 2) : (r & 7) | (((r >> 5) & 1) << 3);
}

typedef int i32x2 __attribute__((ext_vector_type(2)));

// 16 columns x 32 rows of bytes -> the lane's column, eight rows a read: within
// a quarter of the wave, lanes 2 r and 2 r + 1 address the 16 bytes of row r,
// and lane i receives column i of the eight rows.
template <int kRowBytes>
__device__ __forceinline__ i32x8 frag_transposed(const uint8_t *tile, int chunk, int fr, int fq) {
  const int r = 32 * fq + (fr >> 1);   // rows r + 8 t share r's swizzle
  const uint8_t *lane_base = tile + r * kRowBytes + ((chunk ^ swz_tr<kRowBytes>(r)) << 4) + 8 * (fr & 1);
  i32x8 v;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (__attribute__((address_space(3))) i32x2 *)(uintptr_t)lds_addr(lane_base + t * 8 * kRowBytes));
    v[2 * t] = w.x;
    v[2 * t + 1] = w.y;
  }
  return v;
}

// A scale that no kernel of this library writes while one reads it: loaded
// through the scalar cache, which vector-memory waits do not count.
__device__ __forceinline__ float load_uniform(const float *p, int64_t i) {
  return *(const __attribute__((address_space(4))) float *)(uintptr_t)(p + i);
}

__device__ __forceinline__ int exponent_of(float pow2) { return (int)((__float_as_uint(pow2) >> 23) & 0xFFu); }

// silu(g) * u; the reciprocal instruction is within one ulp; the exponential
// overflows to infinity for g below -88, where the sigmoid is 0 to fp32's
// precision.
__device__ __forceinline__ float gated(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Row `row` of a tile with `left` rows of the matrix from its first (at least
// one): rows past the matrix re-read its last.
__device__ __forceinline__ uint32_t tile_row(int row, int64_t left) {
  return (uint32_t)min(row, (int)min(left, (int64_t)kBlock * 2) - 1);
}

// Four consecutive outputs of a row: one store (kVec; the row has all four), or
// one each for the `left` that are inside the row.
template <bool kBf16Out, bool kVec>
__device__ __forceinline__ void store4(void *p, int64_t idx, f32x4 v, int left) {
  if (kVec && kBf16Out) {
    *(u32x2 *)((uint16_t *)p + idx) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  } else if (kVec) {
    *(f32x4 *)((float *)p + idx) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) store_out(p, kBf16Out, idx + e, v[e]);
  }
}

// h, and with them g and u, of four consecutive features.
template <bool kBf16Out, bool kVec>
__device__ __forceinline__ void store_gated(void *h, void *g_out, void *u_out, int64_t idx, f32x4 g, f32x4 u, int left) {
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = gated(g[e], u[e]);
  store4<kBf16Out, kVec>(h, idx, v, left);
  if (g_out) {
    store4<kBf16Out, kVec>(g_out, idx, g, left);
    store4<kBf16Out, kVec>(u_out, idx, u, left);
  }
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles.
//
// Workgroup: 512 threads = 8 waves, 4 x 2, a wave 64 columns by 128 rows (4 x 8
// MFMA tiles, two waves per SIMD).  kGated's 256 rows are 128 features of both
// projections: in each half 64 gate rows and the 64 up rows of the same
// features, so gate accumulators (row tiles 0..3) and up accumulators (4..7) of
// an output sit in one lane.
//
// Operands reach a two-stage LDS ring by direct global->LDS transfers (block
// kb + 1 is loaded while kb is computed), issued where the block-scaled GEMM
// measured them cheapest: the columns' 32 by waves 0-3 at the top of the block,
// the rows' 32 by all waves after their first MFMAs.  The rescale of an MFMA's
// partial runs three MFMAs behind it.
//
// Persistent: one workgroup per CU walks the tiles, and a tile's first transfers
// go out before the previous tile's stores.
//
// Measured: kGated 8192 x 18432 x 7168 with g and u stored 1.85-1.95 ms, 2.2-2.3
// PFLOP/s (the first, simple kernel: 11.2 ms).  The matrix cores are busy 59% of the cycles, at 1.6-1.8
// GHz: under this load the clock, not a queue, gives way, so that evening out
// the last round or moving the transfers changes little.
// ---------------------------------------------------------------------------
constexpr int kBigTile = 256, kBigThreads = 512;

struct BigSmem {
  uint8_t a[2][kBigTile * kBlock];
  uint8_t b[2][kBigTile * kBlock];
  float as[2][kBigTile], bs[2][kBigTile];
};

// Tile of workgroup turn `it`: workgroups are dealt round-robin to the eight
// XCDs, so turns it, it + 8, ... get consecutive tiles of one XCD's contiguous
// share (they then share its L2); tiles run in groups of four column tiles
// across the row tiles.
__device__ __forceinline__ void big_tile_coords(int it, int tiles_a, int tiles_b, int &ta, int &tb) {
  const int ntiles = tiles_a * tiles_b, base = ntiles / 8, rest = ntiles % 8, xcd = it % 8;
  const int tile = xcd * base + min(xcd, rest) + it / 8;
  constexpr int kGroup = 4;
  const int group = tile / (kGroup * tiles_b), first = group * kGroup;
  const int ga = min(tiles_a - first, kGroup), idx = tile - group * kGroup * tiles_b;
  ta = first + idx % ga;
  tb = idx / ga;
}

// The workgroup's tiles: position it = start, then next(it), below p's count.
template <TileMode kMode, bool kMx, bool kBf16Out, bool kVec, typename Next>
__device__ __forceinline__ void big_tiles(const TileArgs &p, BigSmem &sm, int start, Next next) {
  static_assert(kMode == TileMode::kGated || kMx, "gradient scales are powers of two");
  constexpr bool kGatedMode = kMode == TileMode::kGated, kInputMode = kMode == TileMode::kInput;
  constexpr bool kWeightMode = kMode == TileMode::kWeight;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = p.nkb, ntiles = p.tiles_a * p.tiles_b;
  const int wa = (wave >> 1) * 64, wb = wave & 1;   // wave's columns, and half of the rows
  const int fr = lane & 15, fq = lane >> 4;
  // transfers: lane p of an 8-row group fills chunk slot p % 8 of row p / 8;
  // columns' group 8 d + g by wave d < 4, rows' group 4 w + i by every wave w
  // (transposed rows are 256 bytes: groups of four, slot p % 16 of row p / 16)
  const bool dma_wave = wave < 4;
  const int dw = wave & 3, dr = lane >> 3, ds = lane & 7;
  const uint32_t lds_a = lds_addr(&sm.a[0][0]), lds_b = lds_addr(&sm.b[0][0]);
  const uint32_t lds_as = lds_addr(&sm.as[0][0]), lds_bs = lds_addr(&sm.bs[0][0]);
  const uint32_t s_off = (uint32_t)lane * 4;

  uint32_t a_off[8], b_off[4];   // from the tile's own base
  const uint8_t *a_base = nullptr, *b_base = nullptr;
  const float *as_base = nullptr, *bs_base = nullptr;
  auto set_offsets = [&](int64_t a0, int64_t b0) {   // rows past an edge re-read the last one
    a_base = p.a + a0 * p.lda;
    b_base = kInputMode ? p.b0 + b0 : (kGatedMode && (wave & 2) ? p.b1 : p.b0) + b0 * p.ldb;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const int row = 8 * (8 * dw + g) + dr;
      a_off[g] = tile_row(row, p.rows_a - a0) * (uint32_t)p.lda + ((ds ^ swz(row)) << 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kInputMode) {   // 128 features x 256 of the weights' columns
        const int row = 4 * (4 * wave + i) + (lane >> 4);
        const int col = ((lane & 15) ^ swz_tr<256>(row)) << 4;
        b_off[i] = row * (uint32_t)p.ldb + tile_row(col, p.rows_b - 15 - b0);
      } else {
        const int row = 8 * (4 * wave + i) + dr;   // kGated: half row / 128, projection (row / 64) % 2
        const int r = kGatedMode ? (row >> 7) * 64 + (row & 63) : row;
        b_off[i] = tile_row(r, p.rows_b - b0) * (uint32_t)p.ldb + ((ds ^ swz(row)) << 4);
      }
    }
    as_base = p.a_s + a0 + 64 * dw;
    // the last tile's second half may lie past the matrix: any rows' scales do there
    if (kWeightMode) bs_base = p.b0_s + min(b0 + 64 * dw, p.rows_b - 64);
  };
  auto issue_a = [&](int kb, int s) {
    const uint8_t *ab = a_base + (int64_t)kb * kBlock;
#pragma unroll
    for (int g = 0; g < 8; ++g) lds_dma16(ab, a_off[g], lds_a + s * (kBigTile * kBlock) + (8 * dw + g) * 1024);
    lds_dma4(as_base + (int64_t)kb * p.a_stride, s_off, lds_as + s * (kBigTile * 4) + dw * 256);
  };
  auto issue_b = [&](int kb, int s) {
    const uint8_t *bb;
    if (kInputMode)   // b1 - b0 leads from the first weight to the second
      bb = b_base + (kb < p.half ? 0 : p.b1 - p.b0) + (int64_t)(kb < p.half ? kb : kb - p.half) * kBlock * p.ldb;
    else
      bb = b_base + (int64_t)kb * kBlock;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      lds_dma16(bb, b_off[i], lds_b + s * (kBigTile * kBlock) + (4 * wave + i) * 1024);
    if (kWeightMode && !dma_wave)
      lds_dma4(bs_base + (int64_t)kb * p.b_stride, s_off, lds_bs + s * (kBigTile * 4) + dw * 256);
  };

  bool prologue_done = false;
  for (int it = start, following; it < ntiles; it = following) {
    following = next(it);
    int ta, tb;
    big_tile_coords(it, p.tiles_a, p.tiles_b, ta, tb);
    const int64_t a0 = (int64_t)ta * kBigTile, b0 = (int64_t)tb * (kGatedMode ? kBigTile / 2 : kBigTile);
    // kInput: the wave's 128 columns of the weights lie in one block column
    const int64_t wcol = min(b0 / kBlock + wb, p.rows_b / kBlock - 1);
    if (!prologue_done && nkb > 0) {
      set_offsets(a0, b0);
      if (dma_wave) issue_a(0, 0);
      issue_b(0, 0);
    }
    const bool stage0_landed = prologue_done;

    f32x4 acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 prt[4];
    float sc[2][4];   // column scale * weight scale, per projection
#pragma unroll
    for (int q = 0; q < 4; ++q) prt[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[0][i] = sc[1][i] = 0.f;
    auto rescale = [&](int qp) {   // MFMA qp = 4 j + i
      const int ip = qp % 4, jp = qp / 4;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[ip][jp][e] = __builtin_fmaf(prt[qp % 4][e], sc[kGatedMode ? jp / 4 : 0][kMx ? 0 : ip], acc[ip][jp][e]);
    };

    auto step = [&](int kb, int cur, bool landed) {
      float w0 = 0.f, w1 = 0.f;
      if (kGatedMode) {
        w0 = load_uniform(p.b0_s, (int64_t)tb * nkb + kb);
        w1 = load_uniform(p.b1_s, (int64_t)tb * nkb + kb);
      } else if (kInputMode) {
        w0 = load_uniform(kb < p.half ? p.b0_s : p.b1_s,
                          (int64_t)(kb < p.half ? kb : kb - p.half) * (p.rows_b / kBlock) + wcol);
      }
      if (!landed) {
        wait_dma_all();
        workgroup_barrier();   // stage cur landed for every wave; stage cur ^ 1 no longer read
      }
      if (dma_wave && kb + 1 < nkb) issue_a(kb + 1, cur ^ 1);
      // retire the scalar loads now: while one is outstanding every LDS wait
      // would be a full drain
      if (!kWeightMode) asm volatile("" ::"s"(w0), "s"(w1));
      float sa[4], sb[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) sa[i] = sm.as[cur][wa + 16 * i + fr];
      if (kWeightMode) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sb[j] = sm.bs[cur][wb * 128 + 16 * j + fr];
      }
      auto read_b = [&](int j) {
        if (kInputMode) return frag_transposed<256>(sm.b[cur], 8 * wb + j, fr, fq);
        const int r = wb * 128 + 16 * j + fr;
        return frag_from_lds(&sm.b[cur][r * kBlock], fq, r);
      };
      i32x8 bcur = read_b(0), bnext;
      __builtin_amdgcn_sched_barrier(0);
      i32x8 af[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = wa + 16 * i + fr;
        af[i] = frag_from_lds(&sm.a[cur][r * kBlock], fq, r);
        __builtin_amdgcn_sched_barrier(0);
      }
      // the previous block's last rescale, while these reads are in flight
      if (!kWeightMode) {
#pragma unroll
        for (int qp = 29; qp < 32; ++qp) rescale(qp);
      }
      int ea[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ea[i] = exponent_of(sa[i]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j + 1 < 8) bnext = read_b(j + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = 4 * j + i;
          if (kWeightMode)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bcur, af[i], acc[i][j], 0, 0, 0,
                                                                         exponent_of(sb[j]), 0, ea[i]);
          else if (kMx)
            prt[q % 4] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                bcur, af[i], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, ea[i]);
          else
            prt[q % 4] = mfma_e4m3_16x16x128(bcur, af[i], f32x4{0.f, 0.f, 0.f, 0.f});
          // unconditional, so that no branch splits the unrolled loop (the last
          // block re-reads itself into the stage no one reads again)
          if (j == 2 && i == 0) issue_b(min(kb + 1, nkb - 1), cur ^ 1);
          if (!kWeightMode) {
            if (q == 3) {
#pragma unroll
              for (int r = 0; r < (kMx ? 1 : 4); ++r) {
                sc[0][r] = kMx ? w0 : sa[r] * w0;
                sc[1][r] = kMx ? w1 : sa[r] * w1;
              }
            }
            if (q >= 3) rescale(q - 3);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if (j + 1 < 8) bcur = bnext;
      }
    };
#pragma nounroll
    for (int kb = 0; kb < nkb; ++kb) step(kb, kb & 1, kb == 0 && stage0_landed);
    if (!kWeightMode) {
#pragma unroll
      for (int qp = 29; qp < 32; ++qp) rescale(qp);
    }
    wait_dma_all();

    // the next tile's first transfers go out, and are waited for, before this
    // tile's stores, which then drain while that tile computes
    prologue_done = false;
    if (following < ntiles && nkb > 0) {
      workgroup_barrier();
      int nta, ntb;
      big_tile_coords(following, p.tiles_a, p.tiles_b, nta, ntb);
      set_offsets((int64_t)nta * kBigTile, (int64_t)ntb * (kGatedMode ? kBigTile / 2 : kBigTile));
      if (dma_wave) issue_a(0, 0);
      issue_b(0, 0);
      wait_dma_all();
      workgroup_barrier();
      prologue_done = true;
    }

#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = a0 + wa + 16 * i + fr;
      if (row >= p.rows_a) continue;
      if (kGatedMode) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t col = b0 + 64 * wb + 16 * j + 4 * fq;
          if (col < p.rows_b)
            store_gated<kBf16Out, kVec>(p.out0, p.out1, p.out2, row * p.rows_b + col, acc[i][j], acc[i][j + 4],
                                        (int)min((int64_t)4, p.rows_b - col));
        }
      } else if (b0 + 128 * wb < p.rows_b) {   // whole blocks of 128 columns
        const int64_t f = p.rows_a / 2;
        const bool second = kWeightMode && row >= f;
        const int64_t at = (second ? row - f : row) * p.rows_b + b0 + 128 * wb + 4 * fq;
#pragma unroll
        for (int j = 0; j < 8; ++j) store4<kBf16Out, true>(second ? p.out1 : p.out0, at + 16 * j, acc[i][j], 4);
      }
    }
  }
}

template <TileMode kMode, bool kMx, bool kBf16Out, bool kVec>
__global__ __launch_bounds__(kBigThreads) void e4m3_big_kernel(const TileArgs p) {
  __shared__ __attribute__((aligned(1024))) BigSmem sm;
  big_tiles<kMode, kMx, kBf16Out, kVec>(p, sm, blockIdx.x, [](int it) { return it + (int)gridDim.x; });
}

// ---------------------------------------------------------------------------
// 128 x 128 tiles.
//
// Workgroup: 384 threads = 4 compute waves, 2 x 2, a wave 64 x 64 (4 x 4 MFMA
// tiles, one wave per SIMD), and two movers, one per operand, that issue all
// global->LDS transfers (with the scales) into a four-slot ring, three blocks
// of 128 ahead: with one workgroup per CU that is 96 KB in flight, what it takes
// to cover the latency at these sizes.  A transfer instruction holds its wave
// until the CU accepts it (16-18 cycles each, 36 a block); issued by the compute
// waves they cost more than the block's MFMAs.  A block's fragments are read to
// registers while the block before it feeds the MFMAs; one barrier per block
// hands the ring on.
//
// Split contraction: `parts` workgroups share a tile and store FP32 partials; a
// second kernel adds them in part order and finishes the tile.  (Finished by the
// last part to arrive, behind device-scope stores and a counter, the same split
// took 4 us longer at 211 x 2300 x 7168: one workgroup then reads all parts.)
//
// Measured there: 18.5 us, and 4 for the sums, for 72 tiles of 56 blocks, which
// bring 132 MB to LDS (35 MB of them new).  64 x 18432 x 7168: 75-81 us for 264
// MB, two rounds of tiles, the second an eighth full.
// ---------------------------------------------------------------------------
constexpr int kMidTile = 128, kMidThreads = 384, kMidSlots = 4;
constexpr int kMidPartsMax = 16;

struct MidSlot {
  uint8_t a[kMidTile * kBlock];
  uint8_t b[kMidTile * kBlock];
  float as[kMidTile], bs[kMidTile];
};

// Column tile i of wave `wave` (column half wave / 2, row half wave % 2): where
// its row tiles' partials lie, 256 floats apart, and how it is finished.
__device__ __forceinline__ float *mid_partial(const TileArgs &p, int tile, int part, int wave, int i, int lane) {
  return p.partials + ((size_t)tile * p.parts + part) * (kMidTile * kMidTile) + wave * 4096 + i * 1024 + lane * 4;
}

template <TileMode kMode, bool kBf16Out, bool kVec>
__device__ __forceinline__ void mid_finish(const TileArgs &p, int ta, int tb, int wave, int i, int lane,
                                           const f32x4 (&acc)[4]) {
  const int fr = lane & 15, fq = lane >> 4, wb = wave & 1;
  const int64_t row = (int64_t)ta * kMidTile + (wave >> 1) * 64 + 16 * i + fr;
  if (row >= p.rows_a) return;
  if (kMode == TileMode::kGated) {   // row tiles gate 0, 1, up 0, 1
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t col = (int64_t)tb * (kMidTile / 2) + 32 * wb + 16 * j + 4 * fq;
      if (col < p.rows_b)
        store_gated<kBf16Out, kVec>(p.out0, p.out1, p.out2, row * p.rows_b + col, acc[j], acc[j + 2],
                                    (int)min((int64_t)4, p.rows_b - col));
    }
  } else {
    const int64_t f = p.rows_a / 2;
    const bool second = kMode == TileMode::kWeight && row >= f;
    const int64_t at = (second ? row - f : row) * p.rows_b + (int64_t)tb * kMidTile + 64 * wb + 4 * fq;
#pragma unroll
    for (int j = 0; j < 4; ++j) store4<kBf16Out, true>(second ? p.out1 : p.out0, at + 16 * j, acc[j], 4);
  }
}

// kMx: the columns' scales are powers of two and go into the MFMA.
// Workgroup `block` of the `total` that the product takes.
template <TileMode kMode, bool kMx, bool kBf16Out, bool kVec>
__device__ __forceinline__ void mid_tile(const TileArgs &p, int block, int total, MidSlot *ring) {
  static_assert(kMode == TileMode::kGated || kMx, "gradient scales are powers of two");
  constexpr bool kGatedMode = kMode == TileMode::kGated, kInputMode = kMode == TileMode::kInput;
  constexpr bool kWeightMode = kMode == TileMode::kWeight;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fq = lane >> 4, dr = lane >> 3, ds = lane & 7;
  const int wa = (wave >> 1) * 64, wb = wave & 1;   // wave's columns, and half of the rows

  // XCD x (workgroups are dealt to the eight round-robin) takes a contiguous
  // share of the order part, row tile, column tile: neighbours share weights
  const int xcd = block % 8;
  const int lin = xcd * (total / 8) + min(xcd, total % 8) + block / 8;
  const int ta = lin % p.tiles_a, tb = lin / p.tiles_a % p.tiles_b, part = lin / (p.tiles_a * p.tiles_b);
  const int per = (p.nkb + p.parts - 1) / p.parts;
  const int kb0 = min(p.nkb, part * per), kb1 = min(p.nkb, kb0 + per);

  const int64_t a0 = (int64_t)ta * kMidTile;
  const int64_t b0 = (int64_t)tb * (kGatedMode ? kMidTile / 2 : kMidTile);
  if (wave >= 4) {
    // movers: lane p of an 8-row group fills chunk slot p % 8 of row p / 8; rows
    // past an edge re-read the last one
    const bool rows_mover = wave == 5;
    uint32_t off[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = 8 * i + dr;
      if (!rows_mover)
        off[i] = tile_row(row, p.rows_a - a0) * (uint32_t)p.lda + ((ds ^ swz(row)) << 4);
      else if (kGatedMode)   // half row / 64, projection (row / 32) % 2
        off[i] = tile_row((row >> 6) * 32 + (row & 31), p.rows_b - b0) * (uint32_t)p.ldb + ((ds ^ swz(row)) << 4);
      else
        off[i] = row * (uint32_t)p.ldb + ((ds ^ (kInputMode ? swz_tr<kBlock>(row) : swz(row))) << 4);
    }
    const uint32_t lds_ring = lds_addr(&ring[0]) + (rows_mover ? kMidTile * kBlock : 0);
    const uint32_t s_off = (uint32_t)lane * 4;
    constexpr int kDmaA = 18, kDmaB = kWeightMode ? 18 : 16;   // transfers per block
    static_assert(3 * kDmaA < 64, "the wait counter's range");
    auto issue = [&](int kb) {   // past the end: the last block again, so that every block counts the same
      const uint32_t slot = lds_ring + (uint32_t)((kb - kb0) % kMidSlots) * (uint32_t)sizeof(MidSlot);
      const int kc = min(kb, kb1 - 1);
      if (!rows_mover) {
        const uint8_t *base = p.a + a0 * p.lda + (int64_t)kc * kBlock;
#pragma unroll
        for (int i = 0; i < 16; ++i) lds_dma16(base, off[i], slot + i * 1024);
        const float *s = p.a_s + a0 + (int64_t)kc * p.a_stride;
        lds_dma4(s, s_off, slot + 2 * kMidTile * kBlock);
        lds_dma4(s + 64, s_off, slot + 2 * kMidTile * kBlock + 256);
      } else {
        const uint8_t *base = p.b0 + (kInputMode ? b0 : b0 * p.ldb), *base1 = nullptr;
        if (kInputMode)   // b1 - b0 leads from the first weight to the second
          base += (kc < p.half ? 0 : p.b1 - p.b0) + (int64_t)(kc < p.half ? kc : kc - p.half) * kBlock * p.ldb;
        else
          base += (int64_t)kc * kBlock;
        if (kGatedMode) base1 = base + (p.b1 - p.b0);
#pragma unroll
        for (int i = 0; i < 16; ++i) lds_dma16(kGatedMode && (i & 4) ? base1 : base, off[i], slot + i * 1024);
        if (kWeightMode) {
          const float *s = p.b0_s + b0 + (int64_t)kc * p.b_stride;
          lds_dma4(s, s_off, slot + kMidTile * kBlock + kMidTile * 4);
          lds_dma4(s + 64, s_off, slot + kMidTile * kBlock + kMidTile * 4 + 256);
        }
      }
    };
    auto wait_behind2 = [&]() {   // all but the two youngest blocks landed
      if (rows_mover)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kDmaB) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kDmaA) : "memory");
    };
    if (kb0 < kb1) {
      issue(kb0);
      issue(kb0 + 1);
      issue(kb0 + 2);
      wait_behind2();
      workgroup_barrier();
      for (int kb = kb0; kb < kb1; ++kb) {
        issue(kb + 3);   // into the slot of kb - 1, whose reads ended before the last barrier
        wait_behind2();  // kb + 1 landed
        workgroup_barrier();
      }
      wait_dma_all();   // transfers past the end, before the workgroup's LDS is released
    }
    return;
  }

  f32x4 acc[4][4];   // [column tile][row tile]; kGated: row tiles gate 0, 1, up 0, 1
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Block {
    i32x8 a[4], b[4];
    float sa[4], sb[4], w[2];   // column scales; kWeight: row scales; weight block scales
  };
  auto load_scales = [&](int kb, Block &v) {
    const int kc = min(kb, kb1 - 1);
    if (kGatedMode) {
      v.w[0] = load_uniform(p.b0_s, (b0 / kBlock) * p.nkb + kc);
      v.w[1] = load_uniform(p.b1_s, (b0 / kBlock) * p.nkb + kc);
    } else if (kInputMode) {
      v.w[0] = v.w[1] = load_uniform(kc < p.half ? p.b0_s : p.b1_s, (int64_t)(kc < p.half ? kc : kc - p.half) * p.tiles_b + tb);
    }
  };
  auto read = [&](int kb, Block &v) {
    const MidSlot &s = ring[(kb - kb0) % kMidSlots];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kInputMode) {
        v.b[j] = frag_transposed<kBlock>(s.b, 4 * wb + j, fr, fq);
      } else {
        const int r = 64 * wb + 16 * j + fr;
        v.b[j] = frag_from_lds(&s.b[r * kBlock], fq, r);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = wa + 16 * i + fr;
      v.a[i] = frag_from_lds(&s.a[r * kBlock], fq, r);
      v.sa[i] = s.as[wa + 16 * i + fr];
      v.sb[i] = kWeightMode ? s.bs[64 * wb + 16 * i + fr] : 1.0f;
    }
  };
  auto compute = [&](const Block &v) {
    if (kWeightMode) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v.b[j], v.a[i], acc[i][j], 0, 0, 0,
                                                                       exponent_of(v.sb[j]), 0, exponent_of(v.sa[i]));
      return;
    }
    // the rescale of an MFMA's partial runs three MFMAs behind it
    f32x4 prt[4];
    auto rescale = [&](int q) {
      const int i = q % 4, j = q / 4;
      const float w = v.w[kGatedMode ? j / 2 : 0], sc = kMx ? w : v.sa[i] * w;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(prt[q % 4][e], sc, acc[i][j][e]);
    };
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int i = q % 4, j = q / 4;
      prt[q % 4] = kMx ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                             v.b[j], v.a[i], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, exponent_of(v.sa[i]))
                       : mfma_e4m3_16x16x128(v.b[j], v.a[i], f32x4{0.f, 0.f, 0.f, 0.f});
      if (q >= 3) rescale(q - 3);
    }
#pragma unroll
    for (int q = 13; q < 16; ++q) rescale(q);
  };
  auto step = [&](int kb, const Block &cur, Block &next) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // block kb's reads ended: its slot may be refilled
    workgroup_barrier();                                 // kb + 1 landed
    read(kb + 1, next);   // all of it goes out before the MFMAs, which cover it
    load_scales(kb + 1, next);
    __builtin_amdgcn_sched_barrier(0);
    compute(cur);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (kb0 < kb1) {
    Block even, odd;
    workgroup_barrier();
    read(kb0, even);
    load_scales(kb0, even);
    int kb = kb0;
#pragma nounroll
    for (; kb + 1 < kb1; kb += 2) {
      step(kb, even, odd);
      step(kb + 1, odd, even);
    }
    if (kb < kb1) {
      workgroup_barrier();   // the movers' last
      compute(even);
    }
  }

  const int tile = tb * p.tiles_a + ta;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.parts > 1) {
      float *out = mid_partial(p, tile, part, wave, i, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) *(f32x4 *)(out + j * 256) = acc[i][j];
    } else {
      mid_finish<kMode, kBf16Out, kVec>(p, ta, tb, wave, i, lane, acc[i]);
    }
  }
}

template <TileMode kMode, bool kMx, bool kBf16Out, bool kVec>
__global__ __launch_bounds__(kMidThreads) void e4m3_mid_kernel(const TileArgs p) {
  __shared__ __attribute__((aligned(1024))) MidSlot ring[kMidSlots];
  mid_tile<kMode, kMx, kBf16Out, kVec>(p, blockIdx.x, gridDim.x, ring);
}

// Adds a tile's partials in part order: block 4 tile + i the column tiles i of
// the tile's four waves (256 threads).
template <TileMode kMode, bool kBf16Out, bool kVec>
__device__ __forceinline__ void mid_reduce(const TileArgs &p, int block) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = block >> 2, i = block & 3;
  f32x4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = *(const f32x4 *)(mid_partial(p, tile, 0, wave, i, lane) + j * 256);
#pragma unroll 4
  for (int q = 1; q < p.parts; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += *(const f32x4 *)(mid_partial(p, tile, q, wave, i, lane) + j * 256);
  mid_finish<kMode, kBf16Out, kVec>(p, tile % p.tiles_a, tile / p.tiles_a, wave, i, lane, acc);
}

template <TileMode kMode, bool kBf16Out, bool kVec>
__global__ __launch_bounds__(256) void e4m3_reduce_kernel(const TileArgs p) {
  mid_reduce<kMode, kBf16Out, kVec>(p, blockIdx.x);
}

// How a product of `nkb` blocks is launched: 256 x 256 tiles, or 128 x 128
// tiles with the contraction in `parts`.
struct TilePlan {
  bool big = true;
  int tiles_a = 0, tiles_b = 0, parts = 1;
  size_t partial_bytes = 0;

  void fill(TileArgs &a) const {
    a.tiles_a = tiles_a;
    a.tiles_b = tiles_b;
    a.parts = parts;
  }
};

// The cheaper of the two by their time on a CU: a round of tiles takes so much
// per block of 128 and so much besides, and a split product's second kernel so
// much more.  Measured (gated_ffn, us, 256 against 128 tiles): 2048 x 2048 x 2048
// 34 and 37, 4096 x 1024 x 1024 23 and 28, 512 x 4096 x 4096 49 and 28,
// 700 x 1000 x 896 17 and 12; 211 x 2300 x 7168 76, 38 and 25 in three parts,
// 300 x 640 x 4096 49, 26 and 21 in eight.
constexpr double kBigBlockUs = 1.65, kBigRoundUs = 8.0, kMidBlockUs = 0.65, kMidRoundUs = 7.5, kSplitUs = 5.0;

// cols: rows of the columns operand; rows: rows of the rows operand in tiles of
// row_tile (of a 256 x 256 tile; half that in a 128 x 128 one).
inline TilePlan tile_plan(int64_t cols, int64_t rows, int row_tile, int nkb, int cus) {
  auto ceil_div = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  if (cus <= 0) cus = 256;
  TilePlan big, mid;
  big.tiles_a = (int)ceil_div(cols, kBigTile);
  big.tiles_b = (int)ceil_div(rows, row_tile);
  const double big_us = (double)ceil_div((int64_t)big.tiles_a * big.tiles_b, cus) * (nkb * kBigBlockUs + kBigRoundUs);
  mid.big = false;
  mid.tiles_a = (int)ceil_div(cols, kMidTile);
  mid.tiles_b = (int)ceil_div(rows, row_tile / 2);
  const int64_t tiles = (int64_t)mid.tiles_a * mid.tiles_b;
  if (tiles == 0) return big;   // nothing to launch
  double mid_us = (double)ceil_div(tiles, cus) * (nkb * kMidBlockUs + kMidRoundUs);
  // fill the CUs once; four blocks a part at least, or the ring never runs full
  const int64_t most = min(min((int64_t)cus / tiles, (int64_t)nkb / 4), (int64_t)kMidPartsMax);
  if (most >= 2) {
    const int per = (int)ceil_div(nkb, most);
    const int parts = (int)ceil_div(nkb, per);   // parts that get any, as the kernel divides them
    const double split_us = per * kMidBlockUs + kMidRoundUs + kSplitUs;
    if (parts >= 2 && split_us < mid_us) {
      mid_us = split_us;
      mid.parts = parts;
      mid.partial_bytes = (size_t)tiles * parts * kMidTile * kMidTile * sizeof(float);
    }
  }
  return mid_us < big_us ? mid : big;
}

// Launch by plan.  a.partials: the plan's bytes, if any.  kVec: every four
// outputs of a row make one aligned store.
template <TileMode kMode, bool kMx, bool kBf16Out, bool kVec>
inline hipError_t launch_tiles(const TilePlan &plan, TileArgs a, int cus, hipStream_t stream) {
  if (cus <= 0) cus = 256;
  plan.fill(a);
  const int64_t tiles = (int64_t)plan.tiles_a * plan.tiles_b;
  if (plan.big) {
    const dim3 grid((unsigned)(tiles < cus ? tiles : cus));
    hipLaunchKernelGGL((e4m3_big_kernel<kMode, kMx, kBf16Out, kVec>), grid, dim3(kBigThreads), 0, stream, a);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(tiles * plan.parts));
  hipLaunchKernelGGL((e4m3_mid_kernel<kMode, kMx, kBf16Out, kVec>), grid, dim3(kMidThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.parts == 1) return e;
  hipLaunchKernelGGL((e4m3_reduce_kernel<kMode, kBf16Out, kVec>), dim3((unsigned)(tiles * 4)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8bsq
