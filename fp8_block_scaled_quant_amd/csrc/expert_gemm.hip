// Products of the experts' rows with their own block-scaled E4M3 weights, for
// gfx950: out[r] = a[r] W[e]^T for offsets[e] <= r < offsets[e + 1], or with two
// weights silu(a[r] Wg[e]^T) * (a[r] Wu[e]^T).  Each 128-wide K block's partial is
// multiplied by a_s[r, kb] * w_s[e, j / 128, kb] and added in FP32.
//
// How many rows an expert has is known on the device alone.  Every workgroup reads
// the offsets, works out the tiles of all experts, and takes its share of them;
// the launch depends on sizes only.  Within an expert the tiles of one piece of
// weight follow each other, so that it comes from HBM once.
//
// Three kernels: tiles of 16 or 64 rows by 128 rows of weights, with transfers many
// blocks ahead, for few rows an expert (bound by the weights' bytes); of 256 by 256,
// for many (bound by the matrix cores); and of 16 by 32 or 64, four K blocks at a
// time, where these are no more than the CUs (bound by the chain along K).
#include "device_cus.h"
#include "e4m3_tiles.h"
#include "expert_launch.h"

#include <math.h>
#include <type_traits>


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
  int tiles_f, blocks_f;    // tiles and 128-wide blocks of the features
  bool out_bf16;
};

// The experts' rows as the offsets give them, in order and inside the matrix
// whatever the offsets hold, and their token tiles' numbers.  These fit 16 bits: the
// rows make at most 65535 * 16 / 64 tiles of 64, and an expert one more; tiles of 16
// are taken up to eight rows an expert or some hundred tiles (product_shape).
struct Table {
  int *begin;        // [experts + 1] expert's first row; the last: where the rows behind begin
  uint16_t *first;   // [experts + 1] its first token tile; the last: their number

  __device__ __forceinline__ Table(uint8_t *at, int experts)
      : begin((int *)at), first((uint16_t *)(begin + experts + 1)) {}
  static constexpr size_t bytes(int64_t experts) { return (size_t)(experts + 1) * sizeof(int) + (size_t)(experts + 2) / 2 * 4; }
};

// The 256-row kernel's tiles of up to 128 rows, an expert's last, are a list of
// their own behind the others: they take half as long, and in one list some
// workgroups would get more of the long ones than others.
struct SplitTable {
  int begin[kMaxExperts + 1], first[kMaxExperts + 1];
  int half[kMaxExperts + 1];    // experts before with such a tile; the last: their number
};

__device__ __forceinline__ int wave_max_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v = max(v, o);
  }
  return v;
}

__device__ __forceinline__ int wave_sum_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// By all kThreads threads, kThreads experts at a time.
template <int kThreads, int kTokens, typename T>
__device__ __forceinline__ void build_table(const ProductArgs &p, T &t) {
  constexpr bool kSplit = std::is_same<T, SplitTable>::value;
  __shared__ int top[kThreads / 64], sum[kThreads / 64], halves[kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  auto inside = [&](int v) { return min(max(v, 0), (int)p.rows); };
  int rows_before = inside(p.offsets[0]), tiles_before = 0, halves_before = 0;
  for (int e0 = 0; e0 < p.experts; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    const int m = wave_max_scan(e < p.experts ? inside(p.offsets[e + 1]) : 0, lane);
    if (lane == 63) top[wave] = m;
    __syncthreads();
    int before = rows_before;
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) before = max(before, top[w]);
      rows_before = max(rows_before, top[w]);
    }
    const int prev = __shfl_up(m, 1), begin = lane ? max(prev, before) : before, end = max(m, before);
    const int tiles = (end - begin + (kSplit ? kTokens / 2 : kTokens) - 1) / kTokens;
    const int half = kSplit && end - begin > tiles * kTokens ? 1 : 0;
    const int s = wave_sum_scan(tiles, lane);
    const uint64_t with_half = __ballot(half);
    if (lane == 63) {
      sum[wave] = s;
      halves[wave] = __popcll(with_half);
    }
    __syncthreads();
    int at = tiles_before, half_at = halves_before;
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) {
        at += sum[w];
        half_at += halves[w];
      }
      tiles_before += sum[w];
      halves_before += halves[w];
    }
    if (e < p.experts) {
      t.begin[e] = begin;
      t.first[e] = at + s - tiles;
      if constexpr (kSplit) t.half[e] = half_at + __popcll(with_half & (((uint64_t)1 << lane) - 1));
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    t.begin[p.experts] = rows_before;
    t.first[p.experts] = tiles_before;
    if constexpr (kSplit) t.half[p.experts] = halves_before;
  }
  __syncthreads();
}

// A tile: `left` rows from row0, and the features from f0 (clipped at f).
struct Tile {
  int expert, row0, left;
  int64_t f0;
};

// The last expert whose entry is at most q: with prefix sums, the one that q is in.
// The same in every lane.
__device__ __forceinline__ int expert_of(const int *prefix, int experts, uint32_t q, int lane) {
  int e = 0;
  for (int e0 = 1; e0 <= experts; e0 += 64)
    e += __popcll(__ballot(e0 + lane <= experts && (uint32_t)prefix[min(e0 + lane, experts)] <= q));
  return __builtin_amdgcn_readfirstlane(e);
}

// Two entries a lane; entry 0, which is 0, always counts.
__device__ __forceinline__ int expert_of(const uint16_t *prefix, int experts, uint32_t q, int lane) {
  typedef uint32_t __attribute__((may_alias)) Pair;
  int e = -1;
  for (int e0 = 0; e0 <= experts; e0 += 128) {
    const int i = e0 + 2 * lane;
    const uint32_t two = ((const Pair *)prefix)[min(i, experts) / 2];
    e += __popcll(__ballot(i <= experts && (two & 0xFFFFu) <= q)) + __popcll(__ballot(i < experts && two >> 16 <= q));
  }
  return __builtin_amdgcn_readfirstlane(e);
}

// Position of turn `it` in a list: workgroups are dealt round-robin to the eight
// XCDs, so turns it, it + 8, ... get consecutive positions of one XCD's contiguous
// share (they then share its L2).
__device__ __forceinline__ uint32_t xcd_share(uint32_t it, uint32_t all) {
  const uint32_t xcd = it % 8;
  return xcd * (all / 8) + min(xcd, all % 8) + it / 8;
}

// Tile of turn `it` below `ntiles`.  An expert's tiles run in groups of four token
// tiles across the weights' tiles.
template <int kTokens, int kFeatures, typename T>
__device__ __forceinline__ Tile locate(const ProductArgs &p, const T &t, uint32_t it, uint32_t ntiles, int lane) {
  Tile r;
  uint32_t long_tiles = ntiles;
  if constexpr (std::is_same<T, SplitTable>::value) {
    long_tiles = (uint32_t)__builtin_amdgcn_readfirstlane(t.first[p.experts]) * (uint32_t)p.tiles_f;
    if (it >= long_tiles) {
      // the last expert first: its weights were read last, and may still be in a cache
      const uint32_t tile = xcd_share(it - long_tiles, ntiles - long_tiles), q = tile / (uint32_t)p.tiles_f;
      const uint32_t halves = (uint32_t)__builtin_amdgcn_readfirstlane(t.half[p.experts]);
      r.expert = expert_of(t.half, p.experts, halves - 1 - q, lane);
      const int tokens = __builtin_amdgcn_readfirstlane(t.first[r.expert + 1]) - __builtin_amdgcn_readfirstlane(t.first[r.expert]);
      r.row0 = __builtin_amdgcn_readfirstlane(t.begin[r.expert]) + tokens * kTokens;
      r.left = __builtin_amdgcn_readfirstlane(t.begin[r.expert + 1]) - r.row0;
      r.f0 = (int64_t)(tile - q * (uint32_t)p.tiles_f) * kFeatures;
      return r;
    }
  }
  const uint32_t tile = xcd_share(it, long_tiles);
  r.expert = expert_of(t.first, p.experts, tile / (uint32_t)p.tiles_f, lane);
  const int first = __builtin_amdgcn_readfirstlane(t.first[r.expert]);
  const uint32_t tokens = (uint32_t)(__builtin_amdgcn_readfirstlane(t.first[r.expert + 1]) - first);
  constexpr uint32_t kGroup = 4;
  const uint32_t rem = tile - (uint32_t)first * (uint32_t)p.tiles_f, group = rem / (kGroup * (uint32_t)p.tiles_f);
  const uint32_t across = min(tokens - group * kGroup, kGroup), idx = rem - group * kGroup * (uint32_t)p.tiles_f;
  const uint32_t tf = idx / across;
  r.row0 = __builtin_amdgcn_readfirstlane(t.begin[r.expert]) + (int)(group * kGroup + idx - tf * across) * kTokens;
  r.left = min(__builtin_amdgcn_readfirstlane(t.begin[r.expert + 1]) - r.row0, kTokens);
  r.f0 = (int64_t)tf * kFeatures;
  return r;
}

// Zeros in the rows behind the experts', by all workgroups' `threads` first threads.
__device__ __forceinline__ void clear_behind(const ProductArgs &p, int behind, int threads) {
  const int64_t size = p.out_bf16 ? 2 : 4;
  uint8_t *begin = (uint8_t *)p.out + behind * p.f * size, *end = (uint8_t *)p.out + p.rows * p.f * size;
  const int64_t self = (int64_t)blockIdx.x * threads + threadIdx.x, all = (int64_t)gridDim.x * threads;
  uint8_t *inner = (uint8_t *)(((uintptr_t)begin + 15) & ~(uintptr_t)15), *inner_end = (uint8_t *)((uintptr_t)end & ~(uintptr_t)15);
  if (inner >= inner_end) {   // a few elements
    for (int64_t i = self; i < (end - begin) / 2; i += all) ((uint16_t *)begin)[i] = 0;
    return;
  }
  for (int64_t i = self; i < (inner_end - inner) / 16; i += all) ((u32x4 *)inner)[i] = u32x4{0, 0, 0, 0};
  for (int64_t i = self; i < (inner - begin) / 2; i += all) ((uint16_t *)begin)[i] = 0;
  for (int64_t i = self; i < (end - inner_end) / 2; i += all) ((uint16_t *)inner_end)[i] = 0;
}

typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));

// Four consecutive outputs of a row, which may start on any element; one by one
// where they pass its end.
__device__ __forceinline__ void store_four(const ProductArgs &p, int64_t row, int64_t col, f32x4 v) {
  const int64_t at = row * p.f + col;
  if (col + 4 <= p.f) {
    if (p.out_bf16)
      *(u32x2_at2 *)((uint16_t *)p.out + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else
      *(f32x4_at4 *)((float *)p.out + at) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (col + e < p.f) store_out(p.out, p.out_bf16, at + e, v[e]);
}

// A row's outputs in two neighbouring 16-wide tiles, `col` the first's first.  bf16:
// eight consecutive ones a lane instead of four in each tile, so that a store covers
// 64 bytes of a row.  The swap leaves tile 0's columns in the even groups of 16 lanes
// and tile 1's in the odd ones.  (5300 rows of 6746, on any 2 bytes: 47 us, 98 with
// stores of one element.)
__device__ __forceinline__ void store_pair(const ProductArgs &p, bool there, int64_t row, int64_t col, int fq, f32x4 v0, f32x4 v1) {
  if (!p.out_bf16) {
    if (there && col + 4 * fq < p.f) store_four(p, row, col + 4 * fq, v0);
    if (there && col + 16 + 4 * fq < p.f) store_four(p, row, col + 16 + 4 * fq, v1);
    return;
  }
  const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16x2(v0[0], v0[1]), pack_bf16x2(v1[0], v1[1]), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16x2(v0[2], v0[3]), pack_bf16x2(v1[2], v1[3]), false, false);
  const u32x4 v = {lo[0], hi[0], lo[1], hi[1]};
  const int64_t first = col + 16 * (fq & 1) + 8 * (fq >> 1);
  uint16_t *to = (uint16_t *)p.out + row * p.f + first;
  if (there && first + 8 <= p.f) {
    *(u32x4_at2 *)to = v;
  } else if (there) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (first + e < p.f) to[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
  }
}

__device__ __forceinline__ f32x4 gated4(f32x4 g, f32x4 u) {
  f32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = gated(g[i], u[i]);
  return v;
}

// ---------------------------------------------------------------------------
// Few rows an expert: kTokens rows by 128 rows of weights.
//
// Four compute waves, and movers that issue all global->LDS transfers into a ring
// of kSlots blocks of 128, kSlots - 1 ahead, over the ends of tiles: a workgroup's
// blocks are one sequence.  One barrier a block hands the ring on.  Two workgroups a
// CU fill each other's waits, and keep 64 and 96 KB of weights in flight together,
// enough to stream them at HBM's rate (one workgroup with their LDS and fragments
// read a block ahead: 64 experts of 2300 x 1408 with 64 rows each 49 us for 40, 16 of
// 2 x 512 x 1024 with 8 rows 7.0 for 6.1, large weights the same).  So that they fit
// with 1024 experts too, the tables hold tile numbers of 16 bits and the ring starts on
// 128 bytes (1024 experts, two workgroups a CU and one: 64 rows each of 2 x 512 x 512
// 137 and 182 us, 48 of 2 x 256 x 1024 127 and 147, 8 of 2 x 512 x 1024 193 and 209; one
// row of 128 x 256, weights in the cache, 12 and 21).
//
// Measured: one token at eight experts of 2 x 2048 x 7168 43.3 us, 235 MB at 5.4 TB/s
// (a 1 GiB copy: 5.1; a wave per 16 features without LDS: 83 us); 8 rows each at 64
// experts 318 us, 1.9 GB at 6.0 TB/s; 66 rows each, unevenly, at 64 of 2300 x 1408 58
// us, 3.9 TB/s: experts above 64 rows take more tiles, 3.6 rounds of them.
// ---------------------------------------------------------------------------
constexpr int kStreamRows = 128;   // of weights, a tile
constexpr int kRingAlign = 128;    // whole rows; both kernels' rings are one symbol, and so of one alignment

template <int kTokens>
struct StreamShape {
  static constexpr int kSlots = kTokens == 64 ? 3 : 4;     // two workgroups' in a CU's LDS
  static constexpr int kMovers = kTokens == 64 ? 2 : 4;    // of weights; one more of a
  static constexpr int kThreads = 64 * (4 + kMovers + 1);
  static constexpr int kAcross = kTokens == 64 ? 2 : 4;    // compute waves along the weights' rows
  static constexpr int kI = kTokens / 16 / (4 / kAcross);  // MFMA tiles of a wave along the tokens,
  static constexpr int kJ = kStreamRows / 16 / kAcross;    // and along the weights
  static constexpr int kScales = 64;                       // a's, a block; those past the tile's rows are copies
  static constexpr int kSlotBytes = (kTokens + kStreamRows) * kBlock + kScales * 4;
  static constexpr int kDmaA = kTokens / 8 + 1, kDmaB = 16 / kMovers;   // transfers a block and mover
  static_assert((kSlots - 1) * (kDmaA > kDmaB ? kDmaA : kDmaB) < 64, "the wait counter's range");

  // of LDS that a launch asks for; the scan's, a place for each wave and three sums, is
  // the kernel's own
  static constexpr size_t lds(int64_t experts) { return (size_t)kSlots * kSlotBytes + Table::bytes(experts); }
  static_assert(3 * (kThreads / 64) * sizeof(int) <= kRingAlign && kSlotBytes % kRingAlign == 0 &&
                    2 * (lds(kMaxExperts) + kRingAlign) <= 160 * 1024, "two workgroups a CU");
};

template <bool kGated, int kTokens>
__global__ __launch_bounds__(StreamShape<kTokens>::kThreads, kTokens == 64 ? 4 : 5) void product_stream_kernel(const ProductArgs p) {
  using S = StreamShape<kTokens>;
  constexpr int kFeatures = kGated ? kStreamRows / 2 : kStreamRows;
  constexpr int kWaveRows = kStreamRows / S::kAcross;   // of weights, a compute wave; gated: gate's, then up's
  constexpr int kAhead = S::kSlots - 1;
  extern __shared__ __attribute__((aligned(kRingAlign))) uint8_t ring[];
  Table table(ring + S::kSlots * S::kSlotBytes, p.experts);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fq = lane >> 4, dr = lane >> 3, ds = lane & 7;
  build_table<S::kThreads, kTokens>(p, table);
  const uint32_t ntiles = (uint32_t)__builtin_amdgcn_readfirstlane(table.first[p.experts]) * (uint32_t)p.tiles_f;
  const int nkb = p.nkb;
  const uint32_t mine = blockIdx.x < ntiles ? (ntiles - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  const int64_t blocks = (int64_t)mine * nkb;
  auto tile_of = [&](uint32_t i) { return locate<kTokens, kFeatures>(p, table, blockIdx.x + i * gridDim.x, ntiles, lane); };

  if (wave >= 4) {
    // Movers: the first of a and its scales, the others of the weights.  Past the
    // end they issue the last block again, so that every block counts the same.
    if (blocks == 0) return;
    uint32_t turn = 0;
    int kb = 0, slot = 0;
    auto drive = [&](auto enter, auto issue, auto wait_landed) __attribute__((always_inline)) {
#pragma unroll 1
      for (int64_t s = 0; s < blocks + kAhead; ++s) {
        if (kb == 0) enter(tile_of(turn));
        issue((int64_t)kb, lds_addr(ring) + (uint32_t)slot * S::kSlotBytes);   // into the slot of block s - kSlots, whose reads ended before the last barrier
        slot = slot + 1 == S::kSlots ? 0 : slot + 1;
        if (kb + 1 < nkb) {
          ++kb;
        } else if (turn + 1 < mine) {
          ++turn;
          kb = 0;
        }
        if (s >= kAhead - 1) {
          wait_landed();   // all but the youngest kAhead - 1 blocks
          workgroup_barrier();
        }
      }
      wait_dma_all();   // transfers past the end, before the workgroup's LDS is released
    };
    // lane p of an 8-row group fills chunk slot p % 8 of row p / 8; rows past an
    // edge re-read the last one
    if (wave == 4) {
      uint32_t off[kTokens / 8], s_off = 0;
      const uint8_t *base = nullptr;
      const float *scales = nullptr;
      drive(
          [&](const Tile &t) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kTokens / 8; ++i) {
              const int row = 8 * i + dr;
              off[i] = (uint32_t)min(row, t.left - 1) * (uint32_t)p.k + ((ds ^ swz(row)) << 4);
            }
            s_off = (uint32_t)min(lane, t.left - 1) * (uint32_t)nkb * 4;
            base = p.a + (int64_t)t.row0 * p.k;
            scales = p.a_s + (int64_t)t.row0 * nkb;
          },
          [&](int64_t kb, uint32_t to) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kTokens / 8; ++i) lds_dma16(base + kb * kBlock, off[i], to + i * 1024);
            lds_dma4(scales + kb, s_off, to + (kTokens + kStreamRows) * kBlock);
          },
          [&]() __attribute__((always_inline)) { asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * S::kDmaA) : "memory"); });
    } else {
      const int group0 = (wave - 5) * S::kDmaB;   // of the weights' 16 groups of 8 rows
      uint32_t off[S::kDmaB];
      const uint8_t *base0 = nullptr, *base1 = nullptr;
      drive(
          [&](const Tile &t) __attribute__((always_inline)) {
            const int left = (int)min((int64_t)kFeatures, p.f - t.f0);
#pragma unroll
            for (int i = 0; i < S::kDmaB; ++i) {
              const int row = 8 * (group0 + i) + dr;
              const int feature = kGated ? row / kWaveRows * (kWaveRows / 2) + row % (kWaveRows / 2) : row;
              off[i] = (uint32_t)min(feature, left - 1) * (uint32_t)p.k + ((ds ^ swz(row)) << 4);
            }
            const int64_t at = ((int64_t)t.expert * p.f + t.f0) * p.k;
            base0 = p.w0 + at;
            base1 = kGated ? p.w1 + at : base0;
          },
          [&](int64_t kb, uint32_t to) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < S::kDmaB; ++i) {
              const bool up = kGated && (8 * (group0 + i) / (kWaveRows / 2) & 1);
              lds_dma16((up ? base1 : base0) + kb * kBlock, off[i], to + kTokens * kBlock + (group0 + i) * 1024);
            }
          },
          [&]() __attribute__((always_inline)) { asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * S::kDmaB) : "memory"); });
    }
    return;
  }

  const int wa = wave / S::kAcross * (S::kI * 16), wb = wave % S::kAcross;
  if (blocks > 0) {
    struct Block {
      i32x8 a[S::kI], b[S::kJ];
      float sa[S::kI], w[2];
    };
    f32x4 acc[S::kI][S::kJ];   // gated: row tiles gate's, then up's
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < S::kI; ++i)
#pragma unroll
        for (int j = 0; j < S::kJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    // the block read next, and the tile being computed
    uint32_t turn = 0;
    int kb = 0, slot = 0;
    Tile ahead = tile_of(0), tile = ahead;
    auto read = [&](Block &v) __attribute__((always_inline)) {
      const uint8_t *a = ring + slot * S::kSlotBytes, *b = a + kTokens * kBlock;
      const float *as = (const float *)(b + kStreamRows * kBlock);
      const int64_t at = ((int64_t)ahead.expert * p.blocks_f + ahead.f0 / kBlock) * nkb + kb;
      v.w[0] = load_uniform(p.w0_s, at);
      if (kGated) v.w[1] = load_uniform(p.w1_s, at);
#pragma unroll
      for (int j = 0; j < S::kJ; ++j) {
        const int r = kWaveRows * wb + 16 * j + fr;
        v.b[j] = frag_from_lds(b + r * kBlock, fq, r);
      }
#pragma unroll
      for (int i = 0; i < S::kI; ++i) {
        const int r = wa + 16 * i + fr;
        v.a[i] = frag_from_lds(a + r * kBlock, fq, r);
        v.sa[i] = as[r];
      }
      slot = slot + 1 == S::kSlots ? 0 : slot + 1;
      if (kb + 1 < nkb) {
        ++kb;
      } else if (turn + 1 < mine) {
        ++turn;
        kb = 0;
        ahead = tile_of(turn);
      }
    };
    auto compute = [&](const Block &v) __attribute__((always_inline)) {
      // the rescale of an MFMA's partial runs behind the next ones
      constexpr int kN = S::kI * S::kJ, kBehind = kN < 4 ? kN - 1 : 3;
      f32x4 prt[kBehind + 1];
      auto rescale = [&](int q) {
        const int i = q % S::kI, j = q / S::kI;
        const float sc = v.sa[i] * v.w[kGated && j >= S::kJ / 2 ? 1 : 0];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(prt[q % (kBehind + 1)][e], sc, acc[i][j][e]);
      };
#pragma unroll
      for (int q = 0; q < kN; ++q) {
        prt[q % (kBehind + 1)] = mfma_e4m3_16x16x128(v.b[q / S::kI], v.a[q % S::kI], f32x4{0.f, 0.f, 0.f, 0.f});
        if (q >= kBehind) rescale(q - kBehind);
      }
#pragma unroll
      for (int q = kN - kBehind; q < kN; ++q) rescale(q);
    };
    auto finish = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < S::kI; ++i) {
        if (wa + 16 * i >= tile.left) break;
        const int r = wa + 16 * i + fr;
        constexpr int kOut = kGated ? S::kJ / 2 : S::kJ;
        auto value = [&](int j) { return kGated ? gated4(acc[i][j], acc[i][(j + S::kJ / 2) % S::kJ]) : acc[i][j]; };
        const int64_t col = tile.f0 + (kGated ? kWaveRows / 2 : kWaveRows) * wb;
        if constexpr (kOut == 1) {
          if (r < tile.left && col + 4 * fq < p.f) store_four(p, tile.row0 + r, col + 4 * fq, value(0));
        } else {
#pragma unroll
          for (int j = 0; j < kOut; j += 2) store_pair(p, r < tile.left, tile.row0 + r, col + 16 * j, fq, value(j), value(j + 1));
        }
      }
    };
    Block v;
    clear();
#pragma nounroll
    for (int64_t s = 0; s < blocks; ++s) {
      workgroup_barrier();   // block s landed
      const bool last = kb + 1 == nkb;
      read(v);
      if (wa < tile.left) compute(v);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: its slot may be refilled
      if (last) {
        finish();
        clear();
        tile = ahead;   // the next block's
      }
    }
    workgroup_barrier();   // the movers' last
  }
  clear_behind(p, table.begin[p.experts], 256);
}

// ---------------------------------------------------------------------------
// Few tiles: 16 rows by 32 or 64 rows of weights (gated: of gate's and up's, half
// each), a workgroup a CU.
//
// With one tile a workgroup the time is a chain along K, and a CU takes data that is in
// no cache at some 55 GB/s at best.  So small tiles spread the weights over the CUs, and
// a step of the chain is four K blocks, one to each compute wave.  The waves' sums meet
// in LDS, always in the same order.  Four movers load a block of the step's weights
// each and a fifth a's, two steps ahead (32 rows: four), over the ends of tiles.  They
// go as the movers above do, and a fix to one loop belongs in both.
//
// Measured, weights from HBM (us; the kernel above): one row at each of 8 experts of
// 2 x 256 x 7168 11.0 (22.6; with 64 rows a tile 14.7), of 2 x 512 x 7168 14.4 (24.0),
// of 2 x 1024 x 7168 23.8, 64 rows a tile (27.3); one of 4096 x 4096 7.4 (11.2); 16 rows
// at each of 8 of 2 x 256 x 7168 12.4 (29.9), 128 rows at one of 2 x 512 x 7168 9.5 (25.6).
// ---------------------------------------------------------------------------
constexpr int kLongTokens = 16, kLongParts = 4, kLongThreads = 64 * (2 * kLongParts + 1);

template <int kRows>   // of weights, a tile
struct LongShape {
  static constexpr int kSlots = kRows == 64 ? 3 : 5;
  static constexpr int kJ = kRows / 16;   // MFMA tiles of a block
  static constexpr int kPartBytes = (kLongTokens + kRows) * kBlock + 64 * 4;
  static constexpr int kStepBytes = kLongParts * kPartBytes;
  static constexpr int kJoinBytes = kLongParts * kJ * 64 * (int)sizeof(f32x4);
  static constexpr int kDmaA = kLongParts * (kLongTokens / 8 + 1), kDmaB = kRows / 8;   // transfers a step and mover
  static_assert((kSlots - 1) * (kDmaA > kDmaB ? kDmaA : kDmaB) < 64, "the wait counter's range");
};

template <bool kGated, int kRows>
__global__ __launch_bounds__(kLongThreads) void product_long_kernel(const ProductArgs p) {
  using S = LongShape<kRows>;
  constexpr int kFeatures = kGated ? kRows / 2 : kRows;
  constexpr int kAhead = S::kSlots - 1;
  extern __shared__ __attribute__((aligned(kRingAlign))) uint8_t ring[];
  f32x4 *join = (f32x4 *)(ring + S::kSlots * S::kStepBytes);   // [part][16 rows of weights][lane]
  Table table(ring + S::kSlots * S::kStepBytes + S::kJoinBytes, p.experts);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fq = lane >> 4, dr = lane >> 3, ds = lane & 7;
  build_table<kLongThreads, kLongTokens>(p, table);
  const uint32_t ntiles = (uint32_t)__builtin_amdgcn_readfirstlane(table.first[p.experts]) * (uint32_t)p.tiles_f;
  const int nkb = p.nkb, steps = (nkb + kLongParts - 1) / kLongParts;
  const uint32_t mine = blockIdx.x < ntiles ? (ntiles - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  const int64_t all = (int64_t)mine * steps;
  auto tile_of = [&](uint32_t i) { return locate<kLongTokens, kFeatures>(p, table, blockIdx.x + i * gridDim.x, ntiles, lane); };

  if (wave >= kLongParts) {
    if (all == 0) return;
    uint32_t turn = 0;
    int step = 0, slot = 0;
    // past the end the last step again, and past K its last block, so that every
    // step counts the same
    auto drive = [&](auto enter, auto issue, auto wait_landed) __attribute__((always_inline)) {
#pragma unroll 1
      for (int64_t s = 0; s < all + kAhead; ++s) {
        if (step == 0) enter(tile_of(turn));
        issue(step * kLongParts, lds_addr(ring) + (uint32_t)slot * S::kStepBytes);   // into the slot of step s - S::kSlots, whose reads ended before the last barrier
        slot = slot + 1 == S::kSlots ? 0 : slot + 1;
        if (step + 1 < steps) {
          ++step;
        } else if (turn + 1 < mine) {
          ++turn;
          step = 0;
        }
        if (s >= kAhead - 1) {
          wait_landed();   // all but the youngest kAhead - 1 steps
          workgroup_barrier();
        }
      }
      wait_dma_all();   // transfers past the end, before the workgroup's LDS is released
    };
    if (wave == kLongParts) {
      uint32_t off[kLongTokens / 8], s_off = 0;
      const uint8_t *base = nullptr;
      const float *scales = nullptr;
      drive(
          [&](const Tile &t) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kLongTokens / 8; ++i) {
              const int row = 8 * i + dr;
              off[i] = (uint32_t)min(row, t.left - 1) * (uint32_t)p.k + ((ds ^ swz(row)) << 4);
            }
            s_off = (uint32_t)min(lane, t.left - 1) * (uint32_t)nkb * 4;
            base = p.a + (int64_t)t.row0 * p.k;
            scales = p.a_s + (int64_t)t.row0 * nkb;
          },
          [&](int kb0, uint32_t to) __attribute__((always_inline)) {
#pragma unroll
            for (int q = 0; q < kLongParts; ++q) {
              const int64_t kb = min(kb0 + q, nkb - 1);
#pragma unroll
              for (int i = 0; i < kLongTokens / 8; ++i) lds_dma16(base + kb * kBlock, off[i], to + q * S::kPartBytes + i * 1024);
              lds_dma4(scales + kb, s_off, to + q * S::kPartBytes + (kLongTokens + kRows) * kBlock);
            }
          },
          [&]() __attribute__((always_inline)) { asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * S::kDmaA) : "memory"); });
    } else {
      const int part = wave - kLongParts - 1;
      uint32_t off[kRows / 8];
      const uint8_t *base0 = nullptr, *base1 = nullptr;
      drive(
          [&](const Tile &t) __attribute__((always_inline)) {
            const int left = (int)min((int64_t)kFeatures, p.f - t.f0);
#pragma unroll
            for (int i = 0; i < kRows / 8; ++i) {
              const int row = 8 * i + dr;
              off[i] = (uint32_t)min(row % kFeatures, left - 1) * (uint32_t)p.k + ((ds ^ swz(row)) << 4);
            }
            const int64_t at = ((int64_t)t.expert * p.f + t.f0) * p.k;
            base0 = p.w0 + at;
            base1 = kGated ? p.w1 + at : base0;
          },
          [&](int kb0, uint32_t to) __attribute__((always_inline)) {
            const int64_t kb = min(kb0 + part, nkb - 1);
#pragma unroll
            for (int i = 0; i < kRows / 8; ++i)
              lds_dma16((8 * i < kFeatures ? base0 : base1) + kb * kBlock, off[i],
                        to + part * S::kPartBytes + kLongTokens * kBlock + i * 1024);
          },
          [&]() __attribute__((always_inline)) { asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * S::kDmaB) : "memory"); });
    }
    return;
  }

  if (all > 0) {
    uint32_t turn = 0;
    int step = 0, slot = 0;
    bool joined = false;   // a tile's sums are in LDS, from before the last barrier
    Tile tile = tile_of(0), done = tile;
    f32x4 acc[S::kJ];
#pragma unroll
    for (int j = 0; j < S::kJ; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto sum = [&](int j) {
      f32x4 v = join[j * 64 + lane];
#pragma unroll
      for (int q = 1; q < kLongParts; ++q) v += join[(q * S::kJ + j) * 64 + lane];
      return v;
    };
    auto finish = [&]() __attribute__((always_inline)) {   // 16 features a wave
      const int64_t col = done.f0 + 16 * wave + 4 * fq;
      if (16 * wave >= kFeatures || fr >= done.left || col >= p.f) return;
      store_four(p, done.row0 + fr, col, kGated ? gated4(sum(wave), sum(wave + S::kJ / 2)) : sum(wave));
    };
#pragma nounroll
    for (int64_t s = 0; s < all; ++s) {
      workgroup_barrier();   // step s landed
      const int kb = step * kLongParts + wave;
      if (kb < nkb) {
        const uint8_t *a = ring + slot * S::kStepBytes + wave * S::kPartBytes, *b = a + kLongTokens * kBlock;
        const int64_t at = ((int64_t)tile.expert * p.blocks_f + tile.f0 / kBlock) * nkb + kb;
        const float w0 = load_uniform(p.w0_s, at), w1 = kGated ? load_uniform(p.w1_s, at) : w0;
        const float sa = ((const float *)(b + kRows * kBlock))[fr];
        const i32x8 av = frag_from_lds(a + fr * kBlock, fq, fr);
        i32x8 bv[S::kJ];
#pragma unroll
        for (int j = 0; j < S::kJ; ++j) bv[j] = frag_from_lds(b + (16 * j + fr) * kBlock, fq, 16 * j + fr);
        f32x4 prt[S::kJ];
#pragma unroll
        for (int j = 0; j < S::kJ; ++j) prt[j] = mfma_e4m3_16x16x128(bv[j], av, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int j = 0; j < S::kJ; ++j) {
          const float sc = sa * (kGated && j >= S::kJ / 2 ? w1 : w0);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = __builtin_fmaf(prt[j][e], sc, acc[j][e]);
        }
      }
      slot = slot + 1 == S::kSlots ? 0 : slot + 1;
      if (joined) finish();
      joined = false;
      if (++step == steps) {
        // a tile has two steps at least (product_shape): the last tile's sums were
        // read before the barrier that began this step
#pragma unroll
        for (int j = 0; j < S::kJ; ++j) {
          join[(wave * S::kJ + j) * 64 + lane] = acc[j];
          acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        joined = true;
        done = tile;
        step = 0;
        if (++turn < mine) tile = tile_of(turn);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read, and its sums written: its slot may be refilled
    }
    workgroup_barrier();   // the movers' last
    finish();
  }
  clear_behind(p, table.begin[p.experts], 64 * kLongParts);
}

// ---------------------------------------------------------------------------
// Many rows an expert: 256 rows by 256 rows of weights (gated: 128 features' gate
// and up).
//
// Workgroup: 512 threads = 8 waves, 4 x 2, a wave 64 rows by 128 rows of weights
// (4 x 8 MFMA tiles, two waves per SIMD); gated, in each half 64 gate rows and the
// 64 up rows of the same features.  A two-stage LDS ring by direct global->LDS
// transfers, block kb + 1 loaded while kb is computed, over the ends of tiles.
// The rescale of an MFMA's partial runs three MFMAs behind it.  The loop over K is that
// of big_tiles (e4m3_tiles.h), and a fix to one belongs in both.  Waves whose rows an
// expert does not have skip their MFMAs: a tile of up to 128 rows keeps one wave a
// SIMD.
//
// Measured, 2 x 2048 x 7168: 512 rows at each of 64 experts 902-927 us, 2.1 PFLOP/s;
// 1024 rows 1691-1742, 2.2-2.3; 4096 x 4 choices of 32 experts, unevenly, 535-580 us,
// 1.7 PFLOP/s (four rounds of long tiles and one of short ones, whose weights come
// from HBM again; the matrix cores are busy 43% of the cycles, at 2.05 GHz).  7168 x
// 2048: 512 rows 503-521 us, 4096 x 4 choices 287-296.  What it took (902 and 503):
// scales of four blocks a transfer and the tiles' order (1068 and 592 without), 16
// byte stores (909 and 537 with 8).  What was measured slower: the weights' transfers
// one to two MFMA columns earlier or later (by up to 8%), a's by all eight waves (2-8%),
// lines touched three blocks ahead (8-12%), short tiles on all eight waves, 64 x 64
// each (registers spill: 8-20%).
// ---------------------------------------------------------------------------
template <bool kGated, bool kQuad>
__global__ __launch_bounds__(kBigThreads) void product_big_kernel(const ProductArgs p) {
  constexpr int kFeatures = kGated ? kBigTile / 2 : kBigTile;
  struct Smem {
    uint8_t a[2][kBigTile * kBlock];
    uint8_t b[2][kBigTile * kBlock];
    float as[2][kBigTile * (kQuad ? 4 : 1)];   // by block, or by [row][4 blocks]
  };
  __shared__ __attribute__((aligned(1024))) Smem sm;
  __shared__ SplitTable table;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = p.nkb;
  const int wa = (wave >> 1) * 64, wb = wave & 1;   // wave's rows, and half of the weights' rows
  const int fr = lane & 15, fq = lane >> 4;
  // transfers: lane p of an 8-row group fills chunk slot p % 8 of row p / 8; a's
  // group 8 d + g by wave d < 4, the weights' group 4 w + i by every wave w
  const bool dma_wave = wave < 4;
  const int dw = wave & 3, dr = lane >> 3, ds = lane & 7;
  const uint32_t lds_a = lds_addr(&sm.a[0][0]), lds_b = lds_addr(&sm.b[0][0]), lds_as = lds_addr(&sm.as[0][0]);
  build_table<kBigThreads, kBigTile>(p, table);
  const uint32_t ntiles = (uint32_t)(__builtin_amdgcn_readfirstlane(table.first[p.experts]) +
                                     __builtin_amdgcn_readfirstlane(table.half[p.experts])) * (uint32_t)p.tiles_f;

  uint32_t a_off[8], b_off[4], s_off = 0;   // from the tile's own base
  const uint8_t *a_base = nullptr, *b_base = nullptr;
  const float *as_base = nullptr;
  auto set_offsets = [&](const Tile &t) {   // rows past an edge re-read the last one
    a_base = p.a + (int64_t)t.row0 * p.k;
    as_base = p.a_s + (int64_t)t.row0 * nkb;
    s_off = (uint32_t)min(64 * dw + lane, t.left - 1) * (uint32_t)nkb * 4;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const int row = 8 * (8 * dw + g) + dr;
      a_off[g] = (uint32_t)min(row, t.left - 1) * (uint32_t)p.k + ((ds ^ swz(row)) << 4);
    }
    b_base = (kGated && (wave & 2) ? p.w1 : p.w0) + ((int64_t)t.expert * p.f + t.f0) * p.k;
    const int left = (int)min((int64_t)kFeatures, p.f - t.f0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * (4 * wave + i) + dr;   // gated: half row / 128, projection (row / 64) % 2
      const int r = kGated ? (row >> 7) * 64 + (row & 63) : row;
      b_off[i] = (uint32_t)min(r, left - 1) * (uint32_t)p.k + ((ds ^ swz(row)) << 4);
    }
  };
  int quad = 1;   // kQuad: the buffer that holds the newest four blocks' scales
  auto issue_a = [&](int kb, int s) {
    const uint8_t *ab = a_base + (int64_t)kb * kBlock;
#pragma unroll
    for (int g = 0; g < 8; ++g) lds_dma16(ab, a_off[g], lds_a + s * (kBigTile * kBlock) + (8 * dw + g) * 1024);
    if (!kQuad) {
      lds_dma4(as_base + kb, s_off, lds_as + s * (kBigTile * 4) + dw * 256);
    } else if (kb % 4 == 0) {
      lds_dma16(as_base + kb, s_off, lds_as + (quad ^ 1) * (kBigTile * 16) + dw * 1024);
    }
  };
  auto issue_b = [&](int kb, int s) {
    const uint8_t *bb = b_base + (int64_t)kb * kBlock;
#pragma unroll
    for (int i = 0; i < 4; ++i) lds_dma16(bb, b_off[i], lds_b + s * (kBigTile * kBlock) + (4 * wave + i) * 1024);
  };

  int stage = 0;
  bool landed = false;
  Tile tile;
  if (blockIdx.x < ntiles) {
    tile = locate<kBigTile, kFeatures>(p, table, blockIdx.x, ntiles, lane);
    set_offsets(tile);
    if (dma_wave) issue_a(0, 0);
    issue_b(0, 0);
  }
  for (uint32_t it = blockIdx.x; it < ntiles; it += gridDim.x) {
    const bool more = it + gridDim.x < ntiles;
    Tile next = tile;
    if (more) next = locate<kBigTile, kFeatures>(p, table, it + gridDim.x, ntiles, lane);
    const bool live = wa < tile.left;
    // the wave's features lie in one block column
    const int64_t wcol = min(tile.f0 / kBlock + (kGated ? 0 : wb), (int64_t)p.blocks_f - 1);
    const int64_t w_at = ((int64_t)tile.expert * p.blocks_f + wcol) * nkb;

    f32x4 acc[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 prt[4];
    float sc[2][4];   // row scale * weight scale, per projection
#pragma unroll
    for (int q = 0; q < 4; ++q) prt[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[0][i] = sc[1][i] = 0.f;
    auto rescale = [&](int qp) {   // MFMA qp = 4 j + i
      const int ip = qp % 4, jp = qp / 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[ip][jp][e] = __builtin_fmaf(prt[qp % 4][e], sc[kGated ? jp / 4 : 0][ip], acc[ip][jp][e]);
    };

#pragma nounroll
    for (int kb = 0; kb < nkb; ++kb, stage ^= 1) {
      const int cur = stage;
      const float w0 = load_uniform(p.w0_s, w_at + kb), w1 = kGated ? load_uniform(p.w1_s, w_at + kb) : 0.f;
      if (!landed) {
        wait_dma_all();
        workgroup_barrier();   // stage cur landed for every wave; stage cur ^ 1 no longer read
      }
      landed = false;
      // the next block: the tile's, or the next tile's first (past the last tile the
      // weights' last block again, into the stage no one reads again)
      const bool last = kb + 1 == nkb;
      const int kn = !last ? kb + 1 : more ? 0 : kb;
      if (kQuad && kb % 4 == 0) quad ^= 1;   // the four that begin here have landed
      if (last && more) set_offsets(next);
      if (dma_wave && (!last || more)) issue_a(kn, cur ^ 1);
      // retire the scalar loads now: while one is outstanding every LDS wait
      // would be a full drain
      asm volatile("" ::"s"(w0), "s"(w1));
      if (!live) {
        issue_b(kn, cur ^ 1);
        continue;
      }
      float sa[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sa[i] = kQuad ? sm.as[quad][(wa + 16 * i + fr) * 4 + kb % 4] : sm.as[cur][wa + 16 * i + fr];
      auto read_b = [&](int j) {
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
#pragma unroll
      for (int qp = 29; qp < 32; ++qp) rescale(qp);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j + 1 < 8) bnext = read_b(j + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = 4 * j + i;
          prt[q % 4] = mfma_e4m3_16x16x128(bcur, af[i], f32x4{0.f, 0.f, 0.f, 0.f});
          // unconditional, so that no branch splits the unrolled loop
          if (j == 2 && i == 0) issue_b(kn, cur ^ 1);
          if (q == 3) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              sc[0][r] = sa[r] * w0;
              sc[1][r] = sa[r] * w1;
            }
          }
          if (q >= 3) rescale(q - 3);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (j + 1 < 8) bcur = bnext;
      }
    }
#pragma unroll
    for (int qp = 29; qp < 32; ++qp) rescale(qp);
    // the next tile's first block is waited for before this tile's stores, which
    // then drain while that block is computed
    if (more) {
      wait_dma_all();
      workgroup_barrier();
      landed = true;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (wa + 16 * i >= tile.left) break;
      const int r = wa + 16 * i + fr;
#pragma unroll
      for (int j = 0; j < (kGated ? 4 : 8); j += 2)
        store_pair(p, r < tile.left, tile.row0 + r, tile.f0 + (kGated ? 64 : 128) * wb + 16 * j, fq,
                   kGated ? gated4(acc[i][j], acc[i][(j + 4) % 8]) : acc[i][j],
                   kGated ? gated4(acc[i][j + 1], acc[i][(j + 5) % 8]) : acc[i][j + 1]);
    }
    tile = next;
  }
  wait_dma_all();   // transfers past the end, before the workgroup's LDS is released
  clear_behind(p, table.begin[p.experts], kBigThreads);
}

template <int kTokens>
hipError_t launch_stream(ProductArgs p, bool gated, int cus, hipStream_t stream) {
  const int features = gated ? kStreamRows / 2 : kStreamRows;
  p.tiles_f = (int)((p.f + features - 1) / features);
  using S = StreamShape<kTokens>;
  const size_t lds = S::lds(p.experts);
  const dim3 grid((unsigned)(2 * cus)), block(S::kThreads);
  if (gated)
    hipLaunchKernelGGL((product_stream_kernel<true, kTokens>), grid, block, lds, stream, p);
  else
    hipLaunchKernelGGL((product_stream_kernel<false, kTokens>), grid, block, lds, stream, p);
  return hipGetLastError();
}

template <int kRows>
hipError_t launch_long(ProductArgs p, bool gated, int cus, hipStream_t stream) {
  using S = LongShape<kRows>;
  const int features = gated ? kRows / 2 : kRows;
  p.tiles_f = (int)((p.f + features - 1) / features);
  const size_t lds = (size_t)S::kSlots * S::kStepBytes + S::kJoinBytes + Table::bytes(p.experts);
  const dim3 grid((unsigned)cus), block(kLongThreads);
  if (gated)
    hipLaunchKernelGGL((product_long_kernel<true, kRows>), grid, block, lds, stream, p);
  else
    hipLaunchKernelGGL((product_long_kernel<false, kRows>), grid, block, lds, stream, p);
  return hipGetLastError();
}

// Whether the scales of a row's four blocks are a 16-byte transfer's.
bool scales_by_four(int nkb, const float *a_s) { return nkb % 4 == 0 && ((uintptr_t)a_s & 15) == 0; }

hipError_t launch_big(ProductArgs p, bool gated, int cus, hipStream_t stream) {
  const int features = gated ? kBigTile / 2 : kBigTile;
  p.tiles_f = (int)((p.f + features - 1) / features);
  const dim3 grid((unsigned)cus), block(kBigThreads);
  const bool quad = scales_by_four(p.nkb, p.a_s);
  if (gated) {
    if (quad)
      hipLaunchKernelGGL((product_big_kernel<true, true>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((product_big_kernel<true, false>), grid, block, 0, stream, p);
  } else {
    if (quad)
      hipLaunchKernelGGL((product_big_kernel<false, true>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((product_big_kernel<false, false>), grid, block, 0, stream, p);
  }
  return hipGetLastError();
}

enum class Shape { kLong32, kLong64, kFew, kSome, kMany };

// By the rows an expert has on average, which is all that the host knows; an expert's
// last tile counts as half a one.  Choices that take no part count as rows: where seven
// of eight are at other ranks' experts, 256 tokens' 8 choices at 32 experts of 2 x 2048 x
// 7168 take 192 us, and 157 with those rows alone that are here.  Where tiles of 16 by 32 or 64 fit one round of the
// CUs they win, if the chain along K is long enough for steps of four blocks (us, 128
// rows of weights a tile, 32 and 64: 8 experts of 1024 x 640 with a row 5.7, 5.5 and
// 5.8; 16 of 2 x 512 x 1024 with 8 rows, 256 tiles of 64, 6.8 and 7.2; with a row of 2 x
// 512 x 1536 9.2 and 8.8); beyond a round they do not (8 of 2 x 1280 x 7168, 320 tiles
// of 64: 29.6 and 33.2).  Else, up to eight rows, nearly no expert has more than 16 (us,
// tiles of 16 and 64 rows: 16 experts of 2 x 512 x 1024 6.1 and 7.4, 8 of 2 x 2048 x
// 7168 34.8 and 35.8).  From there on the cheaper of 64 and 256 rows: rounds of tiles on all CUs, each so much per block of 128
// and so much besides, and the weights' bytes, of which some three tenths of the
// shorter show beside the longer.  A partial tile an expert is half of one more on
// average; two tiles of 64 rows share a CU; short tiles of the 256-row kernel, up to
// some 128 rows an expert, cost less and fill up its later rounds.  Measured (64 and 256
// rows): 8 experts of 2 x 2048 x 7168 with 96 rows 48 and 75; 64 of 2300 x 1408 with 96
// rows 47 and 64; 64 of 2 x 2048 x 7168 with 64 rows 445 and 484, with 80 rows 503 and
// 469; 128 of 2 x 768 x 2048 with 64 rows 94 and 109, with 160 rows 148 and 124.
Shape product_shape(int64_t rows, int64_t experts, int64_t f, int64_t k, bool gated, int cus) {
  const double active = (double)min(rows, experts), each = (double)rows / active, nkb = (double)(k / kBlock);
  auto tiles = [&](int weight_rows) {   // of 16 rows
    const double tokens = each / kLongTokens + 0.5, features = gated ? weight_rows / 2 : weight_rows;
    return active * (tokens > 1.0 ? tokens : 1.0) * ceil((double)f / features);
  };
  if (nkb > kLongParts && tiles(32) <= cus) return Shape::kLong32;
  if (nkb >= 12 && tiles(64) <= cus) return Shape::kLong64;
  if (each <= 8) return Shape::kFew;
  auto rounds = [&](double rows_a_tile, double features) {
    const double tokens = each / rows_a_tile + 0.5;
    return active * (tokens > 1.0 ? tokens : 1.0) * ceil((double)f / features) / cus;
  };
  const double weights_us = active * (double)f * (double)k * (gated ? 2.0 : 1.0) / 5.1e6;
  auto with_weights = [&](double us) {
    return us < weights_us ? weights_us + 0.3 * us : us + 0.3 * weights_us;
  };
  const double some = ceil(rounds(64, gated ? 64 : 128)), pairs = floor(some / 2);
  const double some_us = pairs * (nkb * 0.87 + 0.8) + (some - 2 * pairs) * (nkb * 0.5 + 0.8);
  const double many = rounds(256, gated ? 128 : 256), full = each <= 64 ? 0.0 : each >= 192 ? 1.0 : (each - 64) / 128;
  const double many_us = (many <= 3 ? ceil(many) : many + 0.5) * (nkb * (1.2 + 0.4 * full) + 5.0);
  return with_weights(many_us) < with_weights(some_us) ? Shape::kMany : Shape::kSome;
}

}  // namespace

hipError_t launch_expert_product(const uint8_t *a, const float *a_s, const int32_t *offsets, const uint8_t *w0,
                                 const float *w0_s, const uint8_t *w1, const float *w1_s, void *out, bool out_bf16,
                                 int64_t rows, int64_t experts, int64_t f, int64_t k, hipStream_t stream) {
  ProductArgs p = {};
  p.a = a;
  p.a_s = a_s;
  p.offsets = offsets;
  p.w0 = w0;
  p.w1 = w1;
  p.w0_s = w0_s;
  p.w1_s = w1_s;
  p.out = out;
  p.rows = rows;
  p.f = f;
  p.k = k;
  p.experts = (int)experts;
  p.nkb = (int)(k / kBlock);
  p.blocks_f = (int)((f + kBlock - 1) / kBlock);
  p.out_bf16 = out_bf16;
  int cus = current_device_cus();
  if (cus <= 0) cus = 256;
  const bool gated = w1 != nullptr;
  switch (product_shape(rows, experts, f, k, gated, cus)) {
    case Shape::kLong32: return launch_long<32>(p, gated, cus, stream);
    case Shape::kLong64: return launch_long<64>(p, gated, cus, stream);
    case Shape::kFew: return launch_stream<16>(p, gated, cus, stream);
    case Shape::kSome: return launch_stream<64>(p, gated, cus, stream);
    default: return launch_big(p, gated, cus, stream);
  }
}

}  // namespace fp8bsq
