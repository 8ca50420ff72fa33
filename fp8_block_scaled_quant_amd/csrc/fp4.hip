// 4-bit weights for gfx950: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign),
// two to a byte, and one E8M0 scale byte per 32 weights of a row.
#include "device_cus.h"
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
// eight weights each.  Bound by memory: 18432 x 7168 bf16 (334 MB) 56 us,
// 6 TB/s.
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
// y = x W^T.  An E2M1 code times its power-of-two scale is exact in bf16 (scale
// bytes up to 252; 6 times a larger one overflows), and one instruction turns two
// codes and the scale into two bf16, so the group scales cost nothing in the
// product and one FP32 accumulator runs through K.
//
// MFMA 16x16x32 with the weights as the 16-row operand and 16 rows of x as
// columns.  The order of K inside the operands is free as long as both agree:
// lane l takes weight row l % 16 and the whole group 4 step + l / 16 -- 16 bytes
// of codes and one scale -- and feeds it to four MFMAs, eight codes each; x's
// lane reads the same eight k.
//
// The weights' bytes bound the product.  A block is 256 k: 128 bytes of codes a
// row.  Compute waves (`tiles` row tiles of 16, times `parts` that split K) move
// their own 16 rows, whole lines, by direct global->LDS transfers into a
// kDepth-slot ring, and wait for nothing else of their own.  Helper waves bring
// what the weights meet, a step of `blocks` blocks ahead, through registers: the
// scales, and x as bf16 planes (each value once per workgroup; fp32 x is split
// exactly into three bf16, 3 x 8 significand bits, one MFMA each).  One barrier
// per step hands these on; within a step the waves run freely.  Workgroups start
// at different steps: x's rows often lie a multiple of 4 KB apart, and all
// workgroups reading the same part of them at once queue at a few L2 channels
// (16 rows, 18432 x 28672: 137 us in one order for all).
//
// Measured, 18432 x 7168 (70.2 MB of codes and scales): one row 19 us, 97 MB from
// HBM at 5.2 TB/s (each step's 32 bytes of a row's scales bring their line again);
// 16 rows 23-25 us.  Fragments loaded straight to registers, 64 bytes of a row at a
// time, with x read by every wave, took 24 us for one row.
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

// Eight fp32 as the sum of three bf16 each: the upper 16 bits of what is left,
// which ends at bf16's smallest value, 2^-133: exact from |x| = 2^-110 on.
__device__ __forceinline__ void split3(float (&r)[8], u32x4 (&parts)[3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
#pragma unroll
    for (int c = 0; c < 4; ++c) parts[q][c] = high_halves(__float_as_uint(r[2 * c]), __float_as_uint(r[2 * c + 1]));
#pragma unroll
    for (int c = 0; c < 8; ++c) r[c] -= __uint_as_float(__float_as_uint(r[c]) & 0xFFFF0000u);
  }
}

constexpr int kGemvBlock = 256;        // k per block
constexpr int kGemvSlot = 16 * 128;    // bytes of codes a wave takes per block
// 8-value pieces of x that a helper lane carries
constexpr int gemv_pieces(bool bf16) { return bf16 ? 8 : 4; }
constexpr int kGemvBlocksMax = 4;      // blocks per step
constexpr int kGemvComputeMax = 10, kGemvWavesMax = 16;

struct GemvArgs {
  const void *x, *bias;
  const uint8_t *q, *s;
  void *y;
  int64_t m, n, k;
  int rows;                   // of x per workgroup
  int tiles, parts, blocks;   // parts and blocks are powers of two
  // helper waves: x_groups of x_waves each, and s_groups for the scales; group g
  // of n brings the steps g, g + n, ..., so a load has n steps' time
  int x_waves, x_groups, s_groups;
  bool out_bf16;
};

__device__ __forceinline__ int log2_of(int pow2) { return 31 - __builtin_clz(pow2); }

template <bool kBf16X, int kMT, int kDepth>
__global__ __launch_bounds__(64 * kGemvWavesMax) void fp4_gemv_kernel(const GemvArgs p) {
  constexpr int kPlanes = kBf16X ? 1 : 3;
  // codes [compute wave][slot][16 x 128]; scales [2][compute wave][block][16 x 8];
  // x [2][part][block][plane][row][512 bytes]
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int compute = p.tiles * p.parts;
  const int64_t m0 = (int64_t)blockIdx.y * p.rows;
  const int rows = (int)min((int64_t)p.rows, p.m - m0);
  const int ng = (int)(p.k / kGroup), nblk = (ng + 7) / 8, per = (nblk + p.parts - 1) / p.parts;
  const int steps = (per + p.blocks - 1) / p.blocks;
  const int sslot = compute * p.blocks * 128, xslot = p.parts * p.blocks * kPlanes * rows * 512;
  uint8_t *scales = lds + compute * kDepth * kGemvSlot;
  uint8_t *xs = scales + 2 * sslot;
  // the workgroup's steps, in its own order; prefetches past the last wrap around
  const int turn = blockIdx.x % steps;
  auto actual = [&](int step) { return (step + turn) % steps; };

  if (wave >= compute) {
    int helper = wave - compute;
    // a group's turn: step t goes to LDS while step t - 1 is multiplied
    auto run = [&](int group, int groups, auto load, auto store) {
      load(group);
      if (group == 0) {
        store(0);
        load(groups);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      workgroup_barrier();
      int next = group == 0 ? groups : group;   // the step in registers
      for (int step = 0; step < steps; ++step) {
        if (step + 1 == next) {
          store(next);   // into the buffer of step - 1
          next += groups;
          load(next);
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        workgroup_barrier();
      }
    };
    if (helper < p.s_groups) {
      // scales: 16 bytes, two blocks' (one's and eight unused, with one block a
      // step), of (compute wave, row)
      constexpr int kPieces = (kGemvComputeMax * kGemvBlocksMax / 2 * 16 + 63) / 64;
      const int per_row = max(p.blocks / 2, 1), pieces = compute * per_row * 16;
      u32x4 v[kPieces];
      int64_t src[kPieces];   // of actual step 0
      int group[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int idx = i * 64 + lane, wb = idx >> 4, w = wb >> log2_of(per_row), b = 2 * (wb & (per_row - 1));
        const int64_t row = min(((int64_t)blockIdx.x * p.tiles + (w >> log2_of(p.parts))) * 16 + (idx & 15), p.n - 1);
        group[i] = 8 * ((w & (p.parts - 1)) * per + b);
        src[i] = row * ng + group[i];
      }
      auto load = [&](int step) {
        const int ahead = 8 * actual(step) * p.blocks;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int left = ng - group[i] - ahead;
          v[i] = u32x4{0, 0, 0, 0};
          if (i * 64 + lane >= pieces || left <= 0) continue;
          if (src[i] + ahead + 16 <= p.n * ng)   // past the row's end lies the next row's, unused
            __builtin_memcpy(&v[i], p.s + src[i] + ahead, 16);
          else
            for (int c = 0; c < 16 && c < left; ++c) v[i][c >> 2] |= (uint32_t)p.s[src[i] + ahead + c] << (8 * (c & 3));
        }
      };
      auto store = [&](int step) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int idx = i * 64 + lane;
          if (idx >= pieces) continue;
          const int wb = idx >> 4, w = wb >> log2_of(per_row), b = 2 * (wb & (per_row - 1));
          uint8_t *dst = scales + (step & 1) * sslot + ((w * p.blocks + b) * 16 + (idx & 15)) * 8;
          *(u32x2 *)dst = u32x2{v[i][0], v[i][1]};
          if (p.blocks > 1) *(u32x2 *)(dst + 128) = u32x2{v[i][2], v[i][3]};
        }
      };
      run(helper, p.s_groups, load, store);
    } else {
      // x: eight values of (part, block, row)
      constexpr int kPieces = gemv_pieces(kBf16X);
      helper -= p.s_groups;
      int group = 0;
      for (; helper >= p.x_waves; helper -= p.x_waves) ++group;
      const int pieces = p.parts * p.blocks * rows * 32, stride = p.x_waves * 64, inverse = (65535 + rows) / rows;
      u32x4 v[kPieces][kBf16X ? 1 : 2];
      int64_t base[kPieces];   // the row's first value
      int k0[kPieces], dst[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        // (part, block) by the rows' inverse, exact for the at most 512 pieces / 32
        const int idx = i * stride + helper * 64 + lane, pb = ((idx >> 5) * inverse) >> 16, row = (idx >> 5) - pb * rows;
        const int part = pb >> log2_of(p.blocks), b = pb & (p.blocks - 1);
        base[i] = (m0 + row) * p.k;
        k0[i] = (part * per + b) * kGemvBlock + 8 * (idx & 31);
        dst[i] = (pb * kPlanes * rows + row) * 512 + (((idx & 31) ^ (row & 15)) << 4);
      }
      auto load = [&](int step) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          if (i * stride + helper * 64 + lane >= pieces) continue;
          // past the end any x will do: the codes it meets are zero
          const int64_t at = base[i] + min(k0[i] + actual(step) * p.blocks * kGemvBlock, (int)p.k - 8);
          if constexpr (kBf16X) {
            v[i][0] = *(const u32x4 *)((const uint16_t *)p.x + at);
          } else {
            v[i][0] = *(const u32x4 *)((const float *)p.x + at);
            v[i][1] = *(const u32x4 *)((const float *)p.x + at + 4);
          }
        }
      };
      auto store = [&](int step) {
        uint8_t *slot = xs + (step & 1) * xslot;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          if (i * stride + helper * 64 + lane >= pieces) continue;
          if constexpr (kBf16X) {
            *(u32x4 *)(slot + dst[i]) = v[i][0];
          } else {
            float r[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              r[c] = __uint_as_float(v[i][0][c]);
              r[4 + c] = __uint_as_float(v[i][1][c]);
            }
            u32x4 planes[3];
            split3(r, planes);
#pragma unroll
            for (int q = 0; q < 3; ++q) *(u32x4 *)(slot + dst[i] + q * rows * 512) = planes[q];
          }
        }
      };
      run(group, p.x_groups, load, store);
    }
    if (p.parts > 1) {   // the compute waves' sums
      workgroup_barrier();
      workgroup_barrier();
    }
    return;
  }

  const int tile = wave >> log2_of(p.parts), part = wave & (p.parts - 1);
  const int64_t n0 = ((int64_t)blockIdx.x * p.tiles + tile) * 16;
  const int64_t nc = min(n0, p.n - 1);   // rows past the last re-read it
  const int lr = lane & 15, lq = lane >> 4, dr = lane >> 3, ds = lane & 7;
  const int blk0 = part * per, blk1 = min(nblk, blk0 + per);
  const uint8_t *base = p.q + nc * (p.k / 2);
  const uint32_t row_off[2] = {(uint32_t)((min(nc + dr, p.n - 1) - nc) * (p.k / 2)),
                               (uint32_t)((min(nc + 8 + dr, p.n - 1) - nc) * (p.k / 2))};
  const int chunk[2] = {ds ^ swz(dr), ds ^ swz(8 + dr)};
  const uint8_t *ring = lds + wave * kDepth * kGemvSlot;
  const uint32_t lds_ring = lds_addr(ring);
  const int blocks_log2 = log2_of(p.blocks);
  auto block_of = [&](int j) {   // the j-th block of the workgroup's order, in the part
    return (actual(j >> blocks_log2) << blocks_log2) + (j & (p.blocks - 1));
  };
  auto issue = [&](int j) {   // groups past a row's end re-read its last one; so do blocks past the end
    const int blk = max(min(blk0 + block_of(j), blk1 - 1), 0);
    const uint32_t slot = lds_ring + (uint32_t)(j % kDepth) * kGemvSlot;
#pragma unroll
    for (int i = 0; i < 2; ++i) lds_dma16(base, row_off[i] + (uint32_t)min(8 * blk + chunk[i], ng - 1) * 16, slot + i * 1024);
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d) issue(d);
  f32x4 sum[2][kMT];   // of the even and the odd groups: two chains of MFMAs
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) sum[h][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
  workgroup_barrier();
  for (int step = 0; step < steps; ++step) {
    for (int b = 0; b < p.blocks; ++b) {
      const int j = step * p.blocks + b, blk = blk0 + block_of(j);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * (kDepth - 1)) : "memory");   // block j landed
      const uint8_t *slot = ring + j % kDepth * kGemvSlot + lr * 128;
      u32x4 codes[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) codes[h] = *(const u32x4 *)(slot + (((2 * lq + h) ^ swz(lr)) << 4));
      const uint32_t sc = *(const uint16_t *)(scales + (step & 1) * sslot + ((wave * p.blocks + b) * 16 + lr) * 8 + 2 * lq);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: the slot may be refilled
      issue(j + kDepth);
      if (blk >= blk1) continue;
      const uint8_t *xb = xs + (step & 1) * xslot + (part * p.blocks + b) * kPlanes * rows * 512;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool live = 8 * blk + 2 * lq + h < ng;
          const float scale = pow2_scale(live ? (sc >> (8 * h)) & 0xFFu : 127u);
          const bf16x8 w = fp4_to_bf16(live ? codes[h][t] : 0u, scale);
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            const int row = min(16 * mt + lr, rows - 1);   // a column past the last row has no output
            const uint8_t *at = xb + row * 512 + (((8 * lq + 4 * h + t) ^ (row & 15)) << 4);
#pragma unroll
            for (int q = 0; q < kPlanes; ++q)
              sum[h][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, *(const bf16x8 *)(at + q * rows * 512), sum[h][mt],
                                                                   0, 0, 0);
          }
        }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    workgroup_barrier();
  }
  f32x4 acc[kMT];
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt) acc[mt] = sum[0][mt] + sum[1][mt];
  wait_dma_all();   // transfers past the end, before LDS is used anew or released
  if (p.parts > 1) {   // the parts' sums, in part order
    f32x4 *sums = (f32x4 *)lds;
    workgroup_barrier();
    if (part > 0)
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) sums[(wave * kMT + mt) * 64 + lane] = acc[mt];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    workgroup_barrier();
    if (part > 0) return;
    for (int q = 1; q < p.parts; ++q)
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) acc[mt] += sums[((wave + q) * kMT + mt) * 64 + lane];
  }
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt) {
    if (16 * mt + lr >= rows) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t col = n0 + 4 * lq + e;
      if (col < p.n)
        store_out(p.y, p.out_bf16, (m0 + 16 * mt + lr) * p.n + col, acc[mt][e] + bias_at(p.bias, p.out_bf16, col));
    }
  }
}

template <bool kBf16X, int kMT>
hipError_t launch_gemv(GemvArgs a, hipStream_t stream) {
  int cus = current_device_cus();
  if (cus <= 0) cus = 256;
  const int64_t tiles = (a.n + 15) / 16, nblk = (a.k / kGroup + 7) / 8;
  const int rows = a.rows;
  // row tiles that give every CU one workgroup, parts of K up to ten waves, and as
  // many blocks a step as LDS and the helpers' registers hold of x
  constexpr int kPlanes = kBf16X ? 1 : 3;
  a.tiles = (int)min((tiles + cus - 1) / cus, (int64_t)9);
  a.parts = 1;
  while (2 * a.parts * a.tiles <= kGemvComputeMax && 2 * a.parts <= nblk && 2 * a.parts * rows <= 32) a.parts *= 2;
  const int compute = a.tiles * a.parts;
  a.blocks = kGemvBlocksMax;
  while (a.blocks > 1 && (a.parts * a.blocks * rows > 64 || 2 * a.parts * a.blocks * kPlanes * rows * 512 > 64 * 1024))
    a.blocks /= 2;
  constexpr int kLane = 64 * gemv_pieces(kBf16X);
  a.x_waves = (a.parts * a.blocks * rows * 32 + kLane - 1) / kLane;
  const int spare = kGemvWavesMax - compute;
  a.x_groups = max(1, min(4, (spare - 1) / a.x_waves));
  a.s_groups = max(1, min(4, spare - a.x_groups * a.x_waves));
  const size_t rest = (size_t)2 * compute * a.blocks * 128 + (size_t)2 * a.parts * a.blocks * kPlanes * rows * 512;
  const dim3 grid((unsigned)((tiles + a.tiles - 1) / a.tiles), (unsigned)((a.m + rows - 1) / rows));
  const dim3 block(64 * (compute + a.s_groups + a.x_groups * a.x_waves));
  int depth = 0;
  size_t lds = 0;
  for (int d : {8, 6, 4, 3, 2}) {
    depth = d;
    lds = rest + (size_t)compute * d * kGemvSlot;
    if (lds <= 160 * 1024) break;
  }
#define FP8BSQ_GEMV(D) hipLaunchKernelGGL((fp4_gemv_kernel<kBf16X, kMT, D>), grid, block, lds, stream, a)
  switch (depth) {
    case 8: FP8BSQ_GEMV(8); break;
    case 6: FP8BSQ_GEMV(6); break;
    case 4: FP8BSQ_GEMV(4); break;
    case 3: FP8BSQ_GEMV(3); break;
    default: FP8BSQ_GEMV(2); break;
  }
#undef FP8BSQ_GEMV
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp4_weight_quant(const void *w, bool w_bf16, int64_t n, int64_t k, uint8_t *q, uint8_t *s,
                                   hipStream_t stream) {
  // a launch has fewer than 2^32 threads, and more are dropped without an error:
  // 2^34 weights each
  constexpr int64_t kMost = (int64_t)1 << 29;
  const int64_t ngroups = n * (k / kGroup);
  for (int64_t at = 0; at < ngroups; at += kMost) {
    const int64_t part = min(ngroups - at, kMost);
    const dim3 grid((unsigned)((4 * part + 255) / 256)), block(256);
    const uint8_t *from = (const uint8_t *)w + at * kGroup * (w_bf16 ? 2 : 4);
    uint32_t *codes = (uint32_t *)q + at * (kGroup / 8);
    if (w_bf16)
      hipLaunchKernelGGL(fp4_weight_quant_kernel<true>, grid, block, 0, stream, from, part, codes, s + at);
    else
      hipLaunchKernelGGL(fp4_weight_quant_kernel<false>, grid, block, 0, stream, from, part, codes, s + at);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_fp4_gemv(const void *x, bool x_bf16, const uint8_t *q, const uint8_t *s, const void *bias,
                           void *y, bool y_bf16, int64_t m, int64_t n, int64_t k, hipStream_t stream) {
  GemvArgs a = {};
  a.x = x;
  a.bias = bias;
  a.q = q;
  a.s = s;
  a.y = y;
  a.m = m;
  a.n = n;
  a.k = k;
  a.out_bf16 = y_bf16;
  int cus = current_device_cus();
  if (cus <= 0) cus = 256;
  // Rows of x a workgroup: fp32 x takes three planes of LDS, and 32 rows of them
  // leave room for two waves' rings (64 rows, 18432 x 7168: 233 us against 147 by
  // 16; 64 bf16 rows: 59).  Where row tiles leave CUs idle the rows go to several
  // workgroups, which read the weights from the caches (32 fp32 rows,
  // 1000 x 2048: 9 us against 27 with 16 rows or more each).
  const int64_t tiles = (n + 15) / 16, most = x_bf16 ? 64 : 16;
  int64_t rows = m < most ? m : most;
  while (rows > 4 && tiles * ((m + (rows + 1) / 2 - 1) / ((rows + 1) / 2)) <= cus) rows = (rows + 1) / 2;
  a.rows = (int)rows;
  if (!x_bf16) return launch_gemv<false, 1>(a, stream);
  if (rows <= 16) return launch_gemv<true, 1>(a, stream);
  if (rows <= 32) return launch_gemv<true, 2>(a, stream);
  return launch_gemv<true, 4>(a, stream);
}

}  // namespace fp8bsq
