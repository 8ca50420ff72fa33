// Gated feed-forward block for gfx950, forward: h = silu(g) * u with
// g = Q(x) Wg^T and u = Q(x) Wu^T on E4M3 codes and block scales.
//
// One K block of 128 gives, per 16 x 16 output tile and projection, one E4M3
// MFMA whose partial is multiplied by a_s[i, kb] * w_s[j / 128, kb] and added
// in FP32, as in the block-scaled GEMM.  Gate and up accumulators of one
// output element sit in the same lane, so silu(g) * u is formed in registers
// and only h (and, for training, g and u) reaches memory.
#include "device_cus.h"
#include "ffn_launch.h"
#include "mfma_tile.h"

namespace fp8bsq {
namespace {

// silu(g) * u; the exponential overflows to infinity for g below -88, where
// the sigmoid is 0 to fp32's precision.
__device__ __forceinline__ float gated(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// 256 threads = 2 x 2 waves, each wave 32 x 32 outputs of both projections,
// fragments read straight from global memory.  The 64-column workgroup tile
// never straddles a 128-row weight block.
template <bool kBf16Out>
__global__ __launch_bounds__(256) void gated_simple_kernel(
    const uint8_t *__restrict__ a, const float *__restrict__ a_s, const uint8_t *__restrict__ wg,
    const float *__restrict__ wg_s, const uint8_t *__restrict__ wu, const float *__restrict__ wu_s,
    void *__restrict__ h, void *__restrict__ g_out, void *__restrict__ u_out, int64_t m, int64_t f, int64_t k) {
  const int nkb = (int)(k / kBlock);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t m0 = (int64_t)blockIdx.y * 64 + (wave >> 1) * 32;
  const int64_t n0 = (int64_t)blockIdx.x * 64 + (wave & 1) * 32;
  const int64_t b_row = ((int64_t)blockIdx.x * 64) / kBlock;
  const int lr = lane & 15, lk = (lane >> 4) * 32, lq = (lane >> 4) * 4;

  f32x4 acc[2][2][2];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[w][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const i32x8 zero8 = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int kb = 0; kb < nkb; ++kb) {
    i32x8 af[2], bfr[2][2];
    float sa[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = m0 + 16 * i + lr;
      af[i] = row < m ? load_frag(a + row * k + (int64_t)kb * kBlock + lk) : zero8;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t orow = m0 + 16 * i + lq + r;
        sa[i][r] = orow < m ? a_s[orow * nkb + kb] : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t col = n0 + 16 * j + lr;
      const int64_t off = col * k + (int64_t)kb * kBlock + lk;
      bfr[0][j] = col < f ? load_frag(wg + off) : zero8;
      bfr[1][j] = col < f ? load_frag(wu + off) : zero8;
    }
    const float sb[2] = {wg_s[b_row * nkb + kb], wu_s[b_row * nkb + kb]};
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f32x4 p = mfma_e4m3_16x16x128(af[i], bfr[w][j], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[w][i][j][r] = __builtin_fmaf(p[r], sa[i][r] * sb[w], acc[w][i][j][r]);
        }
  }

#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t col = n0 + 16 * j + lr;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t row = m0 + 16 * i + lq + r;
        if (row < m && col < f) {
          const float g = acc[0][i][j][r], u = acc[1][i][j][r];
          store_out(h, kBf16Out, row * f + col, gated(g, u));
          if (g_out) {
            store_out(g_out, kBf16Out, row * f + col, g);
            store_out(u_out, kBf16Out, row * f + col, u);
          }
        }
      }
    }
}

// ---------------------------------------------------------------------------
// Tiled kernel for large M.
//
// Workgroup tile: 256 rows of x by 128 features of both projections, so the
// weight operand is 256 rows too: in each half of 128, 64 gate rows and the 64
// up rows of the same features.  512 threads = 8 waves, 4 x 2; a wave owns 64
// rows by 64 features, gate accumulators in acc[0..3] and up in acc[4..7] of the
// same lanes.  The weights are the MFMA's row operand: a lane then holds four
// consecutive features of one row of x, which leave as one 8-byte store, and
// the row's activation scale is one value per lane.
//
// Operands reach LDS by direct global->LDS transfers into a two-stage ring
// (K block kb + 1 is loaded while kb is computed), issued where the block GEMM
// measured them cheapest: x's 32 by waves 0-3 at the top of the block, the
// weights' 32 by all waves after their first MFMAs.  The rescale of an MFMA's
// partial runs three MFMAs behind it.
//
// Scales: chunks of eight K blocks per row, double-buffered (kTab), or one
// 4-byte transfer per row and K block when K / 128 is not a multiple of four.
// kMx: power-of-two activation scales go into the MFMA as E8M0 exponents, and
// the rescale is by the weight scale alone (bit-identical).
// ---------------------------------------------------------------------------
constexpr int kTileM = 256, kTileF = 128, kTileThreads = 512, kTabKb = 8;

struct GatedSmem {
  uint8_t a[2][kTileM * kBlock];
  uint8_t b[2][2 * kTileF * kBlock];
  union {
    float as[2][kTileM];             // the K block's scales, per stage
    float tab[2][kTileM * kTabKb];   // [32-row block][half][row][4 K blocks]
  };
};

// Tile of workgroup turn `it`: workgroups are dealt round-robin to the eight
// XCDs, so turns it, it + 8, ... get consecutive tiles of one XCD's contiguous
// share (they then share its L2); tiles run in groups of four M tiles across F.
__device__ __forceinline__ void gated_tile_coords(int it, int tiles_m, int tiles_f, int &tm, int &tf) {
  const int ntiles = tiles_m * tiles_f, base = ntiles / 8, rest = ntiles % 8, xcd = it % 8;
  const int tile = xcd * base + min(xcd, rest) + it / 8;
  constexpr int kGroupM = 4;
  const int group = tile / (kGroupM * tiles_f), first = group * kGroupM;
  const int gm = min(tiles_m - first, kGroupM), idx = tile - group * kGroupM * tiles_f;
  tm = first + idx % gm;
  tf = idx / gm;
}

// Four consecutive outputs of a row, or those of them inside it.
template <bool kBf16Out>
__device__ __forceinline__ void store4(void *p, int64_t idx, f32x4 v, bool vec, int left) {
  if (vec && left >= 4) {
    if (kBf16Out)
      *(u32x2 *)((uint16_t *)p + idx) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else
      *(f32x4 *)((float *)p + idx) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) store_out(p, kBf16Out, idx + e, v[e]);
  }
}

template <bool kBf16Out, bool kMx, bool kTab>
__global__ __launch_bounds__(kTileThreads) void gated_tile_kernel(
    const uint8_t *__restrict__ a, const float *__restrict__ a_s, const uint8_t *__restrict__ wg,
    const float *__restrict__ wg_s, const uint8_t *__restrict__ wu, const float *__restrict__ wu_s,
    void *__restrict__ h, void *__restrict__ g_out, void *__restrict__ u_out, int64_t m, int64_t f, int64_t k,
    int tiles_m, int tiles_f, bool vec) {
  __shared__ __attribute__((aligned(1024))) GatedSmem sm;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = (int)(k / kBlock), ntiles = tiles_m * tiles_f;
  const int wm = (wave >> 1) * 64, wc = wave & 1;      // wave's rows of x, and half of the features
  const int fr = lane & 15, fq = lane >> 4;
  // transfers: lane p of an 8-row group fills chunk slot p % 8 of row p / 8; x
  // group 8 d + g by wave d < 4, weight group 4 w + h by every wave w (32 rows,
  // all of one projection)
  const bool dma_wave = wave < 4;
  const int dw = wave & 3, dr = lane >> 3, ds = lane & 7;
  const uint8_t *w_base = (wave & 2) ? wu : wg;
  const uint32_t lds_a = lds_addr(&sm.a[0][0]), lds_b = lds_addr(&sm.b[0][0]), lds_s = lds_addr(&sm.as[0][0]);

  uint32_t a_off[8], b_off[4], s_off[2];
  auto set_offsets = [&](int64_t m0, int64_t f0) {   // rows past an edge re-read the last one
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const int row = 8 * (8 * dw + g) + dr;
      a_off[g] = (uint32_t)(min(m0 + row, m - 1) * k + ((ds ^ swz(row)) << 4));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * (4 * wave + i) + dr;   // of 256: half row / 128, projection (row / 64) % 2
      b_off[i] = (uint32_t)(min(f0 + (row >> 7) * 64 + (row & 63), f - 1) * k + ((ds ^ swz(row)) << 4));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = min(m0 + 32 * (dw + 4 * i) + (lane & 31), m - 1);
      s_off[i] = (uint32_t)(row * nkb * 4 + (kTab ? (lane >> 5) * 16 : 0));
    }
  };
  auto issue_a = [&](int kb, int s) {
    const uint8_t *ab = a + (int64_t)kb * kBlock;
#pragma unroll
    for (int g = 0; g < 8; ++g) lds_dma16(ab, a_off[g], lds_a + s * (kTileM * kBlock) + (8 * dw + g) * 1024);
    if (!kTab) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (lane < 32) lds_dma4(a_s + kb, s_off[i], lds_s + s * (kTileM * 4) + 32 * (dw + 4 * i) * 4);
    }
  };
  auto issue_b = [&](int kb, int s) {
    const uint8_t *bb = w_base + (int64_t)kb * kBlock;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      lds_dma16(bb, b_off[i], lds_b + s * (2 * kTileF * kBlock) + (4 * wave + i) * 1024);
  };
  // scale chunk c into buffer c & 1; in a half-filled last chunk the upper lanes
  // re-read their row's first four scales (in bounds, never used)
  auto issue_tab = [&](int c) {
    const int kb0 = kTabKb * c;
    const bool inside = kb0 + 4 * (lane >> 5) < nkb;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      lds_dma16(a_s, inside ? s_off[i] + (uint32_t)kb0 * 4 : s_off[i] - (uint32_t)(lane >> 5) * 16,
                lds_s + (c & 1) * (kTileM * kTabKb * 4) + (dw + 4 * i) * 1024);
  };

  bool prologue_done = false;
  for (int it = blockIdx.x; it < ntiles; it += gridDim.x) {
    int tm, tf;
    gated_tile_coords(it, tiles_m, tiles_f, tm, tf);
    const int64_t m0 = (int64_t)tm * kTileM, f0 = (int64_t)tf * kTileF;
    const float *gs_row = wg_s + (int64_t)tf * nkb, *us_row = wu_s + (int64_t)tf * nkb;
    if (!prologue_done) {
      set_offsets(m0, f0);
      if (dma_wave) {
        issue_a(0, 0);
        if (kTab) issue_tab(0);
      }
      issue_b(0, 0);
    }
    const bool stage0_landed = prologue_done;

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
      for (int e = 0; e < 4; ++e) acc[ip][jp][e] = __builtin_fmaf(prt[qp % 4][e], sc[jp / 4][kMx ? 0 : ip], acc[ip][jp][e]);
    };

    auto step = [&](int kb, int cur, bool landed) {
      const float sbg = gs_row[kb], sbu = us_row[kb];
      if (!landed) {
        wait_dma_all();
        workgroup_barrier();   // stage cur landed for every wave; stage cur ^ 1 no longer read
      }
      if (dma_wave) {
        if (kb + 1 < nkb) issue_a(kb + 1, cur ^ 1);
        if (kTab && kb % kTabKb == 0 && kb + kTabKb < nkb) issue_tab(kb / kTabKb + 1);
      }
      // retire the scalar loads now: while one is outstanding every LDS wait
      // would be a full drain
      asm volatile("" ::"s"(sbg), "s"(sbu));
      // row wm + 16 i + fr: in 32-row block wm / 32 + i / 2, at row 16 (i % 2) + fr
      const float *tab = &sm.tab[(kb / kTabKb) & 1][((kb % kTabKb) >> 2) * 128 + (kb & 3)];
      float sa[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sa[i] = kTab ? tab[(wm / 32 + i / 2) * 256 + (16 * (i % 2) + fr) * 4] : sm.as[cur][wm + 16 * i + fr];
      auto read_b = [&](int j) {
        const int r = wc * 128 + 16 * j + fr;
        return frag_from_lds(&sm.b[cur][r * kBlock], fq, r);
      };
      i32x8 bcur = read_b(0), bnext;
      __builtin_amdgcn_sched_barrier(0);
      i32x8 af[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = wm + 16 * i + fr;
        af[i] = frag_from_lds(&sm.a[cur][r * kBlock], fq, r);
        __builtin_amdgcn_sched_barrier(0);
      }
      // the previous block's last rescale, while these reads are in flight
#pragma unroll
      for (int qp = 29; qp < 32; ++qp) rescale(qp);
      int ea[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ea[i] = (int)((__float_as_uint(sa[i]) >> 23) & 0xFFu);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j + 1 < 8) bnext = read_b(j + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = 4 * j + i;
          prt[q % 4] = kMx ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                 bcur, af[i], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, ea[i])
                           : mfma_e4m3_16x16x128(bcur, af[i], f32x4{0.f, 0.f, 0.f, 0.f});
          // unconditional, so that no branch splits the unrolled loop (the last
          // block re-reads itself into the stage no one reads again)
          if (j == 2 && i == 0) issue_b(min(kb + 1, nkb - 1), cur ^ 1);
          if (q == 3) {
#pragma unroll
            for (int r = 0; r < (kMx ? 1 : 4); ++r) {
              sc[0][r] = kMx ? sbg : sa[r] * sbg;
              sc[1][r] = kMx ? sbu : sa[r] * sbu;
            }
          }
          if (q >= 3) rescale(q - 3);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (j + 1 < 8) bcur = bnext;
      }
    };
#pragma nounroll
    for (int kb = 0; kb < nkb; ++kb) step(kb, kb & 1, kb == 0 && stage0_landed);
#pragma unroll
    for (int qp = 29; qp < 32; ++qp) rescale(qp);
    wait_dma_all();

    // the next tile's first transfers go out, and are waited for, before this
    // tile's stores, which then drain while that tile computes
    prologue_done = false;
    if (it + (int)gridDim.x < ntiles) {
      workgroup_barrier();
      int ntm, ntf;
      gated_tile_coords(it + gridDim.x, tiles_m, tiles_f, ntm, ntf);
      set_offsets((int64_t)ntm * kTileM, (int64_t)ntf * kTileF);
      if (dma_wave) {
        issue_a(0, 0);
        if (kTab) issue_tab(0);
      }
      issue_b(0, 0);
      wait_dma_all();
      workgroup_barrier();
      prologue_done = true;
    }

#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = m0 + wm + 16 * i + fr;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t col = f0 + 64 * wc + 16 * j + 4 * fq;
        if (row < m && col < f) {
          const f32x4 g = acc[i][j], u = acc[i][j + 4];
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = gated(g[e], u[e]);
          const int left = (int)min((int64_t)4, f - col);
          store4<kBf16Out>(h, row * f + col, v, vec, left);
          if (g_out) {
            store4<kBf16Out>(g_out, row * f + col, g, vec, left);
            store4<kBf16Out>(u_out, row * f + col, u, vec, left);
          }
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_gated_gemm(const uint8_t *a, const float *a_s, const uint8_t *wg, const float *wg_s,
                             const uint8_t *wu, const float *wu_s, void *h, void *g_out, void *u_out,
                             bool a_s_pow2, bool out_bf16, int64_t m, int64_t f, int64_t k, hipStream_t stream) {
  // the tiled kernel's transfers use 32-bit lane offsets from each base
  if (m * k < ((int64_t)1 << 32) && f * k < ((int64_t)1 << 32)) {
    const int64_t tiles_m = (m + kTileM - 1) / kTileM, tiles_f = (f + kTileF - 1) / kTileF;
    int cus = current_device_cus();
    if (cus <= 0) cus = 256;
    const dim3 tgrid((unsigned)(tiles_m * tiles_f < cus ? tiles_m * tiles_f : cus)), tblock(kTileThreads);
    const bool tab = (k / kBlock) % 4 == 0 && ((uintptr_t)a_s & 15) == 0;
    const uintptr_t mask = out_bf16 ? 7 : 15;
    const bool vec = f % 4 == 0 && (((uintptr_t)h | (uintptr_t)g_out | (uintptr_t)u_out) & mask) == 0;
#define FP8BSQ_GATED(BF, MX, TAB)                                                                               \
  hipLaunchKernelGGL((gated_tile_kernel<BF, MX, TAB>), tgrid, tblock, 0, stream, a, a_s, wg, wg_s, wu, wu_s, h, \
                     g_out, u_out, m, f, k, (int)tiles_m, (int)tiles_f, vec)
#define FP8BSQ_GATED_BF(MX, TAB) do { if (out_bf16) FP8BSQ_GATED(true, MX, TAB); else FP8BSQ_GATED(false, MX, TAB); } while (0)
    if (a_s_pow2) {
      if (tab) FP8BSQ_GATED_BF(true, true); else FP8BSQ_GATED_BF(true, false);
    } else {
      if (tab) FP8BSQ_GATED_BF(false, true); else FP8BSQ_GATED_BF(false, false);
    }
#undef FP8BSQ_GATED_BF
#undef FP8BSQ_GATED
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((f + 63) / 64), (unsigned)((m + 63) / 64)), block(256);
  if (out_bf16)
    hipLaunchKernelGGL(gated_simple_kernel<true>, grid, block, 0, stream, a, a_s, wg, wg_s, wu, wu_s, h, g_out,
                       u_out, m, f, k);
  else
    hipLaunchKernelGGL(gated_simple_kernel<false>, grid, block, 0, stream, a, a_s, wg, wg_s, wu, wu_s, h, g_out,
                       u_out, m, f, k);
  return hipGetLastError();
}

}  // namespace fp8bsq
