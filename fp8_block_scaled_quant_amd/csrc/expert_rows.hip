// Tokens' rows to their experts and back, for gfx950.
//
//   dispatch          y[rows[t, j]] = x[t], rows of choices of no expert (~r) zero
//   dispatch_quant    the same with act_quant's codes and scales, once a token
//   combine           out[t] = sum_j w[t, j] y[rows[t, j]], rows below 0 left out
//   combine_backward  dy[rows[t, j]] = w[t, j] dout[t] (~r: zero),
//                     dw[t, j] = <dout[t], y[rows[t, j]]>
//
// All four go by the token: its own row is read (or written) once, the rows of its
// choices are written (or read) once, and nothing is added up by atomics.  Each is
// bound by memory; measured, in bytes that must move against a 1 GiB copy's 5.1 TB/s:
//   dispatch_quant    8192 x 8 rows of 7168, bf16: 118 us, 5.1 TB/s
//   dispatch          1333 x 3 rows of 1001 fp32: 5.2 us, 4.1 TB/s
//   combine           4096 x 8 choices, half taking part, of 2048 bf16: 13.8 us, 6.1 TB/s
//   combine_backward  4096 x 8 rows of 4096 bf16: 113 us, 5.0 TB/s
// Rows that are written, and those that the backward pass reads, go past the caches
// (dispatch 6.2 us otherwise, combine_backward 122); combine's reads do not (15.6).
// A row number outside the sorted rows touches nothing.
#include "expert_launch.h"
#include "quant_block.h"

#include <type_traits>

namespace fp8bsq {
namespace {

constexpr int kThreads = 256;

struct RowArgs {
  const void *x;             // dispatch: tokens; combine: sorted rows; backward: the output's gradient
  const void *y;             // backward: sorted rows
  const int32_t *rows;
  const void *weights;       // or null
  void *out;                 // y | out | dy, or null
  void *scales;              // dispatch_quant: scales; backward: dweights, or null
  int64_t tokens, h;
  int top_k, nrows;
  bool w_bf16, ue8m0;
};

constexpr int kGroup = 8;   // choices whose rows are in flight together

// Up to kGroup of a token's choices.
struct Choices {
  int at[kGroup];      // row, or below 0 where nothing is to be touched
  bool live[kGroup];   // whether an expert has it
};

__device__ __forceinline__ Choices choices_of(const RowArgs &p, int64_t t, int j0) {
  const __attribute__((address_space(4))) int32_t *rows =
      (const __attribute__((address_space(4))) int32_t *)(uintptr_t)(p.rows + t * p.top_k + j0);
  Choices c;
  int r[kGroup];
  if (j0 + kGroup <= p.top_k) {
#pragma unroll
    for (int j = 0; j < kGroup; ++j) r[j] = rows[j];
  } else {
#pragma unroll
    for (int j = 0; j < kGroup; ++j) r[j] = rows[min(j, p.top_k - 1 - j0)];
  }
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    const int at = r[j] < 0 ? ~r[j] : r[j];
    c.at[j] = j0 + j < p.top_k && at < p.nrows ? at : -1;
    c.live[j] = c.at[j] >= 0 && r[j] >= 0;
  }
  return c;
}

__device__ __forceinline__ float weight_of(const RowArgs &p, int64_t c) {
  if (!p.weights) return 1.0f;
  return p.w_bf16 ? __uint_as_float((uint32_t)((const uint16_t *)p.weights)[c] << 16) : ((const float *)p.weights)[c];
}

typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));

// Sixteen bytes of a row, which may start on any element: an unaligned access costs
// less than one an element (1333 x 3 rows of 1001 fp32: 7.6 us by elements).  The
// last of a row may hold `count` elements only.
template <bool kBf16>
struct Piece {
  static constexpr int kCount = kBf16 ? 8 : 4;
  using Wide = std::conditional_t<kBf16, u32x4_at2, u32x4_at4>;
  using Element = std::conditional_t<kBf16, uint16_t, uint32_t>;
  u32x4 bits;

  template <bool kStream = false>
  __device__ __forceinline__ void load(const void *p, int64_t i, int count) {
    const Element *at = (const Element *)p + i;
    if (count == kCount) {
      bits = kStream ? __builtin_nontemporal_load((const Wide *)at) : *(const Wide *)at;
    } else {
      bits = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < kCount; ++e)
        if (e < count) bits[kBf16 ? e / 2 : e] |= (uint32_t)at[e] << (kBf16 ? 16 * (e & 1) : 0);
    }
  }
  template <bool kStream = false>
  __device__ __forceinline__ void store(void *p, int64_t i, int count) const {
    Element *at = (Element *)p + i;
    if (count == kCount) {
      if (kStream) __builtin_nontemporal_store(bits, (Wide *)at); else *(Wide *)at = bits;
    } else {
#pragma unroll
      for (int e = 0; e < kCount; ++e)
        if (e < count) at[e] = (Element)(bits[kBf16 ? e / 2 : e] >> (kBf16 ? 16 * (e & 1) : 0));
    }
  }
  __device__ __forceinline__ float value(int e) const {
    if (!kBf16) return __uint_as_float(bits[e]);
    return __uint_as_float(e & 1 ? bits[e / 2] & 0xFFFF0000u : bits[e / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[kCount]) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      bits[c] = kBf16 ? pack_bf16x2(v[(2 * c) % kCount], v[(2 * c + 1) % kCount]) : __float_as_uint(v[c]);
  }
};

// Threads that share a token, kWidth of them, a piece of its row each: a workgroup,
// and gridDim.y of these, for long rows; a wave or 16 lanes for short ones, which
// leave fewer idle (65536 rows of 32 bf16, combine and its gradient: 35 and 197 us by
// workgroups, 8.1 and 15 by 16 lanes; 8192 x 8 rows of 1000, 125 pieces: 24.1 and 66 by
// workgroups, 24.9 and 71 by waves).
template <int kWidth>
struct Lanes {
  static constexpr int kTokens = kThreads / kWidth;   // of a workgroup
  int64_t piece, first, step;   // the thread's piece, its first token, and how far the next is

  __device__ __forceinline__ Lanes() {
    int slot = threadIdx.x / kWidth;
    if (kWidth >= 64) slot = __builtin_amdgcn_readfirstlane(slot);   // rows' numbers then come by scalar loads
    piece = (int64_t)blockIdx.y * kWidth + threadIdx.x % kWidth;
    first = (int64_t)blockIdx.x * kTokens + slot;
    step = (int64_t)gridDim.x * kTokens;
  }
};

template <bool kBf16, int kWidth>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(const RowArgs p) {
  using P = Piece<kBf16>;
  const Lanes<kWidth> l;
  const int64_t i = l.piece * P::kCount;
  const int count = (int)min((int64_t)P::kCount, p.h - i);
  if (count <= 0) return;
  for (int64_t t = l.first; t < p.tokens; t += l.step) {
    P v;   // bits as they are: a copy keeps NaN's
    v.load(p.x, t * p.h + i, count);
    P none;
    none.bits = u32x4{0, 0, 0, 0};
    for (int j0 = 0; j0 < p.top_k; j0 += kGroup) {
      const Choices c = choices_of(p, t, j0);
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
        if (c.at[j] >= 0) (c.live[j] ? v : none).template store<true>(p.out, c.at[j] * p.h + i, count);
    }
  }
}

// Sixteen lanes own a 1 x 128 block of a token's row.  A workgroup holds whole rows
// (up to 64 blocks of them at a time): a sorted row's scales, 4 bytes a block, are
// then written by one XCD, and for wide rows together.  With a row's blocks spread
// over four workgroups, and so over four XCDs' caches, 8192 x 8 rows of 7168 took
// 149 us for 118 (5.1 TB/s, a copy's rate).
constexpr int kWideBlocks = 64, kSpreadBlocks = kThreads / 16;

template <bool kBf16>
__device__ __forceinline__ u32x2 quantize_at(const RowArgs &p, int64_t t, int nkb, int kb, int sub, float &s) {
  u32x4 v[kBf16 ? 1 : 2];
  load_block<kBf16>(p.x, t * nkb + kb, sub, v);
  return quantize_block<kBf16>(v, p.ue8m0, s);
}

// The scale of a row of zeros, that of the floor on amax.
__device__ __forceinline__ float zero_scale(const RowArgs &p) {
  float s, unused;
  block_scale(0u, p.ue8m0, s, unused);
  return s;
}

// A token a workgroup of 16 lanes a block.
template <bool kBf16>
__global__ __launch_bounds__(16 * kWideBlocks) void dispatch_quant_wide_kernel(const RowArgs p, int nkb) {
  __shared__ float scales[kWideBlocks];
  const int sub = threadIdx.x & 15, b = threadIdx.x >> 4;
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    for (int kb0 = 0; kb0 < nkb; kb0 += kWideBlocks) {
      const int kb = kb0 + b;
      u32x2 codes = {0, 0};
      if (kb < nkb) {   // whole 16-lane groups
        float s;
        codes = quantize_at<kBf16>(p, t, nkb, kb, sub, s);
        if (sub == 0) scales[b] = s;
      }
      __syncthreads();
      for (int j0 = 0; j0 < p.top_k; j0 += kGroup) {
        const Choices c = choices_of(p, t, j0);
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
          if (c.at[j] < 0) continue;
          const int64_t row = (int64_t)c.at[j] * nkb;
          u32x2 *to = (u32x2 *)((uint8_t *)p.out + (row + kb) * kBlock + 8 * sub);
          const u32x2 v = c.live[j] ? codes : u32x2{0, 0};
          if (kb < nkb) *to = v;
          if ((int)threadIdx.x < kWideBlocks && kb0 + (int)threadIdx.x < nkb)
            ((float *)p.scales)[row + kb0 + threadIdx.x] = c.live[j] ? scales[threadIdx.x] : zero_scale(p);
        }
      }
      __syncthreads();   // before the next scales
    }
  }
}

// kSpreadBlocks blocks a workgroup: of as many tokens as these are whole rows of,
// or a piece of one token's.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void dispatch_quant_kernel(const RowArgs p, int nkb) {
  const int sub = threadIdx.x & 15, b = threadIdx.x >> 4, slots = max(1, kSpreadBlocks / nkb);
  const int slot = slots > 1 ? b / nkb : 0, kb = blockIdx.y * kSpreadBlocks + b - slot * nkb;
  if (slot >= slots || kb >= nkb) return;   // whole 16-lane groups
  for (int64_t t = (int64_t)blockIdx.x * slots + slot; t < p.tokens; t += (int64_t)gridDim.x * slots) {
    float s;
    const u32x2 codes = quantize_at<kBf16>(p, t, nkb, kb, sub, s);
    for (int j0 = 0; j0 < p.top_k; j0 += kGroup) {
      const Choices c = choices_of(p, t, j0);
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        if (c.at[j] < 0) continue;
        const int64_t at = (int64_t)c.at[j] * nkb + kb;
        *(u32x2 *)((uint8_t *)p.out + at * kBlock + 8 * sub) = c.live[j] ? codes : u32x2{0, 0};
        if (sub == 0) ((float *)p.scales)[at] = c.live[j] ? s : zero_scale(p);
      }
    }
  }
}

template <bool kBf16, int kWidth>
__global__ __launch_bounds__(kThreads) void combine_kernel(const RowArgs p) {
  using P = Piece<kBf16>;
  const Lanes<kWidth> l;
  const int64_t i = l.piece * P::kCount;
  const int count = (int)min((int64_t)P::kCount, p.h - i);
  if (count <= 0) return;
  for (int64_t t = l.first; t < p.tokens; t += l.step) {
    float sum[P::kCount] = {};
    for (int j0 = 0; j0 < p.top_k; j0 += kGroup) {
      const Choices c = choices_of(p, t, j0);
      P v[kGroup];
      float w[kGroup];
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        w[j] = 0.0f;
        v[j].bits = u32x4{0, 0, 0, 0};   // and not 0 times what a row without an expert holds
        if (c.live[j]) {
          v[j].load(p.x, c.at[j] * p.h + i, count);
          w[j] = weight_of(p, t * p.top_k + j0 + j);
        }
      }
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
#pragma unroll
        for (int e = 0; e < P::kCount; ++e) sum[e] = __builtin_fmaf(w[j], v[j].value(e), sum[e]);
    }
    P out;
    out.set(sum);
    out.store(p.out, t * p.h + i, count);
  }
}

// kWidth threads go through a token's whole row; their partial dot products meet by
// shuffles, and a workgroup's waves' in LDS.
template <bool kBf16, int kWidth>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(const RowArgs p) {
  using P = Piece<kBf16>;
  __shared__ float partial[kThreads / 64][kGroup];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Lanes<kWidth> l;
  for (int64_t t = l.first; t < p.tokens; t += l.step) {
    for (int j0 = 0; j0 < p.top_k; j0 += kGroup) {
      const Choices c = choices_of(p, t, j0);
      float w[kGroup], dot[kGroup] = {};
#pragma unroll
      for (int j = 0; j < kGroup; ++j) w[j] = c.live[j] ? weight_of(p, t * p.top_k + j0 + j) : 0.0f;
      for (int64_t i = l.piece * P::kCount; i < p.h; i += kWidth * P::kCount) {
        const int count = (int)min((int64_t)P::kCount, p.h - i);
        P d, v[kGroup];
        d.load(p.x, t * p.h + i, count);
        if (p.scales) {
#pragma unroll
          for (int j = 0; j < kGroup; ++j)
            if (c.live[j]) v[j].template load<true>(p.y, c.at[j] * p.h + i, count);
        }
        if (p.out) {
#pragma unroll
          for (int j = 0; j < kGroup; ++j) {
            if (c.at[j] < 0) continue;
            P g;
            float scaled[P::kCount];
#pragma unroll
            for (int e = 0; e < P::kCount; ++e) scaled[e] = c.live[j] ? w[j] * d.value(e) : 0.0f;
            g.set(scaled);
            g.template store<true>(p.out, c.at[j] * p.h + i, count);
          }
        }
        if (p.scales) {
#pragma unroll
          for (int j = 0; j < kGroup; ++j)
            if (c.live[j])
#pragma unroll
              for (int e = 0; e < P::kCount; ++e) dot[j] = __builtin_fmaf(d.value(e), v[j].value(e), dot[j]);
        }
      }
      if (!p.scales) continue;
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
#pragma unroll
        for (int s = min(kWidth, 64) / 2; s > 0; s /= 2) dot[j] += __shfl_xor(dot[j], s);
      const int j = threadIdx.x % kWidth;   // the choice that the thread writes
      float sum = 0.0f;
      if (kWidth > 64) {
        if (lane == 0)
#pragma unroll
          for (int g = 0; g < kGroup; ++g) partial[wave][g] = dot[g];
        __syncthreads();
        if (j < kGroup)
#pragma unroll
          for (int v = 0; v < kThreads / 64; ++v) sum += partial[v][j];
        __syncthreads();   // before the next group's partials
      } else {
#pragma unroll
        for (int g = 0; g < kGroup; ++g) sum = j == g ? dot[g] : sum;
      }
      if (j < kGroup && j0 + j < p.top_k) {
        const int64_t c = t * p.top_k + j0 + j;
        if (p.w_bf16)
          ((uint16_t *)p.scales)[c] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
        else
          ((float *)p.scales)[c] = sum;
      }
    }
  }
}

// Workgroups along the tokens: fewer than 2^32 threads in a launch.
unsigned token_groups(int64_t tokens, int64_t across) {
  return (unsigned)min(tokens, ((int64_t)1 << 23) / across);
}

RowArgs row_args(const void *x, const int32_t *rows, const void *weights, bool w_bf16, int64_t tokens, int64_t top_k,
                 int64_t h, void *out) {
  RowArgs p = {};
  p.x = x;
  p.rows = rows;
  p.weights = weights;
  p.w_bf16 = w_bf16;
  p.tokens = tokens;
  p.top_k = (int)top_k;
  p.nrows = (int)(tokens * top_k);
  p.h = h;
  p.out = out;
  return p;
}

int64_t groups_of(int64_t n, int64_t each) { return (n + each - 1) / each; }

}  // namespace

// A kernel by the width that a row of h takes: pieces a thread; `whole`: the threads
// of a token go through its whole row.
#define FP8BSQ_BY_WIDTH(KERNEL, BF, P, WHOLE)                                                          \
  do {                                                                                                 \
    const int64_t pieces = groups_of((P).h, (BF) ? 8 : 4);                                             \
    const int width = pieces > 96 ? 256 : pieces > 32 ? 64 : 16;                                       \
    const int64_t across = (WHOLE) || pieces == 0 ? 1 : groups_of(pieces, width);                      \
    const dim3 grid(token_groups(groups_of((P).tokens, kThreads / width), across), (unsigned)across);  \
    const dim3 block(kThreads);                                                                        \
    if (width == 256)                                                                                  \
      hipLaunchKernelGGL((KERNEL<BF, 256>), grid, block, 0, stream, P);                                \
    else if (width == 64)                                                                              \
      hipLaunchKernelGGL((KERNEL<BF, 64>), grid, block, 0, stream, P);                                 \
    else                                                                                               \
      hipLaunchKernelGGL((KERNEL<BF, 16>), grid, block, 0, stream, P);                                 \
  } while (0)

hipError_t launch_expert_dispatch(const void *x, bool bf16, const int32_t *rows, int64_t tokens, int64_t top_k,
                                  int64_t h, void *y, hipStream_t stream) {
  const RowArgs p = row_args(x, rows, nullptr, false, tokens, top_k, h, y);
  if (bf16)
    FP8BSQ_BY_WIDTH(dispatch_kernel, true, p, false);
  else
    FP8BSQ_BY_WIDTH(dispatch_kernel, false, p, false);
  return hipGetLastError();
}

hipError_t launch_expert_dispatch_quant(const void *x, bool bf16, bool ue8m0, const int32_t *rows, int64_t tokens,
                                        int64_t top_k, int64_t h, uint8_t *y, float *s, hipStream_t stream) {
  RowArgs p = row_args(x, rows, nullptr, false, tokens, top_k, h, y);
  p.scales = s;
  p.ue8m0 = ue8m0;
  const int nkb = (int)(h / kBlock);
  // few tokens: their blocks on more CUs (16 of 7168: 3.3 us, 4.5 on one workgroup a token)
  if (nkb <= kSpreadBlocks || tokens < 256) {
    const int64_t across = groups_of(nkb, kSpreadBlocks), slots = max(1, kSpreadBlocks / nkb);
    const dim3 grid(token_groups(groups_of(tokens, slots), across), (unsigned)across), block(kThreads);
    if (bf16)
      hipLaunchKernelGGL(dispatch_quant_kernel<true>, grid, block, 0, stream, p, nkb);
    else
      hipLaunchKernelGGL(dispatch_quant_kernel<false>, grid, block, 0, stream, p, nkb);
  } else {
    const dim3 grid(token_groups(tokens, 4)), block(64 * (unsigned)groups_of(min(nkb, kWideBlocks), 4));
    if (bf16)
      hipLaunchKernelGGL(dispatch_quant_wide_kernel<true>, grid, block, 0, stream, p, nkb);
    else
      hipLaunchKernelGGL(dispatch_quant_wide_kernel<false>, grid, block, 0, stream, p, nkb);
  }
  return hipGetLastError();
}

hipError_t launch_expert_combine(const void *y, bool bf16, const int32_t *rows, const void *weights, bool w_bf16,
                                 int64_t tokens, int64_t top_k, int64_t h, void *out, hipStream_t stream) {
  const RowArgs p = row_args(y, rows, weights, w_bf16, tokens, top_k, h, out);
  if (bf16)
    FP8BSQ_BY_WIDTH(combine_kernel, true, p, false);
  else
    FP8BSQ_BY_WIDTH(combine_kernel, false, p, false);
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const void *dout, const void *y, bool bf16, const int32_t *rows,
                                          const void *weights, bool w_bf16, int64_t tokens, int64_t top_k, int64_t h,
                                          void *dy, void *dweights, hipStream_t stream) {
  RowArgs p = row_args(dout, rows, weights, w_bf16, tokens, top_k, h, dy);
  p.y = y;
  p.scales = dweights;
  if (bf16)
    FP8BSQ_BY_WIDTH(combine_backward_kernel, true, p, true);
  else
    FP8BSQ_BY_WIDTH(combine_backward_kernel, false, p, true);
  return hipGetLastError();
}

#undef FP8BSQ_BY_WIDTH

}  // namespace fp8bsq
