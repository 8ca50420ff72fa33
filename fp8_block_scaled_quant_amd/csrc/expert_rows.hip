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
// bound by memory.  A row number outside the sorted rows touches nothing.
#include "expert_launch.h"
#include "quant_block.h"

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

// Row of choice c: `live` whether an expert has it; below 0 where it is not to be touched.
__device__ __forceinline__ int row_of(const RowArgs &p, int64_t c, bool &live) {
  const int r = p.rows[c], at = r < 0 ? ~r : r;
  live = r >= 0 && r < p.nrows;
  return at < p.nrows ? at : -1;
}

__device__ __forceinline__ float weight_of(const RowArgs &p, int64_t c) {
  if (!p.weights) return 1.0f;
  return p.w_bf16 ? __uint_as_float((uint32_t)((const uint16_t *)p.weights)[c] << 16) : ((const float *)p.weights)[c];
}

// What a thread moves at a time: 16 bytes (kWide), or one element where rows do
// not start or end on 16 bytes.
template <bool kBf16, bool kWide>
struct Piece {
  static constexpr int kCount = !kWide ? 1 : kBf16 ? 8 : 4;
  float v[kCount];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] = 0.0f;
  }
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    if constexpr (kWide && kBf16) {
      const u32x4 w = *(const u32x4 *)((const uint16_t *)p + i);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[2 * c] = __uint_as_float(w[c] << 16);
        v[2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
      }
    } else if constexpr (kWide) {
      const f32x4 w = *(const f32x4 *)((const float *)p + i);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = w[c];
    } else if constexpr (kBf16) {
      v[0] = __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16);
    } else {
      v[0] = ((const float *)p)[i];
    }
  }
  __device__ __forceinline__ void store(void *p, int64_t i) const {
    if constexpr (kWide && kBf16) {
      u32x4 w;
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = pack_bf16x2(v[2 * c], v[2 * c + 1]);
      *(u32x4 *)((uint16_t *)p + i) = w;
    } else if constexpr (kWide) {
      *(f32x4 *)((float *)p + i) = f32x4{v[0], v[1], v[2], v[3]};
    } else if constexpr (kBf16) {
      ((uint16_t *)p)[i] = (uint16_t)(pack_bf16x2(v[0], 0.0f) & 0xFFFFu);
    } else {
      ((float *)p)[i] = v[0];
    }
  }
};

// Bits as they are: a copy keeps NaN's.
template <typename T>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(const RowArgs p, int64_t pieces) {
  const int64_t i = (int64_t)blockIdx.y * kThreads + threadIdx.x;
  if (i >= pieces) return;
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const T v = ((const T *)p.x)[t * pieces + i];
    for (int j = 0; j < p.top_k; ++j) {
      bool live;
      const int64_t at = row_of(p, t * p.top_k + j, live);
      if (at >= 0) ((T *)p.out)[at * pieces + i] = live ? v : T{};
    }
  }
}

// Sixteen lanes own a 1 x 128 block of a token's row.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void dispatch_quant_kernel(const RowArgs p, int nkb) {
  const int sub = threadIdx.x & 15;
  const int kb = blockIdx.y * (kThreads / 16) + (threadIdx.x >> 4);
  if (kb >= nkb) return;   // whole 16-lane groups
  // a row of zeros: its scale, that of the floor on amax
  float zero_s, unused;
  block_scale(0u, p.ue8m0, zero_s, unused);
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    u32x4 v[kBf16 ? 1 : 2];
    load_block<kBf16>(p.x, t * nkb + kb, sub, v);
    float s;
    const u32x2 codes = quantize_block<kBf16>(v, p.ue8m0, s);
    for (int j = 0; j < p.top_k; ++j) {
      bool live;
      const int64_t at = row_of(p, t * p.top_k + j, live);
      if (at < 0) continue;
      *(u32x2 *)((uint8_t *)p.out + (at * nkb + kb) * kBlock + 8 * sub) = live ? codes : u32x2{0, 0};
      if (sub == 0) ((float *)p.scales)[at * nkb + kb] = live ? s : zero_s;
    }
  }
}

constexpr int kGroup = 8;   // choices whose rows are in flight together

template <bool kBf16, bool kWide>
__global__ __launch_bounds__(kThreads) void combine_kernel(const RowArgs p) {
  using P = Piece<kBf16, kWide>;
  const int64_t i = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * P::kCount;
  if (i >= p.h) return;
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    P sum;
    sum.clear();
    for (int j0 = 0; j0 < p.top_k; j0 += kGroup) {
      P v[kGroup];
      float w[kGroup];
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        bool live = false;
        int64_t at = 0;
        if (j0 + j < p.top_k) at = row_of(p, t * p.top_k + j0 + j, live);
        w[j] = 0.0f;
        if (live) {
          w[j] = weight_of(p, t * p.top_k + j0 + j);
          v[j].load(p.x, at * p.h + i);
        } else {
          v[j].clear();   // and not 0 times what a row without an expert holds
        }
      }
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
#pragma unroll
        for (int c = 0; c < P::kCount; ++c) sum.v[c] = __builtin_fmaf(w[j], v[j].v[c], sum.v[c]);
    }
    sum.store(p.out, t * p.h + i);
  }
}

// A workgroup a token; its threads' partial dot products meet in LDS.
template <bool kBf16, bool kWide>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(const RowArgs p) {
  using P = Piece<kBf16, kWide>;
  __shared__ float partial[kThreads / 64][kGroup];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    for (int j0 = 0; j0 < p.top_k; j0 += kGroup) {
      int64_t at[kGroup];
      bool live[kGroup];
      float w[kGroup], dot[kGroup];
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        at[j] = -1;
        live[j] = false;
        w[j] = dot[j] = 0.0f;
        if (j0 + j < p.top_k) at[j] = row_of(p, t * p.top_k + j0 + j, live[j]);
        if (live[j]) w[j] = weight_of(p, t * p.top_k + j0 + j);
      }
      for (int64_t i = (int64_t)threadIdx.x * P::kCount; i < p.h; i += kThreads * P::kCount) {
        P d, v[kGroup];
        d.load(p.x, t * p.h + i);
        if (p.scales) {
#pragma unroll
          for (int j = 0; j < kGroup; ++j) {
            if (live[j])
              v[j].load(p.y, at[j] * p.h + i);
            else
              v[j].clear();
          }
#pragma unroll
          for (int j = 0; j < kGroup; ++j)
            if (live[j])
#pragma unroll
              for (int c = 0; c < P::kCount; ++c) dot[j] = __builtin_fmaf(d.v[c], v[j].v[c], dot[j]);
        }
        if (p.out) {
#pragma unroll
          for (int j = 0; j < kGroup; ++j) {
            if (at[j] < 0) continue;
            P g;
#pragma unroll
            for (int c = 0; c < P::kCount; ++c) g.v[c] = live[j] ? w[j] * d.v[c] : 0.0f;
            g.store(p.out, at[j] * p.h + i);
          }
        }
      }
      if (!p.scales) continue;
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
#pragma unroll
        for (int s = 32; s > 0; s /= 2) dot[j] += __shfl_xor(dot[j], s);
        if (lane == 0) partial[wave][j] = dot[j];
      }
      __syncthreads();
      if ((int)threadIdx.x < kGroup && j0 + (int)threadIdx.x < p.top_k) {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kThreads / 64; ++v) sum += partial[v][threadIdx.x];
        const int64_t c = t * p.top_k + j0 + threadIdx.x;
        if (p.w_bf16)
          ((uint16_t *)p.scales)[c] = (uint16_t)(pack_bf16x2(sum, 0.0f) & 0xFFFFu);
        else
          ((float *)p.scales)[c] = sum;
      }
      __syncthreads();   // before the next group's partials
    }
  }
}

// Workgroups along the tokens: fewer than 2^32 threads in a launch.
unsigned token_groups(int64_t tokens, int64_t across) {
  return (unsigned)min(tokens, ((int64_t)1 << 23) / across);
}

bool wide(const void *a, const void *b, const void *c, int64_t row_bytes) {
  return row_bytes % 16 == 0 && (((uintptr_t)a | (uintptr_t)b | (uintptr_t)c) & 15) == 0;
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

hipError_t launch_expert_dispatch(const void *x, bool bf16, const int32_t *rows, int64_t tokens, int64_t top_k,
                                  int64_t h, void *y, hipStream_t stream) {
  const RowArgs p = row_args(x, rows, nullptr, false, tokens, top_k, h, y);
  const int64_t bytes = h * (bf16 ? 2 : 4);
  const bool vec = wide(x, y, nullptr, bytes);
  const int64_t pieces = vec ? bytes / 16 : h, across = groups_of(pieces, kThreads);
  const dim3 grid(token_groups(tokens, across), (unsigned)across), block(kThreads);
  if (vec)
    hipLaunchKernelGGL(dispatch_kernel<u32x4>, grid, block, 0, stream, p, pieces);
  else if (bf16)
    hipLaunchKernelGGL(dispatch_kernel<uint16_t>, grid, block, 0, stream, p, pieces);
  else
    hipLaunchKernelGGL(dispatch_kernel<uint32_t>, grid, block, 0, stream, p, pieces);
  return hipGetLastError();
}

hipError_t launch_expert_dispatch_quant(const void *x, bool bf16, bool ue8m0, const int32_t *rows, int64_t tokens,
                                        int64_t top_k, int64_t h, uint8_t *y, float *s, hipStream_t stream) {
  RowArgs p = row_args(x, rows, nullptr, false, tokens, top_k, h, y);
  p.scales = s;
  p.ue8m0 = ue8m0;
  const int nkb = (int)(h / kBlock);
  const int64_t across = groups_of(nkb, kThreads / 16);
  const dim3 grid(token_groups(tokens, across), (unsigned)across), block(kThreads);
  if (bf16)
    hipLaunchKernelGGL(dispatch_quant_kernel<true>, grid, block, 0, stream, p, nkb);
  else
    hipLaunchKernelGGL(dispatch_quant_kernel<false>, grid, block, 0, stream, p, nkb);
  return hipGetLastError();
}

hipError_t launch_expert_combine(const void *y, bool bf16, const int32_t *rows, const void *weights, bool w_bf16,
                                 int64_t tokens, int64_t top_k, int64_t h, void *out, hipStream_t stream) {
  const RowArgs p = row_args(y, rows, weights, w_bf16, tokens, top_k, h, out);
  const bool vec = wide(y, out, nullptr, h * (bf16 ? 2 : 4));
  const int64_t across = groups_of(h, kThreads * (vec ? (bf16 ? 8 : 4) : 1));
  const dim3 grid(token_groups(tokens, across), (unsigned)across), block(kThreads);
#define FP8BSQ_COMBINE(BF, WIDE) hipLaunchKernelGGL((combine_kernel<BF, WIDE>), grid, block, 0, stream, p)
  if (bf16) {
    if (vec) FP8BSQ_COMBINE(true, true); else FP8BSQ_COMBINE(true, false);
  } else {
    if (vec) FP8BSQ_COMBINE(false, true); else FP8BSQ_COMBINE(false, false);
  }
#undef FP8BSQ_COMBINE
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const void *dout, const void *y, bool bf16, const int32_t *rows,
                                          const void *weights, bool w_bf16, int64_t tokens, int64_t top_k, int64_t h,
                                          void *dy, void *dweights, hipStream_t stream) {
  RowArgs p = row_args(dout, rows, weights, w_bf16, tokens, top_k, h, dy);
  p.y = y;
  p.scales = dweights;
  const bool vec = wide(dout, dweights ? y : nullptr, dy, h * (bf16 ? 2 : 4));
  const dim3 grid(token_groups(tokens, 1)), block(kThreads);
#define FP8BSQ_COMBINE(BF, WIDE) hipLaunchKernelGGL((combine_backward_kernel<BF, WIDE>), grid, block, 0, stream, p)
  if (bf16) {
    if (vec) FP8BSQ_COMBINE(true, true); else FP8BSQ_COMBINE(true, false);
  } else {
    if (vec) FP8BSQ_COMBINE(false, true); else FP8BSQ_COMBINE(false, false);
  }
#undef FP8BSQ_COMBINE
  return hipGetLastError();
}

}  // namespace fp8bsq
