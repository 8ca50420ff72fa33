// Global gradient norm over many tensors, and clipping, for gfx950.
//
//     norm = sqrt(sum over all tensors of sum g^2)
//     out  = g * min(1, max_norm / (norm + eps))
//
// Two kernels: sums of squares, one FP64 partial per workgroup (the square of
// any finite fp32 is finite and exact enough there: no overflow at 1e30, no
// underflow at 1e-30), then the scaling, whose workgroups each add the
// partials in one fixed order, so a norm does not depend on which workgroup
// ran first.  Tensor addresses travel in the kernel arguments, kTableTensors a
// launch: nothing is uploaded and nothing kept between calls.  The tensors of a
// table form one sequence of chunks that the workgroups walk.
//
// Bound by memory: the factor needs every gradient before the first is scaled,
// so they are read twice and written once.  396 M elements of bf16 (2.4 GB in
// all) take 435 us, 5.5 TB/s; the second pass backwards, for what the last cache
// still holds, took 440.  240 small tensors take the
// kernels 4.3 and 4.9 us, latency, and the caller's own thread 15 a call.
#include "ffn_launch.h"
#include "device_common.h"

namespace fp8bsq {
namespace {

// A launch's table: 8 KB of kernel arguments.  The runtime takes the segment's
// size from the code object; the tests fill a table to its last entry, eagerly and
// replayed from a graph.  A table more is a pair of launches more: 240 tensors took
// 27 us a call in three tables of 96, under 4 KB each, and 12 in one.
constexpr int kTableTensors = 256;
constexpr int kChunk = 16384;       // elements
constexpr int kClipBlocks = 1024;   // workgroups (and partials) per table, at most

struct Table {
  const void *g[kTableTensors];
  void *out[kTableTensors];
  int64_t numel[kTableTensors];
  int64_t first[kTableTensors];   // the tensor's first chunk
  uint32_t bf16[kTableTensors / 32];
  int32_t count;
  int64_t chunks;
};
static_assert(sizeof(Table) <= 8448, "no kernel argument segment larger than the tested one");

// The tensor that a chunk belongs to: the last one whose first chunk is not
// beyond it (tensors without elements have no chunk).  A wave holds all first
// chunks, loaded at once, and counts: a binary search in the kernel arguments
// waits for eight loads in a row (240 small tensors: 5.5 and 5.8 us a kernel,
// 4.3 and 4.9 so).
struct TensorOf {
  int64_t first[kTableTensors / 64];
  __device__ __forceinline__ explicit TensorOf(const Table &t) {
#pragma unroll
    for (int j = 0; j < kTableTensors / 64; ++j) {
      const int i = 64 * j + (threadIdx.x & 63);
      first[j] = i < t.count ? t.first[i] : INT64_MAX;
    }
  }
  __device__ __forceinline__ int operator()(int64_t chunk) const {
    int n = 0;
#pragma unroll
    for (int j = 0; j < kTableTensors / 64; ++j) n += __popcll(__ballot(first[j] <= chunk));
    return __builtin_amdgcn_readfirstlane(n - 1);
  }
};

// Gradients may be views at any element offset: the 16-byte accesses are
// unaligned ones.
__device__ __forceinline__ u32x4 load16(const void *p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ double square(double acc, float v) { return __builtin_fma((double)v, (double)v, acc); }

// Sum over the 256 threads of a workgroup, in a fixed order, for all of them.
__device__ __forceinline__ double block_sum(double v, double *lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__global__ __launch_bounds__(256) void square_sum_kernel(const Table tab, double *__restrict__ partials) {
  __shared__ double lds[4];
  const TensorOf find_tensor(tab);
  double acc = 0.0;
  for (int64_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    const int i = find_tensor(chunk);
    const int64_t at = (chunk - tab.first[i]) * kChunk;
    const int len = (int)min((int64_t)kChunk, tab.numel[i] - at);
    if ((tab.bf16[i >> 5] >> (i & 31)) & 1u) {
      const uint16_t *p = (const uint16_t *)tab.g[i] + at;
      const int nv = len / 8;
      for (int v = threadIdx.x; v < nv; v += 256) {
        const u32x4 w = load16(p + 8 * v);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc = square(square(acc, bf16_lo(w[c])), bf16_hi(w[c]));
      }
      const int r = 8 * nv + threadIdx.x;
      if (r < len) acc = square(acc, bf16_lo(p[r]));
    } else {
      const float *p = (const float *)tab.g[i] + at;
      const int nv = len / 4;
      for (int v = threadIdx.x; v < nv; v += 256) {
        const u32x4 w = load16(p + 4 * v);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc = square(acc, __uint_as_float(w[c]));
      }
      const int r = 4 * nv + threadIdx.x;
      if (r < len) acc = square(acc, p[r]);
    }
  }
  acc = block_sum(acc, lds);
  if (threadIdx.x == 0) partials[blockIdx.x] = acc;
}

// Norm and factor from all partials; the same in every workgroup.
__device__ __forceinline__ float clip_factor(const double *__restrict__ partials, int n, float max_norm, float eps,
                                             float *__restrict__ norm_out, double *lds) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) sum += partials[i];
  const float norm = (float)sqrt(block_sum(sum, lds));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  // compared before the division: 0 / 0 and infinity / infinity would be NaN,
  // where nothing is to be clipped.  A NaN norm stays NaN.
  const float bound = norm + eps;
  return max_norm >= bound ? 1.0f : max_norm / bound;
}

__global__ __launch_bounds__(256) void clip_norm_kernel(const double *__restrict__ partials, int n,
                                                        float *__restrict__ norm_out) {
  __shared__ double lds[4];
  clip_factor(partials, n, 0.0f, 0.0f, norm_out, lds);
}

__global__ __launch_bounds__(256) void clip_scale_kernel(const Table tab, const double *__restrict__ partials, int n,
                                                         float max_norm, float eps, float *__restrict__ norm_out) {
  __shared__ double lds[4];
  const TensorOf find_tensor(tab);
  const float f = clip_factor(partials, n, max_norm, eps, norm_out, lds);
  for (int64_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    const int i = find_tensor(chunk);
    if (f == 1.0f && tab.out[i] == tab.g[i]) continue;   // in place and nothing to clip
    const int64_t at = (chunk - tab.first[i]) * kChunk;
    const int len = (int)min((int64_t)kChunk, tab.numel[i] - at);
    if ((tab.bf16[i >> 5] >> (i & 31)) & 1u) {
      const uint16_t *p = (const uint16_t *)tab.g[i] + at;
      uint16_t *o = (uint16_t *)tab.out[i] + at;
      const int nv = len / 8;
      for (int v = threadIdx.x; v < nv; v += 256) {
        u32x4 w = load16(p + 8 * v);
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = pack_bf16x2(bf16_lo(w[c]) * f, bf16_hi(w[c]) * f);
        __builtin_memcpy(o + 8 * v, &w, 16);
      }
      const int r = 8 * nv + threadIdx.x;
      if (r < len) o[r] = (uint16_t)(pack_bf16x2(bf16_lo(p[r]) * f, 0.0f) & 0xFFFFu);
    } else {
      const float *p = (const float *)tab.g[i] + at;
      float *o = (float *)tab.out[i] + at;
      const int nv = len / 4;
      for (int v = threadIdx.x; v < nv; v += 256) {
        u32x4 w = load16(p + 4 * v);
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = __float_as_uint(__uint_as_float(w[c]) * f);
        __builtin_memcpy(o + 4 * v, &w, 16);
      }
      const int r = 4 * nv + threadIdx.x;
      if (r < len) o[r] = p[r] * f;
    }
  }
}

int64_t tables(int64_t count) { return (count + kTableTensors - 1) / kTableTensors; }

void fill(Table &t, const void *const *grads, void *const *outs, const int64_t *numel, const int32_t *dtypes,
          int64_t begin, int64_t count) {
  t.count = (int32_t)(count - begin < kTableTensors ? count - begin : kTableTensors);
  t.chunks = 0;
  for (uint32_t &w : t.bf16) w = 0;
  for (int i = 0; i < t.count; ++i) {
    t.g[i] = grads[begin + i];
    t.out[i] = outs ? outs[begin + i] : nullptr;
    t.numel[i] = numel[begin + i];
    t.first[i] = t.chunks;
    t.chunks += (t.numel[i] + kChunk - 1) / kChunk;
    if (dtypes[begin + i]) t.bf16[i >> 5] |= 1u << (i & 31);
  }
}

unsigned grid_of(const Table &t) { return (unsigned)(t.chunks < 1 ? 1 : t.chunks < kClipBlocks ? t.chunks : kClipBlocks); }

}  // namespace

size_t clip_workspace_bytes(int64_t count) {
  return (size_t)(count < 1 ? 1 : tables(count)) * kClipBlocks * sizeof(double);
}

hipError_t launch_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *numel,
                                 const int32_t *dtypes, int64_t count, float max_norm, float eps, float *norm,
                                 void *workspace, hipStream_t stream) {
  double *partials = (double *)workspace;
  int n = 0;
  Table t;
  for (int64_t begin = 0; begin < count; begin += kTableTensors) {
    fill(t, grads, outs, numel, dtypes, begin, count);
    const unsigned grid = grid_of(t);
    hipLaunchKernelGGL(square_sum_kernel, dim3(grid), dim3(256), 0, stream, t, partials + n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    n += (int)grid;
  }
  if (!outs || count == 0) {
    hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(256), 0, stream, partials, n, norm);
    return hipGetLastError();
  }
  for (int64_t begin = 0; begin < count; begin += kTableTensors) {
    if (count > kTableTensors) fill(t, grads, outs, numel, dtypes, begin, count);
    hipLaunchKernelGGL(clip_scale_kernel, dim3(grid_of(t)), dim3(256), 0, stream, t, partials, n, max_norm, eps,
                       begin == 0 ? norm : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp8bsq
