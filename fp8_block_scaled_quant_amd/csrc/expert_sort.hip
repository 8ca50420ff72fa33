// The stable sort of choices by expert, for gfx950: a counting sort.
//
// Choice c of expert e goes to row
//     #{choices of experts below e} + #{choices of e before c}.
// Choices whose number is no expert's take part as one more bucket behind the
// others, so that every row belongs to exactly one choice; their rows are handed
// out as ~row.
//
// A workgroup owns consecutive choices, each of its waves a consecutive part of
// these.  The first kernel counts every workgroup's buckets; the second adds up
// the counts of the workgroups before its own, counts its waves' buckets, and
// then hands out rows 64 choices at a time: the lanes of one bucket find each
// other by ballots over the bucket number's bits, a lane's place among them is
// the number of such lanes below it, and the first of them moves the wave's
// counter on.  Every count is a sum over a fixed set, so equal calls give equal
// rows.  Up to kSingle choices one workgroup does it all, without the first kernel.
#include "device_common.h"
#include "expert_launch.h"

namespace fp8bsq {
namespace {

constexpr int kMaxWaves = 16;
constexpr int64_t kSingle = 4096;       // choices of a single workgroup
constexpr int64_t kChunk = 2048;        // choices a workgroup, at least, of several
constexpr int64_t kMaxGroups = 256;     // whose counts every workgroup reads

struct SortArgs {
  const void *experts;
  int64_t n, chunk;          // choices; choices a workgroup, a multiple of 64 * kMaxWaves where there are several
  int num, groups;           // experts; workgroups
  int32_t *offsets, *rows, *choices;
  uint32_t *counts;          // [group][num + 1], several workgroups only
};

template <bool kWide>
__device__ __forceinline__ int bucket_of(const SortArgs &p, int64_t c) {
  const int64_t id = kWide ? ((const int64_t *)p.experts)[c] : (int64_t)((const int32_t *)p.experts)[c];
  return id >= 0 && id < p.num ? (int)id : p.num;
}

template <bool kWide>
__global__ __launch_bounds__(64 * kMaxWaves) void sort_count_kernel(const SortArgs p) {
  extern __shared__ uint32_t count[];   // [num + 1]
  for (int b = threadIdx.x; b <= p.num; b += blockDim.x) count[b] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min(p.n, begin + p.chunk);
  for (int64_t c = begin + threadIdx.x; c < end; c += blockDim.x) atomicAdd(&count[bucket_of<kWide>(p, c)], 1u);
  __syncthreads();
  for (int b = threadIdx.x; b <= p.num; b += blockDim.x) p.counts[(int64_t)blockIdx.x * (p.num + 1) + b] = count[b];
}

template <bool kWide>
__global__ __launch_bounds__(64 * kMaxWaves) void sort_place_kernel(const SortArgs p) {
  // [wave][num + 1] next rows, then [num + 1] all choices' counts and where buckets begin
  extern __shared__ uint32_t lds[];
  const int buckets = p.num + 1, waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t *mine = lds + wave * buckets, *first = lds + waves * buckets;
  for (int b = threadIdx.x; b < waves * buckets; b += blockDim.x) lds[b] = 0;
  __syncthreads();

  const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min(p.n, begin + p.chunk);
  const int64_t per = ((end - begin + blockDim.x - 1) / blockDim.x) * 64;   // choices a wave, whole rounds
  const int64_t wbegin = begin + wave * per, wend = min(end, wbegin + per);
  for (int64_t c = wbegin + lane; c < wend; c += 64) atomicAdd(&mine[bucket_of<kWide>(p, c)], 1u);
  __syncthreads();

  // each bucket's choices: of the waves before (kept), of the workgroups before, of all
  for (int b = threadIdx.x; b < buckets; b += blockDim.x) {
    uint32_t before = 0, all = 0;
    if (p.groups > 1) {
#pragma unroll 8
      for (int g = 0; g < p.groups; ++g) {
        const uint32_t v = p.counts[(int64_t)g * buckets + b];
        before += g < (int)blockIdx.x ? v : 0;
        all += v;
      }
    }
    for (int w = 0; w < waves; ++w) {
      const uint32_t v = lds[w * buckets + b];
      lds[w * buckets + b] = before;
      before += v;
    }
    first[b] = p.groups > 1 ? all : before;
  }
  __syncthreads();

  // where buckets begin: the first wave, a lane consecutive buckets
  if (wave == 0) {
    const int per_lane = (buckets + 63) / 64, b0 = min(lane * per_lane, buckets), b1 = min(b0 + per_lane, buckets);
    uint32_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += first[b];
    uint32_t scan = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t v = __shfl_up(scan, d);
      if (lane >= d) scan += v;
    }
    uint32_t at = scan - sum;
    for (int b = b0; b < b1; ++b) {
      const uint32_t v = first[b];
      first[b] = at;
      if (blockIdx.x == 0) p.offsets[b] = (int32_t)at;   // the last bucket begins where the experts' rows end
      at += v;
    }
  }
  __syncthreads();

  const int bits = 32 - __builtin_clz(p.num);
  for (int64_t c0 = wbegin; c0 < wend; c0 += 64) {
    const int64_t c = c0 + lane;
    const bool there = c < wend;
    const int b = there ? bucket_of<kWide>(p, c) : 0;
    uint64_t same = __ballot(there);
    for (int i = 0; i < bits; ++i) {
      const uint64_t set = __ballot((b >> i) & 1);
      same &= (b >> i) & 1 ? set : ~set;
    }
    if (there) {
      const uint32_t place = (uint32_t)__popcll(same & (((uint64_t)1 << lane) - 1));
      const uint32_t next = mine[b];
      const uint32_t row = first[b] + next + place;
      p.rows[c] = (int32_t)(b < p.num ? row : ~row);
      p.choices[row] = (int32_t)c;
      // after every lane's read above: a wave's LDS accesses are executed in order
      if (place == 0) mine[b] = next + (uint32_t)__popcll(same);
    }
  }
}

struct SortPlan {
  int64_t chunk;
  int groups, waves;
};

SortPlan sort_plan(int64_t n) {
  SortPlan p;
  if (n <= kSingle) {
    p.groups = 1;
    p.chunk = n;
    p.waves = (int)min((n + 63) / 64, (int64_t)kMaxWaves);
    if (p.waves == 0) p.waves = 1;   // no choices: the offsets all the same
    return p;
  }
  const int64_t groups = min((n + kChunk - 1) / kChunk, kMaxGroups);
  constexpr int64_t kRound = 64 * kMaxWaves;
  p.chunk = ((n + groups - 1) / groups + kRound - 1) / kRound * kRound;
  p.groups = (int)((n + p.chunk - 1) / p.chunk);
  p.waves = kMaxWaves;
  return p;
}

}  // namespace

size_t expert_sort_bytes(int64_t n, int64_t num_experts) {
  const SortPlan plan = sort_plan(n);
  return plan.groups > 1 ? (size_t)plan.groups * (size_t)(num_experts + 1) * sizeof(uint32_t) : 0;
}

hipError_t launch_expert_sort(const void *experts, bool wide, int64_t n, int64_t num_experts, int32_t *offsets,
                              int32_t *rows, int32_t *choices, void *workspace, hipStream_t stream) {
  const SortPlan plan = sort_plan(n);
  const SortArgs p = {experts, n, plan.chunk, (int)num_experts, plan.groups, offsets, rows, choices, (uint32_t *)workspace};
  const size_t table = (size_t)(num_experts + 1) * sizeof(uint32_t);
  const dim3 grid((unsigned)plan.groups), block(64 * plan.waves);
  if (plan.groups > 1) {
    if (wide)
      hipLaunchKernelGGL(sort_count_kernel<true>, grid, block, table, stream, p);
    else
      hipLaunchKernelGGL(sort_count_kernel<false>, grid, block, table, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (wide)
    hipLaunchKernelGGL(sort_place_kernel<true>, grid, block, (plan.waves + 1) * table, stream, p);
  else
    hipLaunchKernelGGL(sort_place_kernel<false>, grid, block, (plan.waves + 1) * table, stream, p);
  return hipGetLastError();
}

}  // namespace fp8bsq
