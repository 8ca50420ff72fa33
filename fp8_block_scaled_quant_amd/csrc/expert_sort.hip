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
//
// Bound by the latency of its steps, not by its bytes.  Measured, of 256 experts, the
// kernels: 8 choices 2.1 us; 65536 choices 2.8 and 7.1.  Whole calls: 64 choices 5.0 us
// (the host's part; by counting over one wave 8.0), 4096 6.4, 65536 9.3, 2^20 21.
// Smaller shares than kChunk choices cost more in counts to add up (2^18 choices: 15.7
// us with 1024, 12.8 with 2048).
#include "device_common.h"
#include "expert_launch.h"

namespace fp8bsq {
namespace {

constexpr int kMaxWaves = 16;
constexpr int64_t kFew = 16;            // choices that one wave counts over
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
  // [wave][num + 1] counts, then places; [num + 1] all choices' counts, then where
  // buckets begin; [num + 1] choices in the workgroups before
  extern __shared__ uint32_t lds[];
  const int buckets = p.num + 1, waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t *mine = lds + wave * buckets, *first = lds + waves * buckets, *before = first + buckets;

  const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min(p.n, begin + p.chunk);
  const int64_t per = ((end - begin + blockDim.x - 1) / blockDim.x) * 64;   // choices a wave, whole rounds
  const int64_t wbegin = begin + wave * per, wend = min(end, wbegin + per);
  // the buckets of the wave's first rounds stay in registers
  constexpr int kHeld = 4;
  int held[kHeld];
#pragma unroll
  for (int r = 0; r < kHeld; ++r) {
    const int64_t c = wbegin + 64 * r + lane;
    held[r] = c < wend ? bucket_of<kWide>(p, c) : -1;
  }
  for (int b = threadIdx.x; b < (waves + 2) * buckets; b += blockDim.x) lds[b] = 0;
  __syncthreads();

  // each bucket's choices in the workgroups before this one, and in all: shares of
  // the workgroups by as many threads as there are, several loads in flight each
  if (p.groups > 1) {
    const int parts = max(1, (int)blockDim.x / buckets), share = (p.groups + parts - 1) / parts;
    for (int i = threadIdx.x; i < parts * buckets; i += blockDim.x) {
      const int part = i / buckets, b = i - part * buckets, g1 = min(p.groups, (part + 1) * share);
      uint32_t prior = 0, all = 0;
      constexpr int kTogether = 12;
      for (int g0 = part * share; g0 < g1; g0 += kTogether) {
        uint32_t v[kTogether];
#pragma unroll
        for (int g = 0; g < kTogether; ++g) v[g] = p.counts[(int64_t)min(g0 + g, g1 - 1) * buckets + b];
#pragma unroll
        for (int g = 0; g < kTogether; ++g) {
          prior += g0 + g < min(g1, (int)blockIdx.x) ? v[g] : 0;
          all += g0 + g < g1 ? v[g] : 0;
        }
      }
      atomicAdd(&first[b], all);
      atomicAdd(&before[b], prior);
    }
  }
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (held[r] >= 0) atomicAdd(&mine[held[r]], 1u);
  for (int64_t c = wbegin + 64 * kHeld + lane; c < wend; c += 64) atomicAdd(&mine[bucket_of<kWide>(p, c)], 1u);
  __syncthreads();

  // the waves' counts to the numbers of choices before theirs
  for (int b = threadIdx.x; b < buckets; b += blockDim.x) {
    uint32_t v[kMaxWaves], at = before[b];
#pragma unroll
    for (int w = 0; w < kMaxWaves; ++w) v[w] = lds[min(w, waves - 1) * buckets + b];
#pragma unroll
    for (int w = 0; w < kMaxWaves; ++w) {
      if (w >= waves) break;
      lds[w * buckets + b] = at;
      at += v[w];
    }
    if (p.groups == 1) first[b] = at;
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

  constexpr int kMaxBits = 11;
  static_assert(kMaxExperts < 1 << kMaxBits, "a bucket's number");
  const int bits = 32 - __builtin_clz(p.num);
  auto place = [&](int64_t c, int b) {   // b below 0: no choice
    const uint64_t there = __ballot(b >= 0);
    uint32_t lo = (uint32_t)there, hi = (uint32_t)(there >> 32);
#pragma unroll
    for (int i = 0; i < kMaxBits; ++i) {
      if (i >= bits) break;
      const uint32_t bit = (uint32_t)(b << (31 - i) >> 31);   // all ones where it is set
      const uint64_t set = __ballot(bit != 0);
      lo &= ~((uint32_t)set ^ bit);
      hi &= ~((uint32_t)(set >> 32) ^ bit);
    }
    const uint64_t same = (uint64_t)hi << 32 | lo;
    if (b >= 0) {
      const uint32_t below = (uint32_t)__popcll(same & (((uint64_t)1 << lane) - 1));
      const uint32_t next = mine[b];
      const uint32_t row = first[b] + next + below;
      p.rows[c] = (int32_t)(b < p.num ? row : ~row);
      p.choices[row] = (int32_t)c;
      // Lanes of one bucket read the counter, and one of them writes it.  The hardware
      // executes a wave's LDS accesses in order; the fences, no instructions themselves,
      // hold the compiler to it: the write stays behind these reads, and the next
      // round's reads behind the write.
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (below == 0) mine[b] = next + (uint32_t)__popcll(same);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (wbegin + 64 * r < wend) place(wbegin + 64 * r + lane, held[r]);
  for (int64_t c = wbegin + 64 * kHeld + lane; c - lane < wend; c += 64) place(c, c < wend ? bucket_of<kWide>(p, c) : -1);
}

// Up to kFew choices: every wave holds them all, and a choice's row and an expert's
// offset are counts over them.
template <bool kWide>
__global__ __launch_bounds__(256) void sort_few_kernel(const SortArgs p) {
  const int lane = threadIdx.x & 63, n = (int)p.n;
  const int mine = lane < n ? bucket_of<kWide>(p, lane) : 0x7FFFFFFF;
  if (threadIdx.x < 64) {
    int row = 0;
    for (int c = 0; c < n; ++c) {
      const int b = __builtin_amdgcn_readlane(mine, c);
      row += b < mine || (b == mine && c < lane) ? 1 : 0;
    }
    if (lane < n) {
      p.rows[lane] = mine < p.num ? row : ~row;
      p.choices[row] = lane;
    }
  }
  for (int e = threadIdx.x; e <= p.num; e += blockDim.x) {
    int below = 0;
    for (int c = 0; c < n; ++c) below += __builtin_amdgcn_readlane(mine, c) < e ? 1 : 0;
    p.offsets[e] = below;
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
  if (n <= kFew) {
    if (wide)
      hipLaunchKernelGGL(sort_few_kernel<true>, dim3(1), dim3(256), 0, stream, p);
    else
      hipLaunchKernelGGL(sort_few_kernel<false>, dim3(1), dim3(256), 0, stream, p);
    return hipGetLastError();
  }
  if (plan.groups > 1) {
    if (wide)
      hipLaunchKernelGGL(sort_count_kernel<true>, grid, block, table, stream, p);
    else
      hipLaunchKernelGGL(sort_count_kernel<false>, grid, block, table, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (wide)
    hipLaunchKernelGGL(sort_place_kernel<true>, grid, block, (plan.waves + 2) * table, stream, p);
  else
    hipLaunchKernelGGL(sort_place_kernel<false>, grid, block, (plan.waves + 2) * table, stream, p);
  return hipGetLastError();
}

}  // namespace fp8bsq
