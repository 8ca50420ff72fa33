// Building blocks of the E4M3 matrix kernels: the MFMA forms, fragment loads,
// direct global->LDS transfers with their waits, and the LDS swizzle.
#pragma once

#include "device_common.h"

namespace fp8bsq {

__device__ __forceinline__ f32x4 mfma_e4m3_16x16x128(const i32x8 &a, const i32x8 &b, f32x4 c) {
  // format 0 = E4M3 for both operands; the literal zero scale operands select
  // the unscaled instruction (no block scaling inside the matrix core).
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// The same MFMA with each A row scaled by 2^(e - 127) inside the matrix core:
// lane l supplies the E8M0 exponent e of the row it feeds (row l % 16); the B
// scale is 1 (E8M0 127).
__device__ __forceinline__ f32x4 mfma_e4m3_16x16x128_mx(const i32x8 &a, const i32x8 &b, int e8m0_a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                          e8m0_a, 0, 127);
}

__device__ __forceinline__ i32x8 load_frag(const uint8_t *p) {
  const uint4 lo = *(const uint4 *)p;
  const uint4 hi = *(const uint4 *)(p + 16);
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z,
               (int)hi.w};
}

// Optional bias of the output's dtype, added to the FP32 accumulator before
// the output rounding; `bias` may be null.
__device__ __forceinline__ float bias_at(const void *bias, bool bf16, int64_t col) {
  if (!bias) return 0.0f;
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t *)bias)[col] << 16)
              : ((const float *)bias)[col];
}

__device__ __forceinline__ void store_out(void *c, bool bf16, int64_t idx, float v) {
  if (bf16)
    ((uint16_t *)c)[idx] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
  else
    ((float *)c)[idx] = v;
}

// LDS rows are 128 bytes (eight 16-byte chunks); chunk c of row r is stored at
// slot c ^ swz(r), so the 16 rows a fragment read touches hit distinct banks.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)((const __attribute__((address_space(3))) void *)p);
}

// 64 lanes x 16 bytes from base + voff (per lane) into LDS [lds, lds + 1024).
__device__ __forceinline__ void lds_dma16(const void *base, uint32_t voff, uint32_t lds) {
  asm volatile("global_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds) : "memory");
}

// active lanes x 4 bytes from base + voff into LDS [lds + 4 * lane].
__device__ __forceinline__ void lds_dma4(const void *base, uint32_t voff, uint32_t lds) {
  asm volatile("global_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds) : "memory");
}

__device__ __forceinline__ void wait_dma_all() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void workgroup_barrier() { asm volatile("s_barrier" ::: "memory"); }

__device__ __forceinline__ i32x8 frag_from_lds(const uint8_t *row_base, int fq, int r) {
  const uint4 *base = (const uint4 *)row_base;
  const uint4 lo = base[(2 * fq) ^ swz(r)];
  const uint4 hi = base[(2 * fq + 1) ^ swz(r)];
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

}  // namespace fp8bsq
