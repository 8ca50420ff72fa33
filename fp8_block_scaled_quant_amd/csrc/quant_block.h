// act_quant's arithmetic on 16 lanes that share a 1 x 128 block, eight values each.
// Include only from translation units compiled with FP contraction off.
#pragma once

#include "quant_common.h"

namespace fp8bsq {

// One 1 x 128 block on 16 lanes, eight values each: codes and scale.
template <bool kBf16>
__device__ __forceinline__ u32x2 quantize_block(const u32x4 (&v)[kBf16 ? 1 : 2], bool ue8m0, float &s) {
  float r;
  if constexpr (kBf16) {
    u16x2 m2 = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(u16x2, v[0][j] & 0x7FFF7FFFu));
    block_scale_fast(row_max_u32((uint32_t)(m2.x > m2.y ? m2.x : m2.y) << 16), ue8m0, s, r);
    return encode_chunk_bf16(v[0], s, r);
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max(v[0][j] & 0x7FFFFFFFu, v[1][j] & 0x7FFFFFFFu));
    block_scale(row_max_u32(top), ue8m0, s, r);
    return u32x2{encode_chunk_f32(v[0], s), encode_chunk_f32(v[1], s)};
  }
}

template <bool kBf16>
__device__ __forceinline__ void load_block(const void *x, int64_t block, int sub, u32x4 (&v)[kBf16 ? 1 : 2]) {
  if constexpr (kBf16) {
    v[0] = ((const u32x4 *)x)[block * 16 + sub];
  } else {
    v[0] = ((const u32x4 *)x)[block * 32 + 2 * sub];
    v[1] = ((const u32x4 *)x)[block * 32 + 2 * sub + 1];
  }
}

}  // namespace fp8bsq
