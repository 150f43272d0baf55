// Device helpers of 4-bit weights.
#pragma once

#include "common.cuh"

namespace moe {

// A scale in both halves of a word.
__device__ __forceinline__ uint32_t q4_twice(bf16 s) {
  const uint32_t b = __bfloat16_as_ushort(s);
  return b | b << 16;
}
// Weights 2 i and 2 i + 1 of a word of codes: (code - 8) scale in bf16.  128 + code
// is the bf16 value whose last four bits are the code; taking 136 from it is exact,
// so the product is rounded once (not at all for scales of five bits: 3 bits by 5).
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int i, uint32_t scale2) {
  uint32_t b = ((word >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  const uint32_t c136 = 0x43084308u;
  __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b),
                             *reinterpret_cast<const __nv_bfloat162*>(&c136));
  v = __hmul2(v, *reinterpret_cast<const __nv_bfloat162*>(&scale2));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 q4_word(uint32_t word, uint32_t scale2) {
  return make_uint4(q4_pair(word, 0, scale2), q4_pair(word, 1, scale2), q4_pair(word, 2, scale2),
                    q4_pair(word, 3, scale2));
}

}  // namespace moe
