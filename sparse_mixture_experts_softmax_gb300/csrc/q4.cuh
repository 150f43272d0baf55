// Device helpers of 4-bit weights.
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ uint32_t q4_fma(uint32_t a, uint32_t b, uint32_t c) {
  const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b),
                                   *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// What turns codes of one scale into weights, (code - 8) scale in bf16.
//
// With the code in the upper four bits of a bf16 mantissa behind 1, the value is
// (16 + code) / 16, and  (16 + code) / 16 (16 scale) - 24 scale  is the weight, in one
// fma and without a rounding where 24 scale is exact: 3 scale has two bits more than
// scale, so scales of up to six significant bits (whose last two bits of a bf16 are
// zeros) take it, beyond the smallest and largest numbers.  For other scales 128 +
// code, the code in the lower four bits of the mantissa, loses 136 (exact) and the
// product with the scale is rounded.  Both give the nearest bf16 value of the weight.
struct Q4Scale {
  uint32_t mul, add;           // both halves alike
  bool fast;
};
__device__ __forceinline__ Q4Scale q4_scale(uint32_t bits) {     // of a bf16 scale
  const uint32_t two = bits | bits << 16, mag = bits & 0x7fffu;
  Q4Scale s;
  s.fast = (bits & 3u) == 0u && mag >= 0x0800u && mag < 0x7800u;
  s.mul = two;
  s.add = 0u;
  if (s.fast) {
    s.mul = two + 0x02000200u;                                   // 16 scale
    s.add = q4_fma(two, 0xc1c0c1c0u, 0u);                        // -24 scale
  }
  return s;
}
// The weights of a word's eight codes.
__device__ __forceinline__ uint4 q4_word_fast(uint32_t w, const Q4Scale& s) {
  constexpr uint32_t M = 0x00780078u, ONE = 0x3f803f80u;
  return make_uint4(q4_fma(((w << 3) & M) | ONE, s.mul, s.add), q4_fma(((w >> 1) & M) | ONE, s.mul, s.add),
                    q4_fma(((w >> 5) & M) | ONE, s.mul, s.add), q4_fma(((w >> 9) & M) | ONE, s.mul, s.add));
}
__device__ __forceinline__ uint32_t q4_pair_any(uint32_t w, uint32_t scale2) {
  uint32_t b = (w & 0x000f000fu) | 0x43004300u;
  const uint32_t c136 = 0x43084308u;
  __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b),
                             *reinterpret_cast<const __nv_bfloat162*>(&c136));
  v = __hmul2(v, *reinterpret_cast<const __nv_bfloat162*>(&scale2));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 q4_word_any(uint32_t w, const Q4Scale& s) {
  return make_uint4(q4_pair_any(w, s.mul), q4_pair_any(w >> 4, s.mul), q4_pair_any(w >> 8, s.mul),
                    q4_pair_any(w >> 12, s.mul));
}
__device__ __forceinline__ uint4 q4_word(uint32_t w, const Q4Scale& s) {
  return s.fast ? q4_word_fast(w, s) : q4_word_any(w, s);
}
// Four words of one scale, one branch.
__device__ __forceinline__ void q4_words(const uint4& w, const Q4Scale& s, uint4 (&v)[4]) {
#ifdef QM
  if (QM == 0) { v[0] = v[1] = v[2] = v[3] = make_uint4(w.x, w.y, w.z, w.w ^ s.mul); return; }
  if (QM == 1) { v[0] = q4_word_fast(w.x, s); v[1] = q4_word_fast(w.y, s);
    v[2] = q4_word_fast(w.z, s); v[3] = q4_word_fast(w.w, s); return; }
  if (QM == 2) { v[0] = q4_word_any(w.x, s); v[1] = q4_word_any(w.y, s);
    v[2] = q4_word_any(w.z, s); v[3] = q4_word_any(w.w, s); return; }
#endif
  if (s.fast) {
    v[0] = q4_word_fast(w.x, s); v[1] = q4_word_fast(w.y, s);
    v[2] = q4_word_fast(w.z, s); v[3] = q4_word_fast(w.w, s);
  } else {
    v[0] = q4_word_any(w.x, s); v[1] = q4_word_any(w.y, s);
    v[2] = q4_word_any(w.z, s); v[3] = q4_word_any(w.w, s);
  }
}

}  // namespace moe
