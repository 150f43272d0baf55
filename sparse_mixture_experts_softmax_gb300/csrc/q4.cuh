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

// The weights of a word's eight codes, (code - 8) scale, for a scale of any bits (in both
// halves of scale2).  128 + code is the bf16 value whose last four bits are the code;
// taking 136 from it is exact, so the product is the only rounding.  SCALED: the weights
// times 2^-8 (also where the scale times 2^-8 would not be a bf16 value).
template <bool SCALED = false>
__device__ __forceinline__ uint4 q4_word(uint32_t w, uint32_t scale2) {
  constexpr uint32_t one = SCALED ? 0x3b803b80u : 0x3f803f80u, less = SCALED ? 0xbf08bf08u : 0xc308c308u;
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    v[i] = q4_fma(q4_fma(b, one, less), scale2, 0x80008000u);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// The same weights times 2^-8, for the products (whose results are multiplied with 2^8,
// exactly), with three instructions for two weights and a shift for eight.  A bf16 value
// whose bits are the number b, 0 <= b < 256, is b 2^-133: so are the smallest (subnormal)
// ones and, beyond 127, the first of the others.  A code in the lower four bits of that
// byte or in its upper four is then a multiple of 2^-133 or 2^-129 as it stands, and
//   code 2^-133 (scale 2^125) - scale 2^-5  =  (code - 8) scale 2^-8
// is one fma, whose only rounding is that of the weight.  The scales for which those
// factors are normal numbers, 2^-121 to 2^3, take it; a warp with another among its
// lanes' goes by q4_word.  Either way a weight below 2^-118 is rounded to a multiple of
// 2^-125 (its 2^-8 to one of 2^-133, the least bf16 number).
//
// Widening is what bounds the products next to HBM.  Measured with every word by q4_word
// and with the short way: one token of the large layer 59.4 and 47.1 us, 64 tokens 578 and
// 388 (decode.cu); its up projection for 32768 rows 868 and 800 (q4_gemm.cu).
constexpr float Q4_UNSCALE = 256.f;
// Bits 15 and 31: whether the two bf16 scales of a word take it (as zeros do).
__device__ __forceinline__ uint32_t q4_fast(uint32_t scales) {
  const uint32_t m = scales & 0x7fff7fffu;
  return (~(m + 0x7fff7fffu) | (m + 0x7d007d00u)) & (0xc0ffc0ffu - m);
}
// Two runs of 32 inputs; bits0, bits1: their scales.
template <bool FAST>
__device__ __forceinline__ void q4_runs(const uint4& w0, const uint4& w1, uint32_t bits0, uint32_t bits1,
                                        uint4 (&v)[2][4]) {
  const uint32_t r[2][4] = {{w0.x, w0.y, w0.z, w0.w}, {w1.x, w1.y, w1.z, w1.w}};
  const uint32_t two[2] = {__byte_perm(bits0, 0u, 0x1010), __byte_perm(bits1, 0u, 0x1010)};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (FAST) {
      const uint32_t low = q4_fma(two[u], 0x7e007e00u, 0x80008000u);             // 2^125
      const uint32_t high = q4_fma(two[u], 0x7c007c00u, 0x80008000u);            // 2^121
      const uint32_t add = q4_fma(two[u], 0xbd00bd00u, 0x80008000u);             // -2^-5
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = r[u][i], x = w >> 8;
        v[u][i] = make_uint4(q4_fma(w & 0x000f000fu, low, add), q4_fma(w & 0x00f000f0u, high, add),
                             q4_fma(x & 0x000f000fu, low, add), q4_fma(x & 0x00f000f0u, high, add));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[u][i] = q4_word<true>(r[u][i], two[u]);
    }
  }
}

// Inclusive scan over the threads of a block (those without a value pass a neutral one):
// the running maximum or the running sum.  part: 32 words of shared memory of its own.
template <bool MAX>
__device__ __forceinline__ int q4_block_scan(int v, int* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = MAX ? max(v, u) : v + u;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v = MAX ? max(v, part[w]) : v + part[w];
  return v;
}
// Thread e's offset, e <= E, of the given ones (nullptr: one expert with all R rows)
// clamped to a sequence that does not decrease within [0, R].  By the whole block, of more
// than E threads.
__device__ __forceinline__ int clamped_offset(const int* offsets, int E, int R, int* part) {
  const int e = threadIdx.x;
  int v = 0;
  if (e <= E) v = offsets != nullptr ? min(max(offsets[e], 0), R) : e * R;
  return q4_block_scan<true>(v, part);
}

}  // namespace moe
