// Weights to 4 bits and back.
//
// Both directions are bound by HBM (2 or 4 bytes of a weight on one side, half a
// byte and its share of a scale on the other).  A warp takes 256 inputs of eight
// outputs: a lane eight inputs of each, which are one word of codes, so that every
// access of the warp is a run of whole sectors; the scales of the eight outputs, next
// to one another in memory, are one 16-byte access of a group's first lane.
#include "kernels.h"
#include "q4.cuh"
#include "q4.h"

namespace moe {
namespace {

constexpr int WARPS = 4, ROWS = 8;

template <typename T> __device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <> __device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <> __device__ __forceinline__ void load8<bf16>(const bf16* p, float (&v)[8]) {
  const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// The part of a matrix that falls to a warp: its first output (of all experts) and
// this lane's first input.
struct Part {
  long long row;
  int k, e, n;
  bool on;                     // the lane has inputs
};
__device__ __forceinline__ bool my_part(const Q4Shape& s, Part& p) {
  const int segments = (s.K + 255) / 256;
  const long long task = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
  const long long block = task / segments;
  p.row = block * ROWS;
  if (p.row >= (long long)s.E * s.N) return false;
  p.k = (int)(task - block * segments) * 256 + (threadIdx.x & 31) * 8;
  p.e = (int)(p.row / s.N);
  p.n = (int)(p.row - (long long)p.e * s.N);
  p.on = p.k < s.K;
  return true;
}
__device__ __forceinline__ long long scales_at(const Q4Shape& s, const Part& p) {
  return ((long long)p.e * ((s.K + s.G - 1) / s.G) + p.k / s.G) * s.N + p.n;
}

// The scale of a group whose largest magnitude is a (finite, >= 0): the smallest value
// of five significant bits that is not below a / 7.  The four bits behind the first stay
// and what follows rounds up; 7 s is exact (3 bits by 5), so it tells where the division
// has rounded down to s.
__device__ __forceinline__ float scale_of(float a) {
  const uint32_t b = (__float_as_uint(a / 7.0f) + 0x7ffffu) & ~0x7ffffu;
  return __uint_as_float(7.0f * __uint_as_float(b) < a ? b + 0x80000u : b);
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32)
q4_quantize_kernel(const Q4Shape s, const T* __restrict__ w, uint32_t* __restrict__ codes,
                   bf16* __restrict__ scales) {
  Part p;
  pdl_begin();
  if (!my_part(s, p)) return;
  float v[ROWS][8];
  const T* from = w + p.row * s.K + p.k;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (p.on) load8(from + (long long)r * s.K, v[r]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) v[r][i] = 0.f;
  }
  float scale[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    // as whole numbers: an infinity and a NaN are larger than every finite value
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[r][i]) & 0x7fffffffu);
    for (int o = 1; o < s.G / 8; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    scale[r] = a < 0x7f800000u ? scale_of(__uint_as_float(a)) : __uint_as_float(0x7fc00000u);
  }
  if (!p.on) return;
  if (p.k % s.G == 0) {
    uint32_t two[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)        // (the lower 16 bits of a scale are zeros)
      two[i] = __float_as_uint(scale[2 * i]) >> 16 | (__float_as_uint(scale[2 * i + 1]) & 0xffff0000u);
    *reinterpret_cast<uint4*>(scales + scales_at(s, p)) = make_uint4(two[0], two[1], two[2], two[3]);
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    uint32_t word = 0x88888888u;
    if (scale[r] > 0.f) {              // (a NaN or a zero: every code is 8)
      // far from the smallest numbers, where 1 / scale is one
      const float up = scale[r] < 0x1p-60f ? 0x1p64f : 1.f;
      const float sc = scale[r] * up, inv = 1.0f / sc;
      const uint32_t half = __float_as_uint(0.5f * sc);
      word = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = v[r][i] * up;
        // 1.5 2^23 + 8: a sum with it is rounded to a whole number, and its last bits
        // are the code.  It may be one off next to a border (1 / scale is rounded), so
        // the remainder, which is exact, decides; half a scale goes to the even code.
        float t = fmaf(x, inv, 12582920.f);
        const float rest = fmaf(-(t - 12582920.f), sc, x);
        if (fabsf(rest) > __uint_as_float(half - (__float_as_uint(t) & 1u)))
          t += copysignf(1.f, rest);
        word |= (__float_as_uint(t) & 15u) << (4 * (i / 2) + 16 * (i % 2));
      }
    }
    codes[((p.row + r) * s.K + p.k) / 8] = word;
  }
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32)
q4_dequantize_kernel(const Q4Shape s, const uint32_t* __restrict__ codes,
                     const bf16* __restrict__ scales, T* __restrict__ w) {
  Part p;
  pdl_begin();
  if (!my_part(s, p) || !p.on) return;
  uint32_t word[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) word[r] = __ldcs(codes + ((p.row + r) * s.K + p.k) / 8);
  const uint4 q = __ldg(reinterpret_cast<const uint4*>(scales + scales_at(s, p)));
  const uint32_t two[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const uint4 v = q4_word(word[r], __byte_perm(two[r / 2], 0u, r % 2 ? 0x3232 : 0x1010));
    T* to = w + (p.row + r) * s.K + p.k;
    if constexpr (sizeof(T) == 2) {
      __stcs(reinterpret_cast<uint4*>(to), v);
    } else {
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        __stcs(reinterpret_cast<uint4*>(to) + h,
               make_uint4(u[2 * h] << 16, u[2 * h] & 0xffff0000u, u[2 * h + 1] << 16,
                          u[2 * h + 1] & 0xffff0000u));
    }
  }
}

long long blocks_of(const Q4Shape& s) {
  const long long tasks = (long long)s.E * (s.N / ROWS) * ((s.K + 255) / 256);
  return (tasks + WARPS - 1) / WARPS;
}

}  // namespace

cudaError_t launch_q4_quantize(int type, const Q4Shape& s, const void* w, void* codes, void* scales,
                               cudaStream_t st) {
  const dim3 grid((unsigned)blocks_of(s)), block(WARPS * 32);
  if (type == 1)
    return launch_pdl(q4_quantize_kernel<bf16>, grid, block, 0, st, s, static_cast<const bf16*>(w),
                      static_cast<uint32_t*>(codes), static_cast<bf16*>(scales));
  return launch_pdl(q4_quantize_kernel<float>, grid, block, 0, st, s, static_cast<const float*>(w),
                    static_cast<uint32_t*>(codes), static_cast<bf16*>(scales));
}

cudaError_t launch_q4_dequantize(int type, const Q4Shape& s, const void* codes, const void* scales,
                                 void* w, cudaStream_t st) {
  const dim3 grid((unsigned)blocks_of(s)), block(WARPS * 32);
  if (type == 1)
    return launch_pdl(q4_dequantize_kernel<bf16>, grid, block, 0, st, s,
                      static_cast<const uint32_t*>(codes), static_cast<const bf16*>(scales),
                      static_cast<bf16*>(w));
  return launch_pdl(q4_dequantize_kernel<float>, grid, block, 0, st, s,
                    static_cast<const uint32_t*>(codes), static_cast<const bf16*>(scales),
                    static_cast<float*>(w));
}

}  // namespace moe
