// Weights to 4 bits and back.
//
// Both directions are bound by HBM (2 or 4 bytes of a weight on one side, half a
// byte and its share of a scale on the other).  A warp takes 256 inputs of eight
// outputs: a lane eight inputs of each, which are one word of codes, so that every
// access of the warp is a run of whole sectors; the scales of the eight outputs, next
// to one another in memory, are one 16-byte access of a group's first lane.
//
// Measured, of a copy's 6.79 TB/s: 2^30 bf16 weights to 4 bits 497 us, 5.4 TB/s (beside
// HBM the instructions for a code count: with a division and a comparison it was 1.00
// ms); 2^29 fp32 weights 359 us, 6.8; back to bf16 (2^30) 397 us, 6.8; back to fp32 (2^29) 520 us,
// 4.7 (a lane's two 16-byte stores are 32 bytes apart from the next lane's).
#include "kernels.h"
#include "q4.cuh"
#include "q4.h"

namespace moe {
namespace {

constexpr int WARPS = 4, ROWS = 8;

// Eight inputs of an output as they lie in memory.
template <typename T> struct Eight;
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  // the largest magnitude's bits; an infinity and a NaN are larger than every number
  __device__ __forceinline__ uint32_t amax() const {
    float v[8];
    get(v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
  }
};
template <> struct Eight<bf16> {
  uint4 q;
  __device__ __forceinline__ void load(const bf16* p) { q = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { q = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t u[4] = {q.x & 0x7fff7fffu, q.y & 0x7fff7fffu, q.z & 0x7fff7fffu, q.w & 0x7fff7fffu};
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(u);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
    return max(b << 16, b & 0xffff0000u);
  }
};

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
// of five significant bits that is not below a / 7 (below 2^-126, where an fp32 number has
// no leading bit of its own, the smallest multiple of 2^-130).  The four bits behind the
// first stay and what follows rounds up.  The factor is the largest fp32 value below 1 / 7, so
// the quotient is at most a last place too small, and 7 s, which is exact (3 bits by 5), tells
// where that has left s one step too small.
__device__ __forceinline__ float scale_of(float a) {
  const uint32_t b = (__float_as_uint(__fmul_rd(a, 0x1.249248p-3f)) + 0x7ffffu) & ~0x7ffffu;
  return __uint_as_float(7.0f * __uint_as_float(b) < a ? b + 0x80000u : b);
}

// The word of eight inputs' codes, for a scale of PLAIN at least.
//
// A sum with 1.5 2^23 + 8 is rounded to a whole number whose last bits are the code.
// Taken with 1 / scale a little (2^-20) too large and too small, the two sums differ only
// where the quotient is a border of two codes or next to one.  Their sum, twice as large,
// has a last place of 2: half of it is the number that both agree on, and where they
// differ the even one, as it has to be on a border.  bf16 weights (8 bits) are on a border
// (4 bits by 5) or 2^-9 apart from it; for fp32 weights `differ` tells what has to be
// taken again.  The words' shifts are multiplications, and what the sums have besides the
// codes is taken from the word at once.
constexpr float PLAIN = 0x1p-100f;
constexpr float CODE0 = 12582920.f;                      // 1.5 2^23 + 8
constexpr uint32_t SUM0 = 0x4bc00008u - 8u;              // of 2 CODE0, whose last bits are 8
__device__ __forceinline__ constexpr int shift_of(int i) { return 4 * (i / 2) + 16 * (i % 2); }
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], float scale, uint32_t& differ) {
  const float inv = __fdividef(1.0f, scale), more = inv * (1.0f + 0x1p-20f), less = inv * (1.0f - 0x1p-20f);
  uint32_t word = 0u, off = 0u;
  differ = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fmaf(v[i], more, CODE0), b = fmaf(v[i], less, CODE0);
    word += __float_as_uint(a + b) * (1u << shift_of(i));
    off += SUM0 * (1u << shift_of(i));
    differ |= __float_as_uint(a) ^ __float_as_uint(b);
  }
  return word - off;
}
// For any scale, the remainder, which is exact, deciding.
__device__ __noinline__ uint32_t codes_of_any(float v0, float v1, float v2, float v3, float v4, float v5,
                                              float v6, float v7, float scale) {
  const float v[8] = {v0, v1, v2, v3, v4, v5, v6, v7};
  if (!(scale > 0.f)) return 0x88888888u;        // a NaN or a zero: every code is 8
  // far from the smallest numbers, where 1 / scale is one
  const float up = scale < 0x1p-60f ? 0x1p64f : 1.f, sc = scale * up, inv = 1.0f / sc;
  const uint32_t half = __float_as_uint(0.5f * sc);
  uint32_t word = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // it may be one off next to a border; half a scale goes to the even code
    const float x = v[i] * up;
    float t = fmaf(x, inv, CODE0);
    const float rest = fmaf(-(t - CODE0), sc, x);
    if (fabsf(rest) > __uint_as_float(half - (__float_as_uint(t) & 1u))) t += copysignf(1.f, rest);
    word |= (__float_as_uint(t) & 15u) << shift_of(i);
  }
  return word;
}

template <int O>
__device__ __forceinline__ void max_over(uint32_t (&a)[ROWS]) {
#pragma unroll
  for (int r = 0; r < ROWS; ++r) a[r] = max(a[r], __shfl_xor_sync(0xffffffffu, a[r], O));
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32)
q4_quantize_kernel(const Q4Shape s, const T* __restrict__ w, uint32_t* __restrict__ codes,
                   bf16* __restrict__ scales) {
  Part p;
  pdl_begin();
  if (!my_part(s, p)) return;
  Eight<T> v[ROWS];
  const T* from = w + p.row * s.K + p.k;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (p.on) v[r].load(from + (long long)r * s.K);
    else v[r].clear();
  }
  uint32_t a[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) a[r] = v[r].amax();
  max_over<1>(a);
  max_over<2>(a);
  if (s.G > 32) max_over<4>(a);
  if (s.G > 64) max_over<8>(a);
  if (!p.on) return;
  float scale[ROWS];
  bool plain = true;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    scale[r] = a[r] < 0x7f800000u ? scale_of(__uint_as_float(a[r])) : __uint_as_float(0x7fc00000u);
    plain = plain && scale[r] >= PLAIN;
  }
  if (p.k % s.G == 0) {
    uint32_t two[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)        // (the lower 16 bits of a scale are zeros)
      two[i] = __byte_perm(__float_as_uint(scale[2 * i]), __float_as_uint(scale[2 * i + 1]), 0x7632);
    *reinterpret_cast<uint4*>(scales + scales_at(s, p)) = make_uint4(two[0], two[1], two[2], two[3]);
  }
  uint32_t* to = codes + (p.row * s.K + p.k) / 8;
#pragma unroll
  for (int r = 0; r < ROWS; ++r, to += s.K / 8) {
    float x[8];
    v[r].get(x);
    uint32_t differ, word;
    if (plain) word = codes_of(x, scale[r], differ);
    if (!plain || (sizeof(T) == 4 && differ != 0u))
      word = codes_of_any(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], scale[r]);
    *to = word;
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
