// The matrix product grouped by expert with 4-bit weights.
#include <float.h>

#include "kernels.h"
#include "q4.cuh"
#include "q4.h"

namespace moe {
namespace {

__device__ __forceinline__ float act_of(int act, float h1, float h3) {
  if (act == 2) return silu_f(h1) * h3;
  if (act == 1) return gelu_tanh_f(h1);
  return act == 0 && h1 < 0.f ? 0.f : h1;        // a NaN stays one
}

// A block: one row, 64 outputs; a warp takes eight of them, its lanes words of K.
__global__ void __launch_bounds__(256) q4_rows_kernel(const Q4Product p) {
  __shared__ int expert;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks_n = (p.N + 63) / 64;
  const int r = blockIdx.x / blocks_n, n0 = (blockIdx.x % blocks_n) * 64 + warp * 8;
  pdl_begin();
  if (threadIdx.x == 0) {
    int prev = p.offsets ? min(max(p.offsets[0], 0), p.R) : 0;
    expert = p.offsets ? -1 : 0;
    for (int e = 0; p.offsets && e < p.E; ++e) {
      const int hi = min(max(p.offsets[e + 1], prev), p.R);
      if (r >= prev && r < hi) { expert = e; break; }
      prev = hi;
    }
  }
  __syncthreads();
  const int e = expert, words = p.K / 8, groups = (p.K + p.G - 1) / p.G;
  if (e < 0) return;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const bf16*>(p.x) + (long long)r * p.K);
  for (int n = n0; n < min(n0 + 8, p.N); ++n) {
    float sum[2] = {0.f, 0.f};
    for (int m = 0; m < (p.act == 2 ? 2 : 1); ++m) {
      const uint32_t* codes = static_cast<const uint32_t*>(m ? p.codes3 : p.codes) +
                              ((long long)e * p.N + n) * words;
      const bf16* scales = static_cast<const bf16*>(m ? p.scales3 : p.scales) + (long long)e * groups * p.N + n;
      for (int j = lane; j < words; j += 32) {
        const uint4 w = q4_word(codes[j], 0x10001u * __bfloat16_as_ushort(scales[(long long)(j * 8 / p.G) * p.N])), v = x[j];
        const uint32_t a[4] = {w.x, w.y, w.z, w.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[m] = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), sum[m]);
          sum[m] = fmaf(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u), sum[m]);
        }
      }
      sum[m] = warp_sum(sum[m]);
    }
    if (p.bias != nullptr) sum[0] += p.bias[(long long)e * p.N + n];
    if (lane == 0)
      static_cast<bf16*>(p.c)[(long long)r * p.N + n] = __float2bfloat16_rn(act_of(p.act, sum[0], sum[1]));
  }
}

}  // namespace

cudaError_t launch_q4_product(const Q4Product& p, cudaStream_t st) {
  if (p.R > 16) return launch_q4_gemm(p, st);
  return launch_pdl(q4_rows_kernel, dim3((unsigned)p.R * ((p.N + 63) / 64)), dim3(256), 0, st, p);
}

}  // namespace moe
