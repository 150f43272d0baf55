// Layer norm over rows of D values with the residual add in front of it, and
// its backward pass with the residual gradient behind it.
//
//   forward    h = x + delta;  m = mean(h);  r = rsqrt(mean((h - m)^2) + eps);
//              z = (h - m) r gamma + beta
//   backward   xh = (h - m) r,  g = dz gamma:
//              dx = dres + r (g - mean(g) - xh mean(g xh)),
//              dgamma = sum_t dz xh,  dbeta = sum_t dz
//
// Both are bound by HBM: a row is read once, held on chip while its sums are
// formed, and written once (forward, 65536 x 4096, bf16 stream and an fp32 delta:
// 409 us, 6.56 TB/s).  The variance is the mean squared deviation
// from the row's mean (two reductions over registers, not sum(h^2) - m^2, which
// cancels when a row's offset is large against its spread).
#include "common.cuh"
#include "kernels.h"
#include "norm.h"

namespace moe {
namespace {

// W consecutive values, widened to fp32.  W = 8 and W = 4 need 16-byte aligned
// rows (D a multiple of 8); W = 1 takes any D.
template <typename T, int W> struct Row;
template <> struct Row<float, 8> {
  static __device__ __forceinline__ void load(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <> struct Row<bf16, 8> {
  static __device__ __forceinline__ void load(const bf16* p, float (&v)[8]) {
    Vec<bf16> q;
    q.load(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = q.get(i);
  }
  static __device__ __forceinline__ void store(bf16* p, const float (&v)[8]) {
    Vec<bf16> q;
#pragma unroll
    for (int i = 0; i < 8; ++i) q.set(i, v[i]);
    q.store(p);
  }
};
template <> struct Row<float, 4> {
  static __device__ __forceinline__ void load(const float* p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Row<bf16, 4> {
  static __device__ __forceinline__ void load(const bf16* p, float (&v)[4]) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
  }
};
template <typename T> struct Row<T, 1> {
  static __device__ __forceinline__ void load(const T* p, float (&v)[1]) { v[0] = to_f(*p); }
  static __device__ __forceinline__ void store(T* p, const float (&v)[1]) { *p = from_f<T>(v[0]); }
};

constexpr int MAX_WARPS = 32;

// Sum of `v` over the blockDim.x threads of a row.  A one-warp row needs no
// barrier; a wider row has its block to itself (blockDim.y = 1), and `slot`
// alternates between uses so that one barrier a sum is enough.
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (blockDim.x == 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  return warp_sum(lane < nw ? red[lane] : 0.f);
}

// One row per blockDim.x threads; a thread holds V pieces of W values, at
// stride blockDim.x * W.
template <typename XT, typename ZT, int W, int V>
__global__ void __launch_bounds__(1024)
norm_fwd_kernel(NormFwd a) {
  __shared__ float red[2][MAX_WARPS];
  pdl_begin();
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.T) return;    // whole warps: a wider row has one row per block
  const int D = a.D, step = blockDim.x * W;
  const long long base = row * D;
  const XT* x = static_cast<const XT*>(a.x) + base;
  float v[V][W];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x * W + i * step;
    if (c < D) {
      Row<XT, W>::load(x + c, v[i]);
      if (a.delta != nullptr) {
        float d[W];
        if (a.delta_type == 0) Row<float, W>::load(static_cast<const float*>(a.delta) + base + c, d);
        else Row<bf16, W>::load(static_cast<const bf16*>(a.delta) + base + c, d);
        // the norm reads the stream as it is stored, so that the backward
        // pass, which reads it from memory, sees the same values
#pragma unroll
        for (int j = 0; j < W; ++j) v[i][j] = to_f(from_f<XT>(v[i][j] + d[j]));
        Row<XT, W>::store(static_cast<XT*>(a.h) + base + c, v[i]);
      }
#pragma unroll
      for (int j = 0; j < W; ++j) s += v[i][j];
    }
  }
  const float inv = 1.0f / (float)D;
  const float mean = row_sum(s, red[0]) * inv;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x * W + i * step;
    if (c < D) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        v[i][j] -= mean;
        s = fmaf(v[i][j], v[i][j], s);
      }
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum(s, red[1]) * inv + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x * W + i * step;
    if (c < D) {
      float g[W], b[W];
      Row<float, W>::load(a.gamma + c, g);
      if (a.beta != nullptr) Row<float, W>::load(a.beta + c, b);
#pragma unroll
      for (int j = 0; j < W; ++j)
        v[i][j] = a.beta != nullptr ? fmaf(v[i][j] * rstd, g[j], b[j]) : v[i][j] * rstd * g[j];
      Row<ZT, W>::store(static_cast<ZT*>(a.z) + base + c, v[i]);
    }
  }
}

// Sums over the blockDim.x threads of a row where a block holds blockDim.y rows:
// a named barrier of the row's own.
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (blockDim.x == 32) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
  const float2 t = lane < (int)(blockDim.x >> 5) ? red[lane] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(t.x), warp_sum(t.y));
}

// 16 (fp32) or 8 (bf16) bytes, four values, into shared memory.
template <typename T>
__device__ __forceinline__ void copy4(uint32_t dst, const T* src) {
  if (sizeof(T) == 4)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// Rows at stride gridDim.x * blockDim.y; a thread keeps the sums of its own
// columns over its rows, and the block writes one partial row of dgamma and of
// dbeta, which norm_cols_kernel adds in a fixed order.  A thread owns V pieces
// of W columns.
//
// W = 4: the next two rows are on their way into shared memory while one is
// summed.  Every thread copies the values that it will read itself, so the copies
// need no barrier, and rows in flight take no registers, which the column sums
// need.  gamma is read again for each row (it stays in L1): held in registers it
// costs spills or the second block of an SM.  65536 x 4096, bf16 stream with a
// residual gradient: 559 us, 6.72 TB/s (the copy rate is 6.79); 631 us with loads
// at the row's turn, 662 us with gamma in registers, 870 us with one block an SM.
// W = 1 (D no multiple of 8) loads at the row's turn: 5003 x 1023 fp32 with a
// residual gradient 37 us, 3 times its bytes' time.  Above D = 8192 a block of
// 1024 threads keeps 16 values a thread and spills: 8192 x 16384 557 us (bf16) and
// 572 us (fp32), 2.0 and 1.8 times their bytes'.
// dres joins before the row's correction, which rounds once more at its size
// (65536 x 4096: 2.8e-7 from the values in 64 bits, an fp32 form that adds it last
// 1.8e-7): kept back it would need eight more registers a thread, or its place in
// shared memory while the next row should be loading.
template <typename XT, int W, int V, int MAXT>
__global__ void __launch_bounds__(MAXT, 1024 / MAXT)
norm_bwd_kernel(NormBwd a, int stages) {
  __shared__ float2 red[2][MAX_WARPS];
  extern __shared__ __align__(16) char ring[];
  pdl_begin();
  const int D = a.D, step = blockDim.x * W;
  const float inv = 1.0f / (float)D;
  float dg[V][W], db[V][W];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) dg[i][j] = db[i][j] = 0.f;
  }
  const long long hop = (long long)gridDim.x * blockDim.y;
  const int row_bytes = D * ((int)sizeof(XT) + 4 + (a.dres != nullptr ? 4 : 0));
  auto slot = [&](int s) { return ring + ((long long)s * blockDim.y + threadIdx.y) * row_bytes; };
  auto put = [&](long long row, int s) {
    if (W == 4 && row < a.T) {
      const long long base = row * D;
      char* to = slot(s);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x * W + i * step;
        if (c < D) {
          const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
          copy4(at + c * 4, a.dz + base + c);
          if (a.dres != nullptr) copy4(at + (D + c) * 4, a.dres + base + c);
          copy4(at + (a.dres != nullptr ? 8 : 4) * D + c * (int)sizeof(XT),
                static_cast<const XT*>(a.h) + base + c);
        }
      }
    }
    if (W == 4) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  float2* mine = red[0] + threadIdx.y * (blockDim.x >> 5);
  int s = 0, phase = 0;
  put(row, 0);
  if (stages == 2) put(row + hop, 1);
  for (; row < a.T; row += hop) {
    const long long base = row * D;
    const float m = a.mean[row], r = a.rstd[row];
    const char* from = slot(s);
    if (W == 4) {
      if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    // dx = (dres + r g) - r (c1 + xh c2): the first part needs no sum over the
    // row, and with it the row's values are all read, so that the row after next
    // takes their place at once
    float xh[V][W], o[V][W];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x * W + i * step;
      if (c < D) {
        float dz[W], e[W], gm[W];
        Row<float, W>::load(a.gamma + c, gm);
        if constexpr (W == 4) {
          Row<float, W>::load(reinterpret_cast<const float*>(from) + c, dz);
          Row<XT, W>::load(reinterpret_cast<const XT*>(from + (a.dres != nullptr ? 8 : 4) * D) + c, xh[i]);
          if (a.dres != nullptr) Row<float, W>::load(reinterpret_cast<const float*>(from) + D + c, e);
        } else {
          Row<float, W>::load(a.dz + base + c, dz);
          Row<XT, W>::load(static_cast<const XT*>(a.h) + base + c, xh[i]);
          if (a.dres != nullptr) Row<float, W>::load(a.dres + base + c, e);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          xh[i][j] = (xh[i][j] - m) * r;
          dg[i][j] = fmaf(dz[j], xh[i][j], dg[i][j]);
          db[i][j] += dz[j];
          const float g = gm[j] * dz[j];
          s1 += g;
          s2 = fmaf(g, xh[i][j], s2);
          o[i][j] = a.dres != nullptr ? fmaf(r, g, e[j]) : r * g;
        }
      }
    }
    put(row + stages * hop, s);
    s = stages == 2 ? s ^ 1 : 0;
    const float2 t = row_sum2(s1, s2, mine + phase * MAX_WARPS);
    phase ^= 1;
    const float c1 = t.x * inv * r, c2 = t.y * inv * r;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x * W + i * step;
      if (c < D) {
#pragma unroll
        for (int j = 0; j < W; ++j) o[i][j] -= fmaf(xh[i][j], c2, c1);
        Row<float, W>::store(a.dx + base + c, o[i]);
      }
    }
  }
  if (W == 4) asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* cols = reinterpret_cast<float*>(ring);      // blockDim.y > 1: [blockDim.y][D] of one sum at a time
  auto emit = [&](const float (&v)[V][W], float* out) {
    if (blockDim.y > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x * W + i * step;
      if (c < D) Row<float, W>::store(blockDim.y > 1 ? cols + threadIdx.y * D + c : out + c, v[i]);
    }
    if (blockDim.y == 1) return;
    __syncthreads();
    for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < D; c += blockDim.x * blockDim.y) {
      float sum = 0.f;
      for (int q = 0; q < (int)blockDim.y; ++q) sum += cols[q * D + c];
      out[c] = sum;
    }
  };
  float* part = a.part + (long long)blockIdx.x * 2 * D;
  emit(dg, part);
  if (a.want_beta) emit(db, part + D);
}

// dgamma and dbeta from the nparts partial rows [nparts][2][D]: 32 columns by
// 32 slices of the partials per block, the slices added in order.
__global__ void __launch_bounds__(1024)
norm_cols_kernel(const float* __restrict__ part, int nparts, int D, float* __restrict__ dgamma,
                 float* __restrict__ dbeta) {
  __shared__ float s[32][33];
  pdl_begin();
  const int c = blockIdx.x * 32 + threadIdx.x, w = blockIdx.y;
  float t = 0.f;
  if (c < D)
    for (int p = threadIdx.y; p < nparts; p += 32) t += part[((long long)p * 2 + w) * D + c];
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  // each warp sums one column over the slices (a fixed tree)
  const float sum = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < D) (w == 0 ? dgamma : dbeta)[col] = sum;
}

// SMs of the part that the library is built for.  A constant, so that the backward
// pass's workspace and the order of its sums do not go with the device.
constexpr int SMS = 152;

// Threads per row and pieces per thread: the fewest threads that hold the row.
struct Shape {
  int W, V, tpr, rows;   // values a piece, pieces a thread, threads a row, rows a block
};
Shape norm_shape(int D, int vmax) {
  Shape s{};
  s.W = D % 8 == 0 ? 8 : 1;
  s.V = s.W == 8 ? vmax : 8;
  const int per = s.W * s.V;
  s.tpr = 32;
  while (s.tpr * per < D && s.tpr < 1024) s.tpr *= 2;
  s.rows = s.tpr == 32 ? 8 : 1;
  return s;
}

}  // namespace

// The backward pass's blocks: 512 threads of as many rows as fit them (1024
// where a row takes that many), two blocks an SM.  More blocks would write more
// partial rows: 4096 x 512 took 15.4 us with 2432 of them.
struct BwdShape {
  int W, V, tpr, rows, blocks;
};
static BwdShape bwd_shape(long long T, int D) {
  BwdShape s{};
  s.W = D % 8 == 0 ? 4 : 1;
  s.V = s.W == 1 ? 8 : D <= 8192 ? 2 : 4;
  s.tpr = 32;
  while (s.tpr * s.W * s.V < D && s.tpr < 1024) s.tpr *= 2;
  s.rows = s.tpr < 512 ? 512 / s.tpr : 1;
  const long long need = (T + s.rows - 1) / s.rows, most = (long long)SMS * (s.tpr > 512 ? 1 : 2);
  s.blocks = (int)(need < most ? need : most);
  return s;
}
int norm_bwd_blocks(long long T, int D) { return bwd_shape(T, D).blocks; }

template <typename XT, typename ZT>
static cudaError_t fwd_t(const NormFwd& a, cudaStream_t st) {
  // few rows (less than two an SM): one piece a thread, for the shortest chain;
  // many: two, for fewer threads a row.  One against two pieces, us, bf16: 1 row of
  // 1024 2.1 / 2.5, of 4096 2.6 / 2.8, of 8192 3.3 / 3.4 (of 256 1.95 / 1.8); 4864
  // rows of 4096 34.4 / 31.8, of 8192 72.0 / 70.2 (of 1024 9.9 / 10.2)
  const Shape s = norm_shape(a.D, a.T < 2 * SMS && a.D <= 8192 ? 1 : 2);
  const dim3 grid((unsigned)((a.T + s.rows - 1) / s.rows)), block(s.tpr, s.rows);
  if (s.W == 1) return launch_pdl(norm_fwd_kernel<XT, ZT, 1, 8>, grid, block, 0, st, a);
  if (s.V == 1) return launch_pdl(norm_fwd_kernel<XT, ZT, 8, 1>, grid, block, 0, st, a);
  return launch_pdl(norm_fwd_kernel<XT, ZT, 8, 2>, grid, block, 0, st, a);
}

cudaError_t launch_norm_fwd(int x_type, int z_type, const NormFwd& a, cudaStream_t st) {
  if (x_type == 0) return z_type == 0 ? fwd_t<float, float>(a, st) : fwd_t<float, bf16>(a, st);
  return z_type == 0 ? fwd_t<bf16, float>(a, st) : fwd_t<bf16, bf16>(a, st);
}

template <typename XT, int W, int V, int MAXT>
static cudaError_t bwd_k(const NormBwd& a, const BwdShape& s, cudaStream_t st) {
  static std::atomic<unsigned long long> attr_done{0};
  constexpr int kMost = 220 * 1024;
  cudaError_t e = ensure_dynamic_smem(norm_bwd_kernel<XT, W, V, MAXT>, kMost, attr_done);
  if (e != cudaSuccess) return e;
  // two stages of the block's rows where they fit (with two blocks an SM up to D = 4096)
  const int stage = W == 4 ? s.rows * a.D * ((int)sizeof(XT) + 4 + (a.dres != nullptr ? 4 : 0)) : 0;
  const int stages = 2 * stage <= kMost ? 2 : 1;
  int smem = stages * stage;
  if (s.rows > 1 && smem < s.rows * a.D * 4) smem = s.rows * a.D * 4;
  return launch_pdl(norm_bwd_kernel<XT, W, V, MAXT>, dim3(s.blocks), dim3(s.tpr, s.rows),
                    (size_t)smem, st, a, stages);
}
template <typename XT>
static cudaError_t bwd_t(const NormBwd& a, cudaStream_t st) {
  const BwdShape s = bwd_shape(a.T, a.D);
  if (s.W == 1) return s.tpr > 512 ? bwd_k<XT, 1, 8, 1024>(a, s, st) : bwd_k<XT, 1, 8, 512>(a, s, st);
  if (s.V == 4) return bwd_k<XT, 4, 4, 1024>(a, s, st);
  return s.tpr > 512 ? bwd_k<XT, 4, 2, 1024>(a, s, st) : bwd_k<XT, 4, 2, 512>(a, s, st);
}

cudaError_t launch_norm_bwd(int x_type, const NormBwd& a, cudaStream_t st) {
  return x_type == 0 ? bwd_t<float>(a, st) : bwd_t<bf16>(a, st);
}

cudaError_t launch_norm_cols(const float* part, int nparts, int D, float* dgamma, float* dbeta,
                             cudaStream_t st) {
  return launch_pdl(norm_cols_kernel, dim3((D + 31) / 32, dbeta != nullptr ? 2 : 1), dim3(32, 32),
                    0, st, part, nparts, D, dgamma, dbeta);
}

}  // namespace moe
