// The matrix product grouped by expert with 4-bit weights, for many rows: on the
// tcgen05 tensor cores, the weights widened to bf16 on the way.
//
//   c[r, f] = act(sum_k w_e[f, k] x[r, k] + bias_e[f])     rows r of expert e
//
// A tile is 128 outputs by up to BN rows of one expert (64 outputs of W and the same
// of W3 for SwiGLU): the outputs are the lanes of the accumulator, the rows its
// columns, so that a tile of few rows wastes no more than the narrow side of the
// instruction (its N is the rows rounded up to 16) and one of many rows reads the
// weights, which have to be widened, once for up to 256 rows.
//
// One persistent block an SM, its warps specialised:
//   warp 0       codes and scales by bulk-tensor copies, 128 inputs at a time;
//   warp 1       the matrix instructions (and the tensor memory);
//   warps 2..5   the epilogue: a lane an output, column by column;
//   warp 6       the rows of x by bulk-tensor copies, 64 inputs at a time;
//   warps 7..14  4-bit to bf16: a thread 32 inputs of an output, written in the
//                128-byte swizzle that the instructions read.
// Two accumulators let a tile's epilogue run beside the next one's products.
// Every wait is bounded (2 s); when one expires the block raises an abort flag and
// the status word, waits for its copies and products in flight, frees its tensor
// memory and returns.
#include "q4.cuh"
#include "q4.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int BM = 128, BK = 64, UK = 16, RAW_K = 128;
constexpr int A_BYTES = BM * BK * 2;                     // 16 KB
constexpr int CODE_BYTES = BM * RAW_K / 2;               // 8 KB
constexpr int RAW_BYTES = CODE_BYTES + BM * (RAW_K / 32) * 2;   // + the scales, up to 1 KB
constexpr int X_BOX = 64;                                // rows of a copy of x
constexpr int W_RAW = 0, W_MMA = 1, W_EPI = 2, W_X = 6, W_WIDEN = 7, N_WIDEN = 8;
constexpr int THREADS = 32 * (W_WIDEN + N_WIDEN);
constexpr int MAX_E = 256;
constexpr int TMEM_COLS = 512;
constexpr long long LIMIT_NS = 2000000000ll;

// Operand stages (64 inputs) and raw stages (128 inputs) by the rows of a tile.
template <int BN> struct Ring;
template <> struct Ring<256> { static constexpr int S = 4, Q = 3; };
template <> struct Ring<128> { static constexpr int S = 4, Q = 10; };
template <> struct Ring<64> { static constexpr int S = 5, Q = 10; };
template <int BN> constexpr int kStage = A_BYTES + BN * BK * 2;
template <int BN> constexpr int kSmem = Ring<BN>::S * kStage<BN> + Ring<BN>::Q * RAW_BYTES;
static_assert(kSmem<256> + 4096 <= 232448 && kSmem<128> + 4096 <= 232448 && kSmem<64> + 4096 <= 232448,
              "shared memory of one block");

struct Params {
  int R, E, N, K, log_g;
  int act;
  int nF, per;                 // tiles along the outputs, outputs of a tile
  const int* offsets;
  const float* bias;
  bf16* c;
  int* status;
};

// Row tiles of the experts: first tile and rows of a tile by expert.
struct Table {
  int offs[MAX_E + 1], first[MAX_E + 1], step[MAX_E];
  int scan[2][16];
};
struct Tile {
  int e, r0, n, f0;
};
__device__ __forceinline__ Tile tile_at(int t, const Params& p, const Table& tb) {
  const int rt = t / p.nF;
  int lo = 0, hi = p.E;        // the largest lo with first[lo] <= rt
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tb.first[mid] <= rt) lo = mid; else hi = mid;
  }
  Tile T;
  T.e = lo;
  T.r0 = tb.offs[lo] + (rt - tb.first[lo]) * tb.step[lo];
  T.n = min(tb.step[lo], tb.offs[lo + 1] - T.r0);
  T.f0 = (t - rt * p.nF) * p.per;
  return T;
}

// Inclusive scan over the block's first MAX_E + 1 threads (others pass the neutral
// element): the running maximum or the running sum.
template <bool MAX>
__device__ __forceinline__ int block_scan(int v, int* part) {
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

// Offsets clamped to a sequence that does not decrease within [0, R], and the row tiles:
// an expert's rows in tiles of equal size, a multiple of 16, so that none is much
// smaller than the others.
template <int BN>
__device__ __forceinline__ void make_table(const Params& p, Table& tb) {
  const int e = threadIdx.x;
  int v = 0;
  if (e <= p.E) v = p.offsets ? min(max(p.offsets[e], 0), p.R) : e * p.R;
  v = block_scan<true>(v, tb.scan[0]);
  if (e <= p.E) tb.offs[e] = v;
  __syncthreads();
  int tiles = 0;
  if (e < p.E) {
    const int rows = tb.offs[e + 1] - v;
    const int least = (rows + BN - 1) / BN;
    const int step = rows ? ((rows + least - 1) / least + 15) & ~15 : 16;
    tiles = (rows + step - 1) / step;
    tb.step[e] = step;
  }
  const int incl = block_scan<false>(tiles, tb.scan[1]);
  if (e < p.E) tb.first[e + 1] = incl;
  if (e == 0) tb.first[0] = 0;
  __syncthreads();
}

__device__ __forceinline__ float act_of(int act, float h) {
  if (act == 1) return gelu_epi(h);
  return act == 0 && h < 0.f ? 0.f : h;          // a NaN stays one
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint32_t lds_scale(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v | (uint32_t)v << 16;
}

template <int BN, bool SWIGLU>
__global__ void __launch_bounds__(THREADS, 1)
q4_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ CUtensorMap tm_s, const __grid_constant__ CUtensorMap tm_w3,
               const __grid_constant__ CUtensorMap tm_s3, const Params p) {
  constexpr int S = Ring<BN>::S, Q = Ring<BN>::Q, STAGE = kStage<BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t raw_full[Q], raw_empty[Q], x_full[S], a_full[S], empty[S];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], drain_mb;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ Table tb;
  volatile int* abort_flag = &abort_word;
  const uint32_t sbase = smem_u32(smem), rbase = sbase + S * STAGE;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < Q; ++i) {
      mbar_init(smem_u32(&raw_full[i]), 1);
      mbar_init(smem_u32(&raw_empty[i]), N_WIDEN);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&x_full[i]), 1);
      mbar_init(smem_u32(&a_full[i]), N_WIDEN);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), 4);
    }
    mbar_init(smem_u32(&drain_mb), 1);
    abort_word = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == W_MMA) tmem_alloc(smem_u32(&tmem_slot), TMEM_COLS);
  pdl_wait();                  // offsets and x may be the previous kernel's
  tc_fence_before();
  make_table<BN>(p, tb);       // (with barriers of the block)
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int total = tb.first[p.E] * p.nF;
  const int nraw = (p.K + RAW_K - 1) / RAW_K, nkb = (p.K + BK - 1) / BK;
  auto wait = [&](uint64_t& mb, uint32_t parity) {
    return wait_bar(smem_u32(&mb), parity, abort_flag, p.status, LIMIT_NS);
  };

  if (warp == W_RAW) {
    if (lane == 0) {
      int q = 0, issued = 0;
      uint32_t ph = 0, last = 0;
      bool ok = true;
      const int ng = RAW_K >> p.log_g;
      for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
        const Tile T = tile_at(t, p, tb);
        for (int j = 0; j < nraw; ++j) {
          if (!wait(raw_empty[q], ph ^ 1u)) { ok = false; break; }
          const uint32_t bar = smem_u32(&raw_full[q]), to = rbase + q * RAW_BYTES, ss = to + CODE_BYTES;
          mbar_arrive_expect_tx(bar, CODE_BYTES + ng * BM * 2);
          if (SWIGLU) {
            tma_load_3d(to, &tm_w, bar, j * (RAW_K / 2), T.f0, T.e);
            tma_load_3d(to + CODE_BYTES / 2, &tm_w3, bar, j * (RAW_K / 2), T.f0, T.e);
            tma_load_3d(ss, &tm_s, bar, T.f0, j * ng, T.e);
            tma_load_3d(ss + ng * BM, &tm_s3, bar, T.f0, j * ng, T.e);
          } else {
            tma_load_3d(to, &tm_w, bar, j * (RAW_K / 2), T.f0, T.e);
            tma_load_3d(ss, &tm_s, bar, T.f0, j * ng, T.e);
          }
          issued |= 1 << q;
          last = (last & ~(1u << q)) | (ph << q);
          if (++q == Q) { q = 0; ph ^= 1u; }
        }
      }
      // every copy has landed before the block goes
      for (int i = 0; i < Q; ++i)
        if (issued >> i & 1) drain_wait(smem_u32(&raw_full[i]), last >> i & 1u, LIMIT_NS);
    }
    __syncwarp();
  } else if (warp == W_X) {
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t ph = 0, last = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
        const Tile T = tile_at(t, p, tb);
        const int boxes = (T.n + X_BOX - 1) / X_BOX;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!wait(empty[s], ph ^ 1u)) { ok = false; break; }
          const uint32_t bar = smem_u32(&x_full[s]), to = sbase + s * STAGE + A_BYTES;
          mbar_arrive_expect_tx(bar, boxes * (X_BOX * BK * 2));
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(to + b * (X_BOX * BK * 2), &tm_x, bar, kb * BK, T.r0 + b * X_BOX);
          issued |= 1 << s;
          last = (last & ~(1u << s)) | (ph << s);
          if (++s == S) { s = 0; ph ^= 1u; }
        }
      }
      for (int i = 0; i < S; ++i)
        if (issued >> i & 1) drain_wait(smem_u32(&x_full[i]), last >> i & 1u, LIMIT_NS);
    }
    __syncwarp();
  } else if (warp == W_MMA) {
    int s = 0, buf = 0;
    uint32_t ph = 0, aph = 0;
    bool ok = true, any = false;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile T = tile_at(t, p, tb);
      if (!__all_sync(0xffffffffu, wait(acc_empty[buf], aph ^ 1u))) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(buf * 256);
      // fp32 accumulator, bf16 operands, both along K; N the rows in steps of 16
      const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)((T.n + 15) / 16 * 2) << 17 |
                             (uint32_t)(BM >> 4) << 24;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!__all_sync(0xffffffffu, wait(x_full[s], ph) && wait(a_full[s], ph))) { ok = false; break; }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t a = sbase + s * STAGE, b = a + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / UK; ++kk)
            mma_bf16(d, smem_desc(a + kk * 32, 16, 1024), smem_desc(b + kk * 32, 16, 1024), idesc,
                     (kb > 0 || kk > 0) ? 1u : 0u);
          mma_commit(smem_u32(&empty[s]));
        }
        any = true;
        __syncwarp();
        if (++s == S) { s = 0; ph ^= 1u; }
      }
      if (!ok) break;
      if (lane == 0) mma_commit(smem_u32(&acc_full[buf]));
      __syncwarp();
      if (++buf == 2) { buf = 0; aph ^= 1u; }
    }
    if (any && lane == 0) {
      mma_commit(smem_u32(&drain_mb));
      drain_wait(smem_u32(&drain_mb), 0, LIMIT_NS);
    }
    __syncwarp();
  } else if (warp >= W_WIDEN) {
    const int w = tid - 32 * W_WIDEN, r = w & 127, half = w >> 7;
    // SwiGLU: 16 outputs of W and the same 16 of W3 share a warp's lanes
    const int row = SWIGLU ? (r >> 4 & 3) * 32 + (r >> 6) * 16 + (r & 15) : r;
    const uint32_t code_at = r * 64, swz = (r >> 1) & 3;
    const int ng = RAW_K >> p.log_g;
    const uint32_t scale_at = CODE_BYTES + (SWIGLU ? (r >> 6) * ng * BM + (r & 63) * 2 : r * 2);
    const uint32_t scale_step = SWIGLU ? BM : BM * 2;
    const uint32_t a_at = row * 128;
    int q = 0, s = 0;
    uint32_t qph = 0, ph = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      for (int j = 0; ok && j < nraw; ++j) {
        if (!__all_sync(0xffffffffu, wait(raw_full[q], qph))) { ok = false; break; }
        const uint32_t raw = rbase + q * RAW_BYTES;
        uint4 code[2];
        uint32_t scale[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          code[h] = lds128(raw + code_at + ((2 * h + half) ^ swz) * 16);
          scale[h] = lds_scale(raw + scale_at + ((h * 64 + half * 32) >> p.log_g) * scale_step);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&raw_empty[q]));
        if (++q == Q) { q = 0; qph ^= 1u; }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k0 = j * RAW_K + h * BK;
          if (k0 >= p.K) break;
          if (!__all_sync(0xffffffffu, wait(empty[s], ph ^ 1u))) { ok = false; break; }
          const uint32_t to = sbase + s * STAGE + a_at;
          // past the last input: zeros, whatever the scale
          const bool on = k0 + half * 32 < p.K;
          const uint32_t c4[4] = {code[h].x, code[h].y, code[h].z, code[h].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts128(to + (((half * 4 + i) ^ (row & 7)) << 4),
                   on ? q4_word(c4[i], scale[h]) : make_uint4(0u, 0u, 0u, 0u));
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&a_full[s]));
          if (++s == S) { s = 0; ph ^= 1u; }
        }
      }
    }
  } else {
    const int quarter = warp & 3;            // of the accumulator's lanes that this warp may read
    int buf = 0;
    uint32_t aph = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      const Tile T = tile_at(t, p, tb);
      if (!__all_sync(0xffffffffu, wait(acc_full[buf], aph))) break;
      tc_fence_after();
      const uint32_t at = tmem + (uint32_t)(buf * 256) + ((uint32_t)(quarter * 32) << 16);
      const int f = T.f0 + (SWIGLU ? quarter * 16 + (lane & 15) : quarter * 32 + lane);
      const bool on = f < p.N;
      const float bias = !SWIGLU && p.bias != nullptr && on ? p.bias[(long long)T.e * p.N + f] : 0.f;
      bf16* c = p.c + (long long)T.r0 * p.N + f;
      for (int col = 0; col < T.n; col += 16) {
        float v[16];
        tmem_ld16(at + col, v);
        tmem_ld_wait();
        if (SWIGLU) {
          // lanes 0..15 have W's outputs, 16..31 W3's: of two columns each half takes one
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const bool up = lane >= 16;
            const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 1], 16);
            const float h1 = up ? got : v[i], h3 = up ? v[i + 1] : got;
            const int n = col + i + (up ? 1 : 0);
            if (on && n < T.n)
              c[(long long)n * p.N] = __float2bfloat16_rn((h1 * sigmoid_epi(h1)) * h3);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (on && col + i < T.n)
              c[(long long)(col + i) * p.N] = __float2bfloat16_rn(act_of(p.act, v[i] + bias));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[buf]));
      if (++buf == 2) { buf = 0; aph ^= 1u; }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* ptr,
            int rank, const uint64_t* dims, const uint64_t* strides, const uint32_t* box) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t estr[3] = {1, 1, 1};
  cuuint64_t d[3], s[2];
  cuuint32_t b[3];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
  }
  for (int i = 0; i < rank - 1; ++i) s[i] = strides[i];
  return fn(m, type, (cuuint32_t)rank, const_cast<void*>(ptr), d, s, b, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool SWIGLU>
cudaError_t launch_t(const CUtensorMap* maps, const Params& p, long long tiles, cudaStream_t st) {
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = ensure_dynamic_smem(q4_gemm_kernel<BN, SWIGLU>, kSmem<BN>, attr_done);
  if (e != cudaSuccess) return e;
  const int sms = sm_count(), grid = tiles < sms ? (int)tiles : sms;
  return launch_pdl(q4_gemm_kernel<BN, SWIGLU>, dim3(grid), dim3(THREADS), kSmem<BN>, st, maps[0], maps[1],
                    maps[2], maps[3], maps[4], p);
}

template <bool SWIGLU>
cudaError_t launch_bn(int bn, const CUtensorMap* maps, const Params& p, long long tiles, cudaStream_t st) {
  if (bn == 64) return launch_t<64, SWIGLU>(maps, p, tiles, st);
  if (bn == 128) return launch_t<128, SWIGLU>(maps, p, tiles, st);
  return launch_t<256, SWIGLU>(maps, p, tiles, st);
}

}  // namespace

cudaError_t launch_q4_gemm(const Q4Product& q, cudaStream_t st) {
  const bool swiglu = q.act == 2;
  Params p{};
  p.R = q.R; p.E = q.E; p.N = q.N; p.K = q.K;
  p.log_g = q.G == 32 ? 5 : q.G == 64 ? 6 : 7;
  p.act = q.act;
  p.per = swiglu ? BM / 2 : BM;
  p.nF = (q.N + p.per - 1) / p.per;
  p.offsets = q.offsets;
  p.bias = q.bias;
  p.c = static_cast<bf16*>(q.c);
  p.status = q.status;
  CUtensorMap maps[5];
  const uint64_t xd[2] = {(uint64_t)q.K, (uint64_t)q.R}, xs[1] = {(uint64_t)q.K * 2};
  const uint32_t xb[2] = {BK, X_BOX};
  bool ok = encode(&maps[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, q.x, 2, xd, xs, xb);
  const uint64_t groups = (uint64_t)q4_groups(q.K, q.G);
  const uint64_t wd[3] = {(uint64_t)q.K / 2, (uint64_t)q.N, (uint64_t)q.E};
  const uint64_t ws[2] = {(uint64_t)q.K / 2, (uint64_t)q.N * (uint64_t)q.K / 2};
  const uint32_t wb[3] = {RAW_K / 2, (uint32_t)p.per, 1};
  const uint64_t sd[3] = {(uint64_t)q.N, groups, (uint64_t)q.E};
  const uint64_t ss[2] = {(uint64_t)q.N * 2, (uint64_t)q.N * groups * 2};
  const uint32_t sb[3] = {(uint32_t)p.per, (uint32_t)(RAW_K / q.G), 1};
  for (int i = 0; i < 2 && ok; ++i) {
    if (i == 1 && !swiglu) {
      maps[3] = maps[1];
      maps[4] = maps[2];
      break;
    }
    ok = encode(&maps[1 + 2 * i], CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_64B,
                i ? q.codes3 : q.codes, 3, wd, ws, wb) &&
         encode(&maps[2 + 2 * i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_NONE,
                i ? q.scales3 : q.scales, 3, sd, ss, sb);
  }
  if (!ok) return cudaErrorInvalidValue;
  const long long mean = q.R / q.E;
  const int bn = mean > 96 ? 256 : mean > 48 ? 128 : 64;
  const long long tiles = ((long long)q.R / 16 + q.E) * p.nF;      // at most
  return swiglu ? launch_bn<true>(bn, maps, p, tiles, st) : launch_bn<false>(bn, maps, p, tiles, st);
}

}  // namespace moe
