// The matrix product grouped by expert with 4-bit weights, for many rows: on the
// tcgen05 tensor cores, the weights widened to bf16 on the way.
//
//   c[r, f] = act(sum_k w_e[f, k] x[r, k] + bias_e[f])     rows r of expert e
//
// A tile is 128 outputs by up to 160 rows of one expert (64 outputs of W and the same of
// W3 for SwiGLU): the outputs are the lanes of the accumulator, the rows its columns,
// so that a tile of few rows wastes no more than the narrow side of the instruction (its
// N is the rows rounded up to 16).  The widened weights are the A operand, which lies in
// tensor memory beside the two accumulators: a lane is an output, and a thread writes 64
// of its inputs with one instruction.
//
// One persistent block an SM, its warps specialised:
//   warp 0       codes and scales by bulk-tensor copies, 128 inputs at a time;
//   warp 1       the matrix instructions (and the tensor memory);
//   warps 2..5   the epilogue: a lane an output, column by column;
//   warp 6       the rows of x by bulk-tensor copies, 128 inputs at a time;
//   warps 7..    4-bit to bf16, in groups of four warps that take 128 inputs in turn.
// Two accumulators let a tile's epilogue run beside the next one's products.
// Every wait is bounded (2 s); when one expires the block raises an abort flag and
// the status word, waits for its copies and products in flight, frees its tensor
// memory and returns.
//
// What bounds it: the matrix instructions (their pipe is 74 to 77 % busy at 160-row tiles,
// the rest being a tile's beginning and end and waits for the widening warps), and with few
// rows an expert the chain of a stage: widening, the issue of its products (some 27 clocks
// each) and the wait for their end.  Measured in bursts of a few calls, 128 experts, 4096
// inputs, 2 x 2048 outputs with SwiGLU: 160 rows an expert 0.39 ms, 1.75 PFLOP/s; 256 rows 0.67
// ms, 1.65; 32768 rows dealt as a router does 0.68 ms (0.77 to 0.82 call after call, under the
// power limit); 16 rows an expert 258 us, 4.4 TB/s of codes, scales and rows.  Without SwiGLU,
// 2048 inputs and 4096 outputs, 256 rows an expert: 0.36 ms, 1.54 PFLOP/s.  One matrix of 4096 x
// 4096 and 65536 rows: 1.12 ms, 1.97 PFLOP/s.
//
// Left behind (the 32768 rows dealt unevenly): widened weights in shared memory as the A
// operand, which take its rate from the rows, 1.19 ms; then 64 inputs a stage and one store
// an output and row in the epilogue, 0.86.  Three stages of rows in place of four: 256 rows
// an expert 0.79 ms, whatever the stages of codes.  Prefetches of the rows into L2 by the
// warp that copies them 0.73 (its own instructions count).  Tiles of 192 rows leave tensor
// memory for two stages of widened weights only; without them 161 to 192 rows of an expert are
// two tiles of 96 (192 rows an expert: 0.60 ms where 160 rows take 0.39).  A look ahead at the
// next stage's barriers that may suspend the warp: 4 us more for a small call.
#include "q4.cuh"
#include "q4.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int BM = 128, BK = 64, UK = 16, RAW_K = 128;
constexpr int CODE_BYTES = BM * RAW_K / 2;               // 8 KB
constexpr int RAW_BYTES = CODE_BYTES + BM * (RAW_K / 32) * 2;   // + the scales, up to 1 KB
// Heights of a copy of x: the least that has a tile's rows.
constexpr int X_BOXES = 7;
__host__ __device__ constexpr int box_rows(int i) { return i < 4 ? 16 * (i + 1) : 32 * (i - 1); }
__host__ __device__ constexpr int box_of(int rows) { return rows <= 64 ? (rows - 1) / 16 : (rows - 1) / 32 + 2; }
static_assert(box_rows(0) == 16 && box_rows(3) == 64 && box_rows(4) == 96 && box_rows(6) == 160, "heights");
static_assert(box_of(1) == 0 && box_of(64) == 3 && box_of(65) == 4 && box_of(96) == 4 && box_of(97) == 5 &&
              box_of(160) == 6, "heights");
constexpr int W_RAW = 0, W_MMA = 1, W_EPI = 2, W_X = 6, W_WIDEN = 7;
constexpr int MAX_E = 256;
constexpr int TMEM_COLS = 512;
constexpr long long LIMIT_NS = 2000000000ll;             // bound of every wait

// Rows of a tile at most, and stages, each of 128 inputs: Q of codes and scales, SA of
// widened weights, SX of rows.  The accumulators take 2 BN of the 512 columns, a stage of
// weights 64.  The groups of widening warps run apart from one another, and copies do
// not land in the order of their issue: of copies a group may only wait on stages whose
// every use is its own (a barrier tells no more than the parity of its phase), so Q is a
// multiple of the groups.  SA is their number, a stage of widened weights each.  The
// products of a stage, whose end frees both its weights and its rows, end in order and are
// told by one barrier (a second one for the weights: 1 to 3 % slower calls): a group waits
// for those of its last stage, and the next ones of that barrier need this group's weights
// first.  Of a tile's last stage, where it has 64 inputs or less, the second half is without
// work.
constexpr int BN = 160, Q = 6, SA = 3, SX = 4;
static_assert(box_of(BN) == X_BOXES - 1 && box_rows(X_BOXES - 1) == BN, "heights");
constexpr int NG = 3, N_WIDEN = 4 * NG, THREADS = 32 * (W_WIDEN + N_WIDEN);
constexpr int X_HALF = BN * BK * 2, X_STAGE = 2 * X_HALF;
constexpr int SMEM = SX * X_STAGE + Q * RAW_BYTES;
static_assert(2 * BN + SA * 64 <= TMEM_COLS && SA == NG && Q % NG == 0 && NG <= SX, "stages");
static_assert(SMEM + 5120 <= 232448, "shared memory of one block");

struct Params {
  int R, E, N, K, log_g;
  int act;
  int nF, per;                 // tiles along the outputs, outputs of a tile
  const int* offsets;
  const float* bias;
  bf16* c;
  int* status;
  long long limit_ns;          // bound of every wait
  int stall;                   // self-test: no copy is issued, the waits run out
};

struct XMaps {
  CUtensorMap box[X_BOXES];
};

// Row tiles of the experts: first tile and rows of a tile by expert.
struct Table {
  int offs[MAX_E + 1], first[MAX_E + 1], step[MAX_E];
  int scan[2][32];
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

// Offsets clamped to a sequence that does not decrease within [0, R], and the row tiles:
// an expert's rows in tiles of equal size, a multiple of 16, so that none is much
// smaller than the others.
__device__ __forceinline__ void make_table(const Params& p, Table& tb) {
  const int e = threadIdx.x;
  const int v = clamped_offset(p.offsets, p.E, p.R, tb.scan[0]);
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
  const int incl = q4_block_scan<false>(tiles, tb.scan[1]);
  if (e < p.E) tb.first[e + 1] = incl;
  if (e == 0) tb.first[0] = 0;
  __syncthreads();
}

// A bounded wait, false once the block has aborted or the limit has passed (which aborts
// the block and records a timeout).  What follows the first look is out of line: the
// loops of the warps are bound by their instructions' latencies.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                       int* status, long long limit_ns) {
  unsigned long long t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    const unsigned long long now = global_ns();
    if (t0 == 0) t0 = now;
    if ((long long)(now - t0) > limit_ns) {
      *abort_flag = 1;
      if (status) atomicExch(status, DEV_STATUS_TIMEOUT);
      return false;
    }
  }
}
// A look at a barrier that returns at once (a try may take its time).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The one lane of a warp that issues.
__device__ __forceinline__ bool elect() {
  uint32_t v;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(v));
  return v != 0;
}

__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
// 32 columns of tensor memory, a lane's own.
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint4 (&v)[2][4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(at), "r"(v[0][0].x), "r"(v[0][0].y), "r"(v[0][0].z), "r"(v[0][0].w), "r"(v[0][1].x),
      "r"(v[0][1].y), "r"(v[0][1].z), "r"(v[0][1].w), "r"(v[0][2].x), "r"(v[0][2].y), "r"(v[0][2].z),
      "r"(v[0][2].w), "r"(v[0][3].x), "r"(v[0][3].y), "r"(v[0][3].z), "r"(v[0][3].w), "r"(v[1][0].x),
      "r"(v[1][0].y), "r"(v[1][0].z), "r"(v[1][0].w), "r"(v[1][1].x), "r"(v[1][1].y), "r"(v[1][1].z),
      "r"(v[1][1].w), "r"(v[1][2].x), "r"(v[1][2].y), "r"(v[1][2].z), "r"(v[1][2].w), "r"(v[1][3].x),
      "r"(v[1][3].y), "r"(v[1][3].z), "r"(v[1][3].w)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// D += A B^T with A in tensor memory.
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ uint32_t lds_scale(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}

template <bool SWIGLU>
__global__ void __launch_bounds__(THREADS, 1)
q4_gemm_kernel(const __grid_constant__ XMaps tm_x, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ CUtensorMap tm_s, const __grid_constant__ CUtensorMap tm_w3,
               const __grid_constant__ CUtensorMap tm_s3, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t raw_full[Q], raw_empty[Q], a_full[SA];
  __shared__ __align__(8) uint64_t x_full[SX], done[SX];
  __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], drain_mb;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ Table tb;
  volatile int* abort_flag = &abort_word;
  const uint32_t sbase = smem_u32(smem), rbase = sbase + SX * X_STAGE;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < Q; ++i) {
      mbar_init(smem_u32(&raw_full[i]), 1);
      mbar_init(smem_u32(&raw_empty[i]), 4);      // (a group's warps)
    }
    for (int i = 0; i < SA; ++i) mbar_init(smem_u32(&a_full[i]), 4);
    for (int i = 0; i < SX; ++i) {
      mbar_init(smem_u32(&x_full[i]), 1);
      mbar_init(smem_u32(&done[i]), 1);
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
  make_table(p, tb);       // (with barriers of the block)
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int total = tb.first[p.E] * p.nF;
  const int nraw = (p.K + RAW_K - 1) / RAW_K, nkb = (p.K + BK - 1) / BK;   // 2 nraw or one less
  auto all_wait = [&](uint32_t bar, uint32_t parity) {     // by a whole warp; bar: its shared address
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
           __all_sync(0xffffffffu, wait_long(bar, parity, abort_flag, p.status, p.limit_ns));
  };

  // The loops below are run by whole warps and only the copies and products by one lane,
  // so that what is the same for all lanes stays in the uniform registers that those
  // instructions take.
  if (warp == W_RAW) {
    const bool issuer = elect();
    const int ng = RAW_K >> p.log_g;
    const uint32_t bytes = CODE_BYTES + ng * BM * 2;
    int q = 0, issued = 0;
    uint32_t ph = 0, last = 0;
    bool ok = p.stall == 0;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile T = tile_at(t, p, tb);
      for (int j = 0; j < nraw; ++j) {
        if (!all_wait(smem_u32(&raw_empty[q]), ph ^ 1u)) { ok = false; break; }
        if (issuer) {
          const uint32_t bar = smem_u32(&raw_full[q]), to = rbase + q * RAW_BYTES, ss = to + CODE_BYTES;
          mbar_arrive_expect_tx(bar, bytes);
          tma_load_3d(to, &tm_w, bar, j * (RAW_K / 2), T.f0, T.e);
          tma_load_3d(ss, &tm_s, bar, T.f0, j * ng, T.e);
          if (SWIGLU) {
            tma_load_3d(to + CODE_BYTES / 2, &tm_w3, bar, j * (RAW_K / 2), T.f0, T.e);
            tma_load_3d(ss + ng * BM, &tm_s3, bar, T.f0, j * ng, T.e);
          }
        }
        issued |= 1 << q;
        last = (last & ~(1u << q)) | (ph << q);
        if (++q == Q) { q = 0; ph ^= 1u; }
      }
    }
    // every copy has landed before the block goes
    for (int i = 0; i < Q; ++i)
      if (issued >> i & 1) drain_wait(smem_u32(&raw_full[i]), last >> i & 1u, p.limit_ns);
    __syncwarp();
  } else if (warp == W_X) {
    const bool issuer = elect();
    int s = 0, issued = 0;
    uint32_t ph = 0, last = 0;
    bool ok = p.stall == 0;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile T = tile_at(t, p, tb);
      const int box = box_of(T.n);
      const uint32_t bytes = box_rows(box) * (BK * 2);
      const CUtensorMap* map = &tm_x.box[box];
      for (int j = 0; j < nraw; ++j) {
        if (!all_wait(smem_u32(&done[s]), ph ^ 1u)) { ok = false; break; }
        if (issuer) {
          const uint32_t bar = smem_u32(&x_full[s]), to = sbase + s * X_STAGE;
          const bool two = 2 * j + 1 < nkb;              // 64 inputs each
          mbar_arrive_expect_tx(bar, two ? 2 * bytes : bytes);
          tma_load_2d(to, map, bar, j * RAW_K, T.r0);
          if (two) tma_load_2d(to + X_HALF, map, bar, j * RAW_K + BK, T.r0);
        }
        issued |= 1 << s;
        last = (last & ~(1u << s)) | (ph << s);
        if (++s == SX) { s = 0; ph ^= 1u; }
      }
    }
    for (int i = 0; i < SX; ++i)
      if (issued >> i & 1) drain_wait(smem_u32(&x_full[i]), last >> i & 1u, p.limit_ns);
    __syncwarp();
  } else if (warp == W_MMA) {
    const bool issuer = elect();
    // a descriptor's upper word (128-byte swizzle, 1024 bytes from eight rows to the
    // next) and the lower one of the first stage
    constexpr uint32_t hi = 1024u >> 4 | 1u << 14 | 2u << 29;
    const uint32_t b0 = sbase >> 4 | 1u << 16, a0 = tmem + 2 * BN;
    int sa = 0, sx = 0, buf = 0;
    uint32_t pa = 0, px = 0, aph = 0;
    bool ok = true, any = false;
    // (the next stage's barriers are looked at while this one's products are on their way)
    bool x_in = false, a_in = false;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile T = tile_at(t, p, tb);
      if (!all_wait(smem_u32(&acc_empty[buf]), aph ^ 1u)) break;
      const uint32_t d = tmem + (uint32_t)(buf * BN);
      // fp32 accumulator, bf16 operands, both along K; N the rows in steps of 16
      const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)((T.n + 15) / 16 * 2) << 17 |
                             (uint32_t)(BM >> 4) << 24;
      for (int j = 0; j < nraw; ++j) {
        if (!__all_sync(0xffffffffu, x_in && a_in) &&
            !(all_wait(smem_u32(&x_full[sx]), px) && all_wait(smem_u32(&a_full[sa]), pa))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = a0 + sa * 64, b = b0 + sx * (X_STAGE >> 4);
        if (issuer) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (2 * j + k < nkb)
#pragma unroll
              for (int kk = 0; kk < BK / UK; ++kk)
                mma_ta(d, a + k * 32 + kk * 8, (uint64_t)hi << 32 | (b + k * (X_HALF >> 4) + kk * 2), idesc,
                       (j > 0 || k > 0 || kk > 0) ? 1u : 0u);
          mma_commit(smem_u32(&done[sx]));
        }
        any = true;
        if (++sa == SA) { sa = 0; pa ^= 1u; }
        if (++sx == SX) { sx = 0; px ^= 1u; }
        x_in = mbar_test(smem_u32(&x_full[sx]), px);
        a_in = mbar_test(smem_u32(&a_full[sa]), pa);
      }
      if (!ok) break;
      if (issuer) mma_commit(smem_u32(&acc_full[buf]));
      if (++buf == 2) { buf = 0; aph ^= 1u; }
    }
    if (any && issuer) {
      mma_commit(smem_u32(&drain_mb));
      drain_wait(smem_u32(&drain_mb), 0, p.limit_ns);
    }
    __syncwarp();
  } else if (warp >= W_WIDEN) {
    // a warp may only write its own quarter of the tensor memory's lanes
    const int group = (warp - W_WIDEN) >> 2, quarter = warp & 3;
    // this lane's output in a raw stage; SwiGLU: 16 outputs of W and the same 16 of W3
    // share a warp's lanes
    const int r = SWIGLU ? (lane >> 4) * 64 + quarter * 16 + (lane & 15) : quarter * 32 + lane;
    const int ng = RAW_K >> p.log_g, swz = (r >> 1) & 3;
    const uint32_t scale_at = CODE_BYTES + (SWIGLU ? (r >> 6) * ng * BM + (r & 63) * 2 : r * 2);
    const uint32_t scale_step = SWIGLU ? BM : BM * 2;
    uint32_t code[4], scale[4];        // where its four runs of 32 codes and their scales lie
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      code[c] = rbase + r * 64 + (c ^ swz) * 16;
      scale[c] = rbase + scale_at + ((c * 32) >> p.log_g) * scale_step;
    }
    const uint32_t to0 = tmem + ((uint32_t)(quarter * 32) << 16) + 2 * BN;
    const int mine = (total - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    const long long raws = (long long)mine * nraw;
    int q = group, j = group, last = group;      // (j: stage of a tile) every NG-th is the group's
    uint32_t qph = 0, ph = 0;
    const uint32_t to = to0 + group * 64;
    for (long long i = group; i < raws; i += NG) {
      if (!all_wait(smem_u32(&raw_full[q]), qph)) break;
      uint4 c4[4];
      uint32_t sc[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        c4[c] = lds128(code[c] + q * RAW_BYTES);
        sc[c] = lds_scale(scale[c] + q * RAW_BYTES);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&raw_empty[q]));
      q += NG;
      if (q >= Q) { q -= Q; qph ^= 1u; }
      while (j >= nraw) j -= nraw;
      if (j == nraw - 1) {             // past the last input: zeros, whatever the scale
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (j * RAW_K + c * 32 >= p.K) sc[c] = 0u;
      }
      j += NG;
      uint4 w[2][2][4];
      const uint32_t ok = q4_fast(__byte_perm(sc[0], sc[1], 0x5410)) & q4_fast(__byte_perm(sc[2], sc[3], 0x5410));
      if (__all_sync(0xffffffffu, (ok & 0x80008000u) == 0x80008000u)) {
        q4_runs<true>(c4[0], c4[1], sc[0], sc[1], w[0]);
        q4_runs<true>(c4[2], c4[3], sc[2], sc[3], w[1]);
      } else {
        q4_runs<false>(c4[0], c4[1], sc[0], sc[1], w[0]);
        q4_runs<false>(c4[2], c4[3], sc[2], sc[3], w[1]);
      }
      if (i >= NG) {                   // the products of its last stage
        if (!all_wait(smem_u32(&done[last]), ph)) break;
        last += NG;
        if (last >= SX) { last -= SX; ph ^= 1u; }
      }
      tc_fence_after();
      tmem_st32(to, w[0]);
      tmem_st32(to + 32, w[1]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&a_full[group]));
    }
  } else {
    const int quarter = warp & 3;            // of the accumulator's lanes that this warp may read
    int buf = 0;
    uint32_t aph = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      const Tile T = tile_at(t, p, tb);
      if (!all_wait(smem_u32(&acc_full[buf]), aph)) break;
      tc_fence_after();
      const uint32_t at = tmem + (uint32_t)(buf * BN) + ((uint32_t)(quarter * 32) << 16);
      const int f = T.f0 + (SWIGLU ? quarter * 16 + (lane & 15) : quarter * 32 + lane);
      const bool on = f < p.N;
      const float bias = !SWIGLU && p.bias != nullptr && on ? p.bias[(long long)T.e * p.N + f] : 0.f;
      // Lanes pair up so that each stores two outputs of every other row: lane and
      // lane ^ 1 (their own outputs), for SwiGLU after lane ^ 16 has given W3's
      const bool odd = lane & 1, upper = lane >= 16;
      uint32_t* c = reinterpret_cast<uint32_t*>(p.c + (long long)T.r0 * p.N + (f & ~1));
      const int half_n = p.N / 2;              // (N is even: a row is a whole number of pairs)
      for (int col = 0; col < T.n; col += 16) {
        float v[16];
        tmem_ld16(at + col, v);
        tmem_ld_wait();
        const int left = T.n - col;
        if (SWIGLU) {
          // lanes 0..15 have W's outputs, 16..31 W3's: of two rows each half takes one
          float u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, upper ? v[2 * i] : v[2 * i + 1], 16);
            const float h1 = Q4_UNSCALE * (upper ? got : v[2 * i]);
            const float h3 = Q4_UNSCALE * (upper ? v[2 * i + 1] : got);
            u[i] = (h1 * sigmoid_epi(h1)) * h3;          // of row 2 i + upper
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? u[i] : u[i + 1], 1);
            const int n = 2 * (i + (odd ? 1 : 0)) + (upper ? 1 : 0);
            const uint32_t two = pair_bf16(odd ? got : u[i], odd ? u[i + 1] : got);
            if (on && n < left) c[(long long)n * half_n] = two;
          }
        } else {
          if (p.act == 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = gelu_epi(fmaf(v[i], Q4_UNSCALE, bias));
          } else if (p.act == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              v[i] = fmaf(v[i], Q4_UNSCALE, bias);
              v[i] = v[i] < 0.f ? 0.f : v[i];            // a NaN stays one
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = fmaf(v[i], Q4_UNSCALE, bias);
          }
          uint32_t* to = c + (odd ? half_n : 0);
#pragma unroll
          for (int i = 0; i < 16; i += 2, to += 2ll * half_n) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
            const uint32_t two = pair_bf16(odd ? got : v[i], odd ? v[i + 1] : got);
            if (on && i + (odd ? 1 : 0) < left) *to = two;
          }
        }
        c += 16ll * half_n;
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

template <bool SWIGLU>
cudaError_t launch_t(const XMaps& x, const CUtensorMap* maps, const Params& p, long long tiles,
                     cudaStream_t st) {
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = ensure_dynamic_smem(q4_gemm_kernel<SWIGLU>, SMEM, attr_done);
  if (e != cudaSuccess) return e;
  const int sms = sm_count(), grid = tiles < sms ? (int)tiles : sms;
  return launch_pdl(q4_gemm_kernel<SWIGLU>, dim3(grid), dim3(THREADS), SMEM, st, x, maps[0], maps[1],
                    maps[2], maps[3], p);
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
  p.limit_ns = q.limit_ns > 0 ? q.limit_ns : LIMIT_NS;
  p.stall = q.stall;
  CUtensorMap maps[4];
  XMaps x;
  const uint64_t xd[2] = {(uint64_t)q.K, (uint64_t)q.R}, xs[1] = {(uint64_t)q.K * 2};
  bool ok = true;
  for (int i = 0; i < X_BOXES && ok; ++i) {
    const uint32_t xb[2] = {BK, (uint32_t)box_rows(i)};
    ok = encode(&x.box[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, q.x, 2, xd, xs, xb);
  }
  const uint64_t groups = (uint64_t)q4_groups(q.K, q.G);
  const uint64_t wd[3] = {(uint64_t)q.K / 2, (uint64_t)q.N, (uint64_t)q.E};
  const uint64_t ws[2] = {(uint64_t)q.K / 2, (uint64_t)q.N * (uint64_t)q.K / 2};
  const uint32_t wb[3] = {RAW_K / 2, (uint32_t)p.per, 1};
  const uint64_t sd[3] = {(uint64_t)q.N, groups, (uint64_t)q.E};
  const uint64_t ss[2] = {(uint64_t)q.N * 2, (uint64_t)q.N * groups * 2};
  const uint32_t sb[3] = {(uint32_t)p.per, (uint32_t)(RAW_K / q.G), 1};
  for (int i = 0; i < 2 && ok; ++i) {
    if (i == 1 && !swiglu) {
      maps[2] = maps[0];
      maps[3] = maps[1];
      break;
    }
    ok = encode(&maps[2 * i], CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_64B,
                i ? q.codes3 : q.codes, 3, wd, ws, wb) &&
         encode(&maps[1 + 2 * i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_NONE,
                i ? q.scales3 : q.scales, 3, sd, ss, sb);
  }
  if (!ok) return cudaErrorInvalidValue;
  const long long tiles = ((long long)q.R / 16 + q.E) * p.nF;      // at most
  return swiglu ? launch_t<true>(x, maps, p, tiles, st) : launch_t<false>(x, maps, p, tiles, st);
}

}  // namespace moe
