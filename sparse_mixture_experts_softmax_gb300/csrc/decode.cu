// The whole MoE layer for a few tokens in one launch: router, selection, expert
// MLPs, combine.
//
// A call of T tokens reads the weights of the at most min(E, T k) experts its
// tokens choose, once; for T up to some tens that is all that bounds it (one
// multiply-add per weight and token against 2 or 4 bytes of HBM traffic).  So
// the kernel is a streaming one: a cooperative grid of one block per SM walks
// the weight rows in order, every warp copying its rows with bulk asynchronous
// copies into a ring of its own in shared memory, and the tokens' activations
// stay on chip.  Two grid barriers separate the three steps that depend on each
// other across blocks:
//   1  logits = x W_g^T            one expert and up to 8 tokens per block
//   -- barrier: the logits
//   2  selection, by every block for itself (cheaper than a third barrier);
//      a = act(W1 x) or SiLU(W1 x) * (W3 x), one weight row per warp at a time
//   -- barrier: the hidden activations; the ring already fills with W2 rows
//   3  y = sum_j gate_j W2 a_j     one row per warp, all rows of an output
//      column in one block, which adds them in j order
// No floating-point atomics: sums are taken in a fixed order.
#include "decode_common.cuh"

namespace moe {
namespace {

constexpr int WARPS = 16, THREADS = WARPS * 32;
constexpr int STAGE = 4096;       // bytes of one stage of a warp's ring
constexpr int NS = 2;             // stages of a ring
constexpr int RING = WARPS * NS * STAGE;
constexpr int TT = 8;             // tokens that share one pass over a weight row

// Eight values of a weight row and of an activation row for one lane, as four
// pairs.  Two bf16 rows are read 8 consecutive values a lane; a row beside an
// fp32 one 4 + 4 values, 128 apart, so that the fp32 reads (16 bytes a lane)
// stay free of bank conflicts.  `left` is the row's remaining length from the
// warp's first value (a multiple of 8); a lane past it contributes zeros.
template <typename WT, typename AT>
struct Lane8 {
  static constexpr bool kWide = sizeof(WT) == 2 && sizeof(AT) == 2;
  template <typename T>
  static __device__ __forceinline__ void load(const T* p, int lane, int left, f32x2 (&v)[4]) {
    if constexpr (kWide) {
      if (lane * 8 < left) {
        const uint4 q = *reinterpret_cast<const uint4*>(p + lane * 8);
        v[0] = widen(q.x); v[1] = widen(q.y); v[2] = widen(q.z); v[3] = widen(q.w);
      } else {
        v[0] = v[1] = v[2] = v[3] = 0;
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h * 128 + lane * 4 < left) {
          if constexpr (sizeof(T) == 2) {
            const uint2 q = *reinterpret_cast<const uint2*>(p + h * 128 + lane * 4);
            v[2 * h] = widen(q.x);
            v[2 * h + 1] = widen(q.y);
          } else {
            const uint4 q = *reinterpret_cast<const uint4*>(p + h * 128 + lane * 4);
            v[2 * h] = pack2(q.x, q.y);
            v[2 * h + 1] = pack2(q.z, q.w);
          }
        } else {
          v[2 * h] = v[2 * h + 1] = 0;
        }
      }
    }
  }
};

// ---- a warp's ring: pieces of weight rows in stages of STAGE bytes.  An item
// is one row, or (PAIR) the rows at `w` and `w + second` side by side.
struct Item {
  const char* w;
  int K;              // values of a row
  int tile;           // token tile
  int row;            // f (up) or the batch's output row (down)
};
struct Ring {
  char* buf;          // this warp's NS stages
  uint32_t bar;       // this warp's NS mbarriers
  uint32_t put, got;  // stages issued / consumed so far
};
// The producer's place in a warp's sequence of items.
struct Cursor {
  int q, k0, K;       // item number, first value of its next piece, its length
  const char* w;
};
// Values of one row that a stage takes.
template <typename WT, bool PAIR>
constexpr int piece() { return STAGE / (int)sizeof(WT) / (PAIR ? 2 : 1); }

// Copies the next piece of the warp's items into its next stage.
template <typename WT, bool PAIR, typename Src>
__device__ __forceinline__ void feed(Ring& r, Cursor& c, int step, int n, const Src& src,
                                     long long second, int lane) {
  if (c.q >= n) return;
  if (c.k0 == 0) {
    const Item it = src(c.q);
    c.w = it.w;
    c.K = it.K;
  }
  constexpr int KC = piece<WT, PAIR>();
  if (lane == 0) {
    const uint32_t s = r.put % NS, bar = r.bar + s * 8, dst = smem_addr(r.buf + s * STAGE);
    const uint32_t bytes = (uint32_t)min(KC, c.K - c.k0) * sizeof(WT);
    const char* from = c.w + (long long)c.k0 * sizeof(WT);
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                 "r"(PAIR ? 2 * bytes : bytes) : "memory");
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "l"(from), "r"(bytes), "r"(bar) : "memory");
    if (PAIR)
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
          ::"r"(dst + STAGE / 2), "l"(from + second), "r"(bytes), "r"(bar) : "memory");
  }
  ++r.put;
  c.k0 += KC;
  if (c.k0 >= c.K) {
    c.k0 = 0;
    c.q += step;
  }
}

// Dot products of an item's rows with NT activation rows (`off`: their first
// values in `act`); refills the ring as it empties it.  The sums are whole on
// every lane.  False when a wait expired.
template <int NT, bool PAIR, typename WT, typename AT, typename Feed>
__device__ __forceinline__ bool dots(Ring& r, int K, const AT* act, const int (&off)[NT], int lane,
                                     const Feed& refill, float (&s0)[NT], float (&s1)[NT]) {
  constexpr int KC = piece<WT, PAIR>();
  f32x2 a0[NT], a1[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) a0[t] = a1[t] = 0;
  for (int k0 = 0; k0 < K; k0 += KC) {
    const uint32_t s = r.got % NS;
    if (!mbar_wait(r.bar + s * 8, (r.got / NS) & 1)) return false;
    const WT* w0 = reinterpret_cast<const WT*>(r.buf + s * STAGE);
    const int len = min(KC, K - k0);
    for (int i = 0; i < len; i += 256) {
      f32x2 p[4], q[4], v[4];
      Lane8<WT, AT>::load(w0 + i, lane, len - i, p);
      if (PAIR) Lane8<WT, AT>::load(w0 + KC + i, lane, len - i, q);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        Lane8<WT, AT>::load(act + off[t] + k0 + i, lane, len - i, v);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          fma2(a0[t], p[u], v[u]);
          if (PAIR) fma2(a1[t], q[u], v[u]);
        }
      }
    }
    __syncwarp();
    ++r.got;
    refill();
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    s0[t] = warp_sum(sum2(a0[t]));
    if (PAIR) s1[t] = warp_sum(sum2(a1[t]));
  }
  return true;
}

// One item for its tile's n tokens: emit(t, s0, s1) on lane t < n.
template <bool PAIR, typename WT, typename AT, typename Feed, typename Off, typename Emit>
__device__ __forceinline__ bool one_item(Ring& r, int n, int K, const AT* act, const Off& off_of,
                                         int lane, const Feed& refill, const Emit& emit) {
  auto pass = [&](auto nt_c) {
    constexpr int NT = decltype(nt_c)::value;
    int off[NT];
    float s0[NT], s1[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) off[t] = off_of(min(t, n - 1));
    if (!dots<NT, PAIR, WT, AT>(r, K, act, off, lane, refill, s0, s1)) return false;
    float h0 = s0[0], h1 = PAIR ? s1[0] : 0.f;
#pragma unroll
    for (int t = 1; t < NT; ++t)
      if (lane == t) {
        h0 = s0[t];
        if (PAIR) h1 = s1[t];
      }
    if (lane < n) emit(lane, h0, h1);
    return true;
  };
  switch (n) {
    case 1: return pass(std::integral_constant<int, 1>{});
    case 2: return pass(std::integral_constant<int, 2>{});
    case 3: return pass(std::integral_constant<int, 3>{});
    case 4: return pass(std::integral_constant<int, 4>{});
    case 5:
    case 6: return pass(std::integral_constant<int, 6>{});
    default: return pass(std::integral_constant<int, 8>{});
  }
}

// Shared-memory plan of a call, the same on host and device.
struct Plan {
  int off_bar, off_idx, off_gate, off_tok, off_slot, off_tile, off_part, off_act;
  int part_rows;      // output rows whose partial results are held at a time
  int act_bytes;      // space for the activations (x, then the hidden values)
};
__host__ __device__ inline int up16(int v) { return (v + 15) & ~15; }
__host__ __device__ inline Plan make_plan(const DecodeArgs& a) {
  Plan p;
  const int R = a.T * a.k;
  const int tiles = (a.E < R ? a.E : R) + R / TT + (a.Fs ? (a.T + TT - 1) / TT : 0);
  // (the router's and the selection's scratch lies where the ring will be)
  int o = RING;
  p.off_bar = o; o += up16(WARPS * NS * 8);
  p.off_idx = o; o += up16(R * 2);
  p.off_gate = o; o += up16(R * 4);
  p.off_tok = o; o += up16(R * 2);
  p.off_slot = o; o += up16(R * 2);
  p.off_tile = o; o += up16(tiles * 8);
  p.off_part = o;
  const int row = (R + (a.Fs ? a.T : 0)) * 4;
  p.part_rows = 24576 / row < 1 ? 1 : 24576 / row;
  if (p.part_rows > 64) p.part_rows = 64;
  o += up16(p.part_rows * row);
  p.off_act = o;
  p.act_bytes = SMEM_MAX - o;
  return p;
}

template <typename WT>
__global__ void __launch_bounds__(THREADS, 1)
decode_kernel(const __grid_constant__ DecodeArgs a) {
  extern __shared__ __align__(128) char sm[];
  __shared__ int flag, n_tiles, n_routed, scan[16];
  const Plan P = make_plan(a);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = a.T, D = a.D, F = a.F, k = a.k, R = T * k;
  const int G = gridDim.x, cta = blockIdx.x;
  const Routing rt{reinterpret_cast<short*>(sm + P.off_idx), reinterpret_cast<float*>(sm + P.off_gate),
                   reinterpret_cast<short*>(sm + P.off_tok), reinterpret_cast<short*>(sm + P.off_slot),
                   reinterpret_cast<Tile*>(sm + P.off_tile), scan};
  const Tile* tiles = rt.tiles;
  float* part = reinterpret_cast<float*>(sm + P.off_part);
  char* act = sm + P.off_act;
  const WT* x = static_cast<const WT*>(a.x);

  const int magic = tid == 0 ? __ldcg(a.ctl + DC_MAGIC) : 0;     // (looked at after the logits)
  if (tid < WARPS * NS)
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(sm + P.off_bar) + tid * 8));
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();

  // ---- 1: logits
  float* scratch = reinterpret_cast<float*>(sm);
  router<WT, WARPS>(a, scratch);
  // the tokens into shared memory while the other blocks finish their logits
  const bool x_in = (long long)T * D * (int)sizeof(WT) <= P.act_bytes;
  if (x_in) {
    const int n16 = T * D * (int)sizeof(WT) / 16;
    for (int i = tid; i < n16; i += THREADS)
      reinterpret_cast<uint4*>(act)[i] = __ldg(reinterpret_cast<const uint4*>(x) + i);
  }
  if (tid == 0) flag = magic == DECODE_MAGIC ? 0 : 2;
  __syncthreads();
  if (flag != 0) {   // the workspace was not initialised: the counters mean nothing
    if (tid == 0) a.ctl[DC_STATUS] = DEV_STATUS_INVALID_INDEX;
    return;
  }
  bool ok = grid_barrier<THREADS>(a.ctl, 0, &flag);
  if (ok) select_all<WARPS>(a, rt, TT, scratch, &n_routed, &n_tiles);
  // the ring's memory held scratch: order those accesses before the copies
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();

  Ring ring{sm + warp * NS * STAGE, smem_addr(sm + P.off_bar) + warp * NS * 8, 0, 0};
  const int nt_r = ok ? n_routed : 0, nt_all = ok ? n_tiles : 0;
  const int gw = warp * G + cta, step = WARPS * G;

  // ---- 2: hidden activations, rows of all blocks' warps in order
  const int rows_r = nt_r * F, rows_up = rows_r + (nt_all - nt_r) * a.Fs;
  auto up_src = [&](int q) {
    Item it;
    const bool routed = q < rows_r;
    const int width = routed ? F : a.Fs, p = routed ? q : q - rows_r;
    it.tile = (routed ? 0 : nt_r) + p / width;
    it.row = p % width;
    it.K = D;
    const long long row = routed ? (long long)tiles[it.tile].e * F + it.row : it.row;
    it.w = static_cast<const char*>(routed ? a.w1 : a.ws1) + row * D * (long long)sizeof(WT);
    return it;
  };
  auto up = [&](auto pair_c, const WT* xs) {
    constexpr bool PAIR = decltype(pair_c)::value;
    // (W3 of the shared branch lies elsewhere than the experts': the distance
    // goes with the item that is being issued)
    const long long second_r = PAIR ? static_cast<const char*>(a.w3) - static_cast<const char*>(a.w1) : 0;
    const long long second_s = PAIR && a.Fs > 0
        ? static_cast<const char*>(a.ws3) - static_cast<const char*>(a.ws1) : 0;
    Cursor cur{gw, 0, 0, nullptr};
    auto refill = [&] {
      feed<WT, PAIR>(ring, cur, step, rows_up, up_src, cur.q < rows_r ? second_r : second_s, lane);
    };
    for (int s = 0; s < NS; ++s) refill();
    for (int q = gw; q < rows_up && ok; q += step) {
      const Item it = up_src(q);
      const Tile tl = tiles[it.tile];
      auto off_of = [&](int t) { return (tl.e >= 0 ? rt.tok[tl.start + t] : tl.start + t) * D; };
      auto emit = [&](int t, float h1, float h3) {
        float v;
        if (PAIR) {
          v = silu_f(h1) * h3;
        } else {
          if (a.b1 != nullptr) h1 += a.b1[(long long)tl.e * F + it.row];
          v = a.act == 1 ? gelu_tanh_f(h1) : fmaxf(h1, 0.f);
        }
        float* o = tl.e >= 0 ? a.hidden + (long long)(tl.start + t) * F
                             : a.hidden_s + (long long)(tl.start + t) * a.Fs;
        __stcg(o + it.row, v);
      };
      ok = one_item<PAIR, WT, WT>(ring, tl.n, D, xs, off_of, lane, refill, emit);
    }
  };
  const WT* xs = x_in ? reinterpret_cast<const WT*>(act) : x;
  if (a.act == 2) up(std::true_type{}, xs);
  else up(std::false_type{}, xs);

  // ---- 3: output rows d = cta, cta + G, ...; the first rows of W2 are on
  // their way before the barrier
  const int rows_own = cta < D ? (D - cta + G - 1) / G : 0;
  const long long a_bytes = ((long long)R * F + (long long)T * a.Fs) * 4;
  const bool a_in = a_bytes <= P.act_bytes;
  const int prow = R + (a.Fs ? T : 0);
  // both hidden buffers from one base (they lie one after the other)
  const float* hid = a_in ? reinterpret_cast<const float*>(act) : a.hidden;
  const int hid_s = a_in ? R * F : (int)(a.hidden_s - a.hidden);
  for (int r0 = 0; r0 < rows_own || r0 == 0; r0 += P.part_rows) {
    const int nr = min(P.part_rows, rows_own - r0), items = nr > 0 ? nr * nt_all : 0;
    auto down_src = [&](int q) {
      Item it;
      it.tile = q % nt_all;
      it.row = q / nt_all;
      const int e = tiles[it.tile].e;
      const long long d = cta + (long long)(r0 + it.row) * G;
      it.K = e >= 0 ? F : a.Fs;
      it.w = static_cast<const char*>(e >= 0 ? a.w2 : a.ws2) +
             (e >= 0 ? ((long long)e * D + d) * F : d * a.Fs) * (long long)sizeof(WT);
      return it;
    };
    Cursor cur{warp, 0, 0, nullptr};
    auto refill = [&] { feed<WT, false>(ring, cur, WARPS, items, down_src, 0, lane); };
    if (ok)
      for (int s = 0; s < NS; ++s) refill();
    if (r0 == 0) {
      const bool all = grid_barrier<THREADS>(a.ctl, 1, &flag);
      ok = ok && all;
      if (a_in && all) {
        const int n1 = R * F / 4, n2 = T * a.Fs / 4;
        for (int i = tid; i < n1; i += THREADS)
          reinterpret_cast<uint4*>(act)[i] = __ldcg(reinterpret_cast<const uint4*>(a.hidden) + i);
        for (int i = tid; i < n2; i += THREADS)
          reinterpret_cast<uint4*>(act)[n1 + i] =
              __ldcg(reinterpret_cast<const uint4*>(a.hidden_s) + i);
      }
      __syncthreads();
    }
    for (int q = warp; q < items && ok; q += WARPS) {
      const Item it = down_src(q);
      const Tile tl = tiles[it.tile];
      auto off_of = [&](int t) {
        const int s = tl.start + t;
        return tl.e >= 0 ? s * F : hid_s + s * a.Fs;
      };
      auto emit = [&](int t, float v, float) {
        part[it.row * prow + (tl.e >= 0 ? 0 : R) + tl.start + t] = v;
      };
      ok = one_item<false, WT, float>(ring, tl.n, it.K, hid, off_of, lane, refill, emit);
    }
    __syncthreads();
    // y[t, d] = sum over j of gate (W2 a + b2), in j order, + the shared branch
    for (int i = tid; i < nr * T; i += THREADS) {
      const int row = i % nr, t = i / nr;
      const long long d = cta + (long long)(r0 + row) * G;
      float v = 0.f;
      for (int j = 0; j < k; ++j) {
        const int s = rt.slot[t * k + j];
        if (s < 0) continue;
        float h = part[row * prow + s];
        if (a.b2 != nullptr) h += a.b2[(long long)rt.idx[t * k + j] * D + d];
        v = fmaf(rt.gate[t * k + j], h, v);
      }
      if (a.Fs > 0) v += part[row * prow + R + t];
      if (ok) static_cast<WT*>(a.y)[(long long)t * D + d] = from_f<WT>(v);
    }
    __syncthreads();
  }
  if (!ok && lane == 0) a.ctl[DC_STATUS] = DEV_STATUS_TIMEOUT;
  // copies still in flight (only after an expired wait) land before the block goes
  while (ring.got != ring.put) {
    mbar_wait(ring.bar + (ring.got % NS) * 8, (ring.got / NS) & 1);
    ++ring.got;
  }
  __syncthreads();
  if (tid == 0) leave(a.ctl);
}

__global__ void decode_init_kernel(int* ctl) {
  pdl_begin();
  if (threadIdx.x < DC_WORDS) ctl[threadIdx.x] = threadIdx.x == DC_MAGIC ? DECODE_MAGIC : 0;
}

int sm_count() {
  static std::atomic<int> n{0};
  int v = n.load(std::memory_order_relaxed);
  if (v == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 0;
    n.store(v, std::memory_order_relaxed);
  }
  return v;
}

}  // namespace

template <typename WT>
static cudaError_t launch_t(const DecodeArgs& a, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> attr_done{0};
  // a block per SM, or fewer where each would have less than 4 KB of weights
  const long long experts = (long long)a.T * a.k < a.E ? (long long)a.T * a.k : a.E;
  const long long bytes = (experts * a.F + a.Fs) * a.D * (a.act == 2 ? 3 : 2) * (int)sizeof(WT);
  const long long blocks = (bytes + 4095) / 4096;
  return launch_cooperative(decode_kernel<WT>, (int)(blocks < sms ? blocks : sms), THREADS,
                            attr_done, st, a);
}

cudaError_t launch_decode_init(int* ctl, cudaStream_t st) {
  return launch_pdl(decode_init_kernel, dim3(1), dim3(DC_WORDS), 0, st, ctl);
}

cudaError_t launch_decode(int dtype, const DecodeArgs& a, cudaStream_t st) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorUnknown;
  if (dtype == 1 && decode_mma_fits(a)) return launch_decode_mma(a, sms, st);
  return dtype == 1 ? launch_t<bf16>(a, sms, st) : launch_t<float>(a, sms, st);
}

}  // namespace moe
