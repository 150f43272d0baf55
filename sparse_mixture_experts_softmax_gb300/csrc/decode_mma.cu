// The MoE layer for a few tokens, bf16 layers, on the tensor cores: the same
// steps as decode.cu, for calls whose experts have several tokens each.
//
// A multiply-add per weight and token on the CUDA cores keeps up with HBM for
// one or two tokens an expert; from there on the products go to mma.sync tiles
// of 16 weight rows by 8 tokens (weights as the row operand, so that a handful
// of tokens wastes no more than the narrow side of a tile).  The tcgen05 path's
// smallest row tile would be 64 weight rows of one expert, too coarse to spread
// a small layer over 152 SMs; its rate is not needed, since HBM bounds the call.
//
// A block takes a contiguous range of items, an item being 16 weight rows (8 of
// W1 and the same 8 of W3 for SwiGLU, so that h1 and h3 meet in one thread)
// over the whole of K for one tile of up to 16 tokens.  The tiles' tokens lie in
// shared memory.  Each of eight warps copies the weights that it multiplies
// itself, 512 bytes of 16 rows at a time, into a double buffer of its own, so
// that no warp waits for another's copies.  KS = 1, 2, 4 or 8 of the warps share
// an item, taking every KS-th such stage of K; their partial tiles are added in
// a fixed order.  The buffers fill with W2 rows while the block waits at the
// grid barrier.  Three barriers: logits, hidden activations, and the
// per-assignment outputs, which a last pass combines in j order.
//
// Measured and left (64 tokens of the large layer, 0.93 ms of HBM traffic): rows
// from HBM straight to registers, 64 bytes of a row to a load, 1.71 ms, and with
// L2 prefetches ahead of them 1.21 ms; one ring of bulk copies for the block, its
// K split over 16 warps, 1.60 to 1.99 ms (a bulk copy takes its thread some 0.1
// us to issue, and the block waits for the slowest warp of every stage).
//
// The hidden activations enter the down projection as the sum of two bf16 values
// (16 bits of the fp32 ones, an error of 2^-17), so that the only rounding to 8
// bits is that of y.
#include "decode_common.cuh"

namespace moe {
namespace {

constexpr int WARPS = 16, THREADS = WARPS * 32;
constexpr int CW = 8, CTHREADS = CW * 32;       // warps that multiply (all of them route)
constexpr int SV = 256;                         // values of a row in a stage
constexpr int STAGE = 16 * SV * 2;
constexpr int NS = 2;                           // stages of a warp

__host__ __device__ constexpr int up16(int v) { return (v + 15) & ~15; }
// Bytes of one row of a tile in shared memory: 64 past a multiple of 128, so
// that the rows of two tokens a quarter-warp reads fall on different banks.
__host__ __device__ inline int row_pitch(int K) { return (K * 2 + 127) / 128 * 128 + 64; }
struct Plan {
  int off_red, off_idx, off_gate, off_tok, off_slot, off_tile, off_at, off_rows, rows_bytes;
};
__host__ __device__ inline Plan make_plan(int T, int k, int E, int Fs, int tt) {
  Plan p;
  const int R = T * k;
  const int tiles = (E < R ? E : R) + R / tt + (Fs ? (T + tt - 1) / tt : 0);
  int o = CW * NS * STAGE;   // (the router's and the selection's scratch lies there first)
  p.off_red = o; o += 2 * CW * 128 * (tt / 8) * 4;
  p.off_idx = o; o += up16(R * 2);
  p.off_gate = o; o += up16(R * 4);
  p.off_tok = o; o += up16(R * 2);
  p.off_slot = o; o += up16(R * 2);
  p.off_tile = o; o += up16(tiles * 8);
  p.off_at = o; o += up16(tiles * 4);
  p.off_rows = o;
  p.rows_bytes = SMEM_MAX - o;
  return p;
}
static_assert((768 + WARPS * 256) * 4 <= CW * NS * STAGE, "scratch");
// Tokens of a tile: 16, or 8 where 16 rows do not fit, or 0.
__host__ __device__ inline int tile_tokens(const DecodeArgs& a) {
  const int width = a.F > a.Fs ? a.F : a.Fs;
  if (a.D > 65536 || width > 65536) return 0;
  const int up = row_pitch(a.D), down = 2 * row_pitch(width);
  for (int tt = 16; tt >= 8; tt -= 8) {
    const int room = make_plan(a.T, a.k, a.E, a.Fs, tt).rows_bytes;
    if (tt * (up > down ? up : down) <= room) return tt;
  }
  return 0;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The block's share of one kind of items: the routed tiles' or the shared
// branch's, of one projection.
struct Part {
  const char* w;               // the matrix (W1 or W2; of all experts)
  long long second;            // bytes from rows 0..7 of an item to its rows 8..15
  int K, width;                // values of a row; rows of an expert's matrix
  int rows;                    // rows of an item in one matrix: 8 (SwiGLU) or 16
  int per;                     // items of a tile
  int t0;                      // first tile
  int lo, hi;                  // items, counted from the first tile
};
// First item of block b's share: the blocks' shares are of equal weight bytes.
__device__ __forceinline__ int share_of(int all_r, int K_r, int all_s, int K_s, int b) {
  const long long bytes_r = (long long)all_r * K_r;
  const long long at = (bytes_r + (long long)all_s * K_s) * b / (int)gridDim.x;
  return at < bytes_r ? (int)(at / K_r) : all_r + (all_s > 0 ? (int)((at - bytes_r) / K_s) : 0);
}
template <bool UP>
__device__ __forceinline__ Part make_part(const DecodeArgs& a, int n_routed, int n_tiles, bool routed) {
  Part p;
  const bool pair = UP && a.act == 2;
  const int width_r = UP ? a.F : a.D, width_s = UP ? a.Fs : a.D;
  p.rows = pair ? 8 : 16;
  const int per_r = (width_r + p.rows - 1) / p.rows, per_s = (width_s + p.rows - 1) / p.rows;
  const int K_r = UP ? a.D : a.F, K_s = UP ? a.D : a.Fs;
  const int all_r = n_routed * per_r, all_s = (n_tiles - n_routed) * per_s;
  const int lo = share_of(all_r, K_r, all_s, K_s, blockIdx.x);
  const int hi = share_of(all_r, K_r, all_s, K_s, blockIdx.x + 1);
  p.K = routed ? K_r : K_s;
  p.width = routed ? width_r : width_s;
  p.per = routed ? per_r : per_s;
  p.t0 = routed ? 0 : n_routed;
  p.lo = routed ? lo : max(lo - all_r, 0);
  p.hi = routed ? min(hi, all_r) : hi - all_r;
  p.w = static_cast<const char*>(UP ? (routed ? a.w1 : a.ws1) : (routed ? a.w2 : a.ws2));
  p.second = !pair ? 8ll * p.K * 2
                   : static_cast<const char*>(routed ? a.w3 : a.ws3) - p.w;
  return p;
}
// Rows 0..7 of block `blk` of tile `t`.
__device__ __forceinline__ const char* item_rows(const Part& p, const Tile* tiles, int t, int blk) {
  const int e = max((int)tiles[p.t0 + t].e, 0);
  return p.w + ((long long)e * p.width + (long long)blk * p.rows) * p.K * 2;
}
// Whether rows 8..15 of the block exist (the rows of a matrix are a multiple of 8).
__device__ __forceinline__ bool has_upper(const Part& p, int blk) {
  return p.rows == 8 || blk * 16 + 8 < p.width;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// A tile's token rows into shared memory (two planes for hidden activations);
// values from K to the next multiple of 32 are zero.  Absent tokens' rows hold
// anything: a column of the mma's result depends on its own token only.
template <bool UP>
__device__ __forceinline__ void load_tile(const DecodeArgs& a, const Routing& rt, const Tile& tl,
                                          int K, int nt8, char* rows) {
  const int pitch = row_pitch(K), pieces = (K + 31) / 32 * 4;      // of 8 values
  const int lo_plane = nt8 * 8 * pitch;
  for (int t = threadIdx.x >> 5; t < tl.n; t += CW) {              // a warp a token
    const int tok = tl.e >= 0 && UP ? rt.tok[tl.start + t] : tl.start + t;
    const bf16* x = static_cast<const bf16*>(a.x) + (long long)tok * a.D;
    const float* h = (tl.e >= 0 ? a.hidden : a.hidden_s) + (long long)tok * K;
#pragma unroll 4
    for (int c = threadIdx.x & 31; c < pieces; c += 32) {
      char* to = rows + t * pitch + c * 16;
      const bool on = c * 8 < K;
      if (UP) {
        *reinterpret_cast<uint4*>(to) =
            on ? __ldg(reinterpret_cast<const uint4*>(x + c * 8)) : make_uint4(0u, 0u, 0u, 0u);
      } else {
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f), q = p;
        if (on) {
          p = __ldcg(reinterpret_cast<const float4*>(h + c * 8));
          q = __ldcg(reinterpret_cast<const float4*>(h + c * 8) + 1);
        }
        const float v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u0 = v[2 * j], u1 = v[2 * j + 1];
          hi[j] = pack_bf16(u0, u1);
          lo[j] = pack_bf16(u0 - __uint_as_float(hi[j] << 16),
                            u1 - __uint_as_float(hi[j] & 0xffff0000u));
        }
        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(to + lo_plane) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
}

// 16 bytes of a weight row into shared memory, zeros where !on.
__device__ __forceinline__ void copy16(uint32_t dst, const char* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 load_rows(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

// One output pair of an item: rows r and r + 8 of the 16, token `tok` of the tile.
template <bool UP>
__device__ __forceinline__ void emit(const DecodeArgs& a, const Tile& tl, int block, int r, int tok,
                                     float v0, float v1) {
  if (tok >= tl.n) return;
  if constexpr (UP) {
    const int width = tl.e >= 0 ? a.F : a.Fs;
    float* o = (tl.e >= 0 ? a.hidden : a.hidden_s) + (long long)(tl.start + tok) * width;
    if (a.act == 2) {
      __stcg(o + block * 8 + r, silu_f(v0) * v1);
      return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = block * 16 + h * 8 + r;
      if (f >= width) break;
      float v = h ? v1 : v0;
      if (a.b1 != nullptr) v += a.b1[(long long)tl.e * a.F + f];
      __stcg(o + f, a.act == 1 ? gelu_tanh_f(v) : fmaxf(v, 0.f));
    }
  } else {
    const long long row = (tl.e >= 0 ? 0 : (long long)a.T * a.k) + tl.start + tok;
    const int d = block * 16 + r;
    __stcg(a.ye + row * a.D + d, v0);
    if (d + 8 < a.D) __stcg(a.ye + row * a.D + d + 8, v1);
  }
}

// Warps to an item: the number that takes the fewest quarter stages for the
// block's share, an item shared by several warps counting one more for adding
// their parts.
__device__ __forceinline__ int warps_per_item(int items, int K) {
  const int stages = (K + SV - 1) / SV;
  int best = 1, cost = 0x7fffffff;
  for (int ks = 1; ks <= CW; ks *= 2) {
    const int c = (items + CW / ks - 1) / (CW / ks) * ((stages + ks - 1) / ks * 4 + (ks > 1 ? 1 : 0));
    if (c < cost) {
      cost = c;
      best = ks;
    }
  }
  return best;
}

// The items of a part, by the multiplying warps.  Where `flag` is given, the grid
// barrier before the down projection stands between the first weight copies and
// the tiles' tokens.
template <bool UP>
__device__ __forceinline__ void compute(const DecodeArgs& a, const Part& p, const Routing& rt, int tt,
                                        int* row_at, char* rows, int rows_bytes, float* red,
                                     uint32_t ring, int* flag) {
  if (p.lo >= p.hi) {
    if (!UP && flag != nullptr) grid_barrier<CTHREADS>(a.ctl, 1, flag);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q8 = (lane & 3) * 8;
  const int K = p.K, KS = warps_per_item(p.hi - p.lo, K), groups = CW / KS;
  const int mine = warp / KS, ks = warp % KS;
  const int stages = (K + SV - 1) / SV, steps = (stages + KS - 1) / KS;
  const int pitch = row_pitch(K);
  const long long item_step = (long long)groups * p.rows * K * 2;

  // the next stage to be copied: item, its tile and block, step; rows 0..7 of it
  int li = p.lo + mine, lt = li / p.per, lb = li % p.per, ls = 0, put_slot = 0;
  const char* lp = li < p.hi ? item_rows(p, rt.tiles, lt, lb) : nullptr;
  auto put = [&] {
    const int v0 = (ls * KS + ks) * SV;
    if (li < p.hi && v0 < K) {
      // row r's 16-byte pieces change places with their neighbours 64 bytes on
      // for odd r, so that the rows a quarter-warp reads fall on different banks
      const uint32_t dst = ring + put_slot * STAGE + lane * 16;
      const bool on = v0 + lane * 8 < K;
      const char* src = lp + (on ? (v0 + lane * 8) * 2 : 0);
#pragma unroll
      for (int r = 0; r < 8; ++r) copy16((dst + r * SV * 2) ^ ((r & 1) << 6), src + (long long)r * K * 2, on);
      if (has_upper(p, lb)) {
        src += p.second;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          copy16((dst + (8 + r) * SV * 2) ^ ((r & 1) << 6), src + (long long)r * K * 2, on);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    put_slot = put_slot + 1 == NS ? 0 : put_slot + 1;
    if (++ls < steps) return;
    ls = 0;
    li += groups;
    lb += groups;
    lp += item_step;
    if (lb >= p.per && li < p.hi) {
      do { lb -= p.per; ++lt; } while (lb >= p.per);
      lp = item_rows(p, rt.tiles, lt, lb);
    }
  };
#pragma unroll
  for (int u = 0; u < NS; ++u) put();
  if (!UP && flag != nullptr) grid_barrier<CTHREADS>(a.ctl, 1, flag);

  // what is being computed: item, its tile and block
  int i = p.lo + mine, it = i / p.per, ib = i % p.per, parity = 0, slot = 0;
  for (int b_lo = p.lo; b_lo < p.hi;) {
    // the tokens of as many of the next tiles as there is room for
    int t = b_lo / p.per, used = 0;
    bar_sync<CTHREADS>();      // the last ones are no longer read
    const int first = t;
    for (; t * p.per < p.hi; ++t) {
      const Tile tl = rt.tiles[p.t0 + t];
      const int nt8 = tl.n <= 8 ? 1 : tt / 8;
      const int need = nt8 * 8 * pitch * (UP ? 1 : 2);
      if (t > first && used + need > rows_bytes) break;
      load_tile<UP>(a, rt, tl, K, nt8, rows + used);
      if (threadIdx.x == 0) row_at[t] = used;
      used += need;
    }
    const int b_hi = min(p.hi, t * p.per);
    b_lo = b_hi;
    bar_sync<CTHREADS>();

    while (i < b_hi) {
      const Tile tl = rt.tiles[p.t0 + it];
      const bool two = tl.n > 8;
      const int plane = (two ? 16 : 8) * pitch;
      const uint32_t at = smem_addr(rows + row_at[it]) + g * pitch + q8 * 2;
      float acc[2][2][4];      // token tiles of 8, chains of dependent products
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[0][0][c] = acc[0][1][c] = acc[1][0][c] = acc[1][1][c] = 0.f;
      for (int s = 0; s < steps; ++s) {
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        __syncwarp();
        const int v0 = (s * KS + ks) * SV;
        const int blocks = min(SV / 32, (K - v0 + 31) / 32);
        const uint32_t from = ring + slot * STAGE + g * SV * 2;
#pragma unroll 4
        for (int u = 0; u < blocks; ++u) {
          const uint32_t wat = (from + u * 64 + q8 * 2) ^ ((g & 1) << 6);
          const uint4 w0 = load_rows(wat), w1 = load_rows(wat + 8 * SV * 2);
          auto products = [&](float (&c0)[4], float (&c1)[4], uint32_t x_at) {
            const uint4 x = load_rows(x_at);
            mma16816(c0, w0.x, w1.x, w0.y, w1.y, x.x, x.y);
            mma16816(c1, w0.z, w1.z, w0.w, w1.w, x.z, x.w);
          };
          const uint32_t x_at = at + (v0 + u * 32) * 2;
          products(acc[0][0], acc[0][1], x_at);
          if (!UP) products(acc[0][0], acc[0][1], x_at + plane);
          if (two) {
            products(acc[1][0], acc[1][1], x_at + 8 * pitch);
            if (!UP) products(acc[1][0], acc[1][1], x_at + plane + 8 * pitch);
          }
        }
        __syncwarp();
        put();
        slot = slot + 1 == NS ? 0 : slot + 1;
      }
      const int nt = two ? 2 : 1;
      if (KS == 1) {
#pragma unroll
        for (int t8 = 0; t8 < 2; ++t8)
          if (t8 < nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              emit<UP>(a, tl, ib, g, t8 * 8 + (lane & 3) * 2 + c, acc[t8][0][c] + acc[t8][1][c],
                       acc[t8][0][c + 2] + acc[t8][1][c + 2]);
      } else {
        // partial tiles of the item's warps; two buffers, so one barrier an item is enough
        float* buf = red + parity * CW * (tt / 8) * 128 + mine * KS * (tt / 8) * 128;
        parity ^= 1;
#pragma unroll
        for (int t8 = 0; t8 < 2; ++t8)
          if (t8 < nt)
            *reinterpret_cast<float4*>(buf + (ks * nt + t8) * 128 + lane * 4) = make_float4(
                acc[t8][0][0] + acc[t8][1][0], acc[t8][0][1] + acc[t8][1][1],
                acc[t8][0][2] + acc[t8][1][2], acc[t8][0][3] + acc[t8][1][3]);
        asm volatile("bar.sync %0, %1;" ::"r"(2 + mine), "r"(KS * 32) : "memory");
        for (int o = ks * 32 + lane; o < nt * 64; o += KS * 32) {
          const int t8 = o / 64, l = (o % 64) / 2, c = o % 2;
          float v0 = 0.f, v1 = 0.f;
          for (int q = 0; q < KS; ++q) {
            const float* part = buf + (q * nt + t8) * 128 + l * 4 + c;
            v0 += part[0];
            v1 += part[2];
          }
          emit<UP>(a, tl, ib, l >> 2, t8 * 8 + (l & 3) * 2 + c, v0, v1);
        }
      }
      i += groups;
      ib += groups;
      while (ib >= p.per) { ib -= p.per; ++it; }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__global__ void __launch_bounds__(THREADS, 1)
decode_mma_kernel(const __grid_constant__ DecodeArgs a, const int tt) {
  extern __shared__ __align__(128) char sm[];
  __shared__ int flag, n_tiles, n_routed, scan[16];
  const Plan P = make_plan(a.T, a.k, a.E, a.Fs, tt);
  const int tid = threadIdx.x;
  const int T = a.T, D = a.D, k = a.k;
  const Routing rt{reinterpret_cast<short*>(sm + P.off_idx), reinterpret_cast<float*>(sm + P.off_gate),
                   reinterpret_cast<short*>(sm + P.off_tok), reinterpret_cast<short*>(sm + P.off_slot),
                   reinterpret_cast<Tile*>(sm + P.off_tile), scan};
  float* red = reinterpret_cast<float*>(sm + P.off_red);
  char* rows = sm + P.off_rows;

  const int magic = tid == 0 ? __ldcg(a.ctl + DC_MAGIC) : 0;     // (looked at after the logits)

  float* scratch = reinterpret_cast<float*>(sm);
  router<bf16, WARPS>(a, scratch);
  if (tid == 0) flag = magic == DECODE_MAGIC ? 0 : 2;
  __syncthreads();
  if (flag != 0) {   // the workspace was not initialised: the counters mean nothing
    if (tid == 0) a.ctl[DC_STATUS] = DEV_STATUS_INVALID_INDEX;
    return;
  }
  const bool ok = grid_barrier<THREADS>(a.ctl, 0, &flag);
  if (ok) select_all<WARPS>(a, rt, tt, scratch, &n_routed, &n_tiles);
  const int nr = ok ? n_routed : 0, nt = ok ? n_tiles : 0;

  int* row_at = reinterpret_cast<int*>(sm + P.off_at);
  const int warp = tid >> 5;
  if (warp < CW) {
    const uint32_t ring = smem_addr(sm) + warp * NS * STAGE;
#pragma unroll 1
    for (int shared = 0; shared < (a.Fs > 0 ? 2 : 1); ++shared)
      compute<true>(a, make_part<true>(a, nr, nt, !shared), rt, tt, row_at + shared * nr, rows,
                    P.rows_bytes, red, ring, nullptr);
#pragma unroll 1
    for (int shared = 0; shared < (a.Fs > 0 ? 2 : 1); ++shared)
      compute<false>(a, make_part<false>(a, nr, nt, !shared), rt, tt, row_at + shared * nr, rows,
                     P.rows_bytes, red, ring, shared ? nullptr : &flag);
    grid_barrier<CTHREADS>(a.ctl, 2, &flag);
  }
  __syncthreads();
  if (flag == 0) {
    // y[t, d] = sum over j of gate (Y_e + b2), + the shared branch: eight lanes
    // take the assignments of four values of y, and a fixed tree adds them
    const int quads = D / 4, j0 = tid & 7, terms = k + (a.Fs > 0 ? 1 : 0);
    const int step = gridDim.x * (THREADS / 8);
    for (int i0 = (blockIdx.x * THREADS + tid) / 8; i0 < T * quads; i0 += 2 * step) {
      float4 v[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = min(i0 + u * step, T * quads - 1), t = i / quads, d = (i % quads) * 4;
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int j = j0; j < terms; j += 8) {
          const int s = j < k ? rt.slot[t * k + j] : T * k + t;
          if (s < 0) continue;
          float4 h = __ldcg(reinterpret_cast<const float4*>(a.ye + (long long)s * D + d));
          if (a.b2 != nullptr) {           // (a layer with biases has no shared branch)
            const float4 q = __ldg(reinterpret_cast<const float4*>(
                a.b2 + (long long)rt.idx[t * k + j] * D + d));
            h.x += q.x; h.y += q.y; h.z += q.z; h.w += q.w;
          }
          const float w = j < k ? rt.gate[t * k + j] : 1.f;
          v[u].x = fmaf(w, h.x, v[u].x); v[u].y = fmaf(w, h.y, v[u].y);
          v[u].z = fmaf(w, h.z, v[u].z); v[u].w = fmaf(w, h.w, v[u].w);
        }
      }
      // (the eight lanes of an output run through the loop together)
      const uint32_t m8 = 0xffu << (tid & 24);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          v[u].x += __shfl_xor_sync(m8, v[u].x, o); v[u].y += __shfl_xor_sync(m8, v[u].y, o);
          v[u].z += __shfl_xor_sync(m8, v[u].z, o); v[u].w += __shfl_xor_sync(m8, v[u].w, o);
        }
        const int i = i0 + u * step;
        if (j0 == 0 && i < T * quads)
          *reinterpret_cast<uint2*>(static_cast<bf16*>(a.y) + (long long)i * 4) =
              make_uint2(pack_bf16(v[u].x, v[u].y), pack_bf16(v[u].z, v[u].w));
      }
    }
  }
  __syncthreads();
  if (tid == 0) leave(a.ctl);
}

}  // namespace

bool decode_mma_fits(const DecodeArgs& a) { return tile_tokens(a) > 0; }

cudaError_t launch_decode_mma(const DecodeArgs& a, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> attr_done{0};
  // a block per SM, or fewer where each would have less than 8 KB of weights
  const long long experts = (long long)a.T * a.k < a.E ? (long long)a.T * a.k : a.E;
  const long long bytes = (experts * a.F + a.Fs) * a.D * (a.act == 2 ? 3 : 2) * 2;
  const long long blocks = (bytes + 8191) / 8192;
  return launch_cooperative(decode_mma_kernel, (int)(blocks < sms ? blocks : sms), THREADS,
                            attr_done, st, a, tile_tokens(a));
}

}  // namespace moe
