// The whole MoE layer for a few tokens in one launch: router, selection, expert
// MLPs, shared branch, combine.
//
// A call of T tokens reads the weights of the at most min(E, T k) experts that
// its tokens choose; for T up to some tens that is all that bounds it (a
// multiply-add per weight and token against 2 or 4 bytes of HBM traffic), as long
// as an expert's tokens fit one tile: every further tile reads its weights again
// (8 experts, k = 2, D = 4096, 64 tokens: 437 us at F = 4096 with tiles of 5, 1570
// at F = 8192 with tiles of 2, where the bytes alone would take 119 and 237).  So the
// kernel is a streaming one: a cooperative grid of one block per SM, with three
// grid barriers between the steps that depend on one another across blocks:
//   1  logits = x W_g^T
//   -- barrier: the logits
//   2  selection, by every block for itself (cheaper than another barrier);
//      a = act(W1 x) or SiLU(W1 x) * (W3 x)
//   -- barrier: the hidden activations; the buffers fill with W2 rows meanwhile
//   3  y_j = W2 a_j of every assignment
//   -- barrier, and a last pass that combines them with the gates
// No floating-point atomics: sums are taken in a fixed order.
//
// In 2 and 3 a block takes a contiguous range of items of equal bytes, an item
// being 16 weight rows (8 of W1 and the same 8 of W3 for SwiGLU, so that h1 and
// h3 meet in one thread) over the whole of K for one tile of tokens, up to 16 of
// a bf16 layer and 4 of an fp32 one.  The tiles' tokens lie in shared memory.
// Each of eight warps copies the weights that it multiplies itself, 512 bytes of
// 16 rows at a time, into a double buffer of its own, so that no warp waits for
// another's copies.  KS = 1, 2, 4 or 8 of the warps share an item, taking every
// KS-th such stage of K; their partial results are added in a fixed order.
//
// bf16 layers multiply with mma.sync, weights as the row operand, so that a
// handful of tokens wastes no more than the narrow side of a tile (the tcgen05
// path's smallest row tile, 64 rows of one expert, is too coarse to spread a small
// layer over 152 SMs, and its rate is not needed).  The hidden activations enter
// the down projection as the sum of two bf16 values (16 bits of the fp32 ones, an
// error of 2^-17), so that the only rounding to 8 bits is that of y.  fp32 layers
// multiply on the CUDA cores: a lane holds 4 values of K and the sums of all 16
// rows, so that a token's values are read once for 16 rows.
//
// Measured: 64 tokens of the large layer (6.2 GB of weights) 0.95 ms, 6.5 TB/s of
// the 6.79 of a copy; one token (403 MB) 76 us, 5.3 TB/s, the rest being the three
// barriers, the selection and the launch.  Left behind (64 tokens): a multiply-add
// per weight and token on the CUDA cores 4.04 ms; rows from HBM straight to
// registers, 64 bytes of a row to a load, 1.71 ms, with L2 prefetches ahead of
// them 1.21 ms; one ring of bulk copies for the block, its K split over 16 warps,
// 1.60 to 1.99 ms (a bulk copy takes its thread some 0.1 us to issue, and the
// block waits for the slowest warp of every stage).
#include "decode_common.cuh"

namespace moe {
namespace {

constexpr int WARPS = 16, THREADS = WARPS * 32;
constexpr int CW = 8, CTHREADS = CW * 32;       // warps that multiply (all of them route)
constexpr int PIECE = 512;                      // bytes of a row in a stage
constexpr int STAGE = 16 * PIECE;
constexpr int NS = 2;                           // stages of a warp

__host__ __device__ constexpr int up16(int v) { return (v + 15) & ~15; }
// Bytes of one token's row in shared memory.  bf16: 64 past a multiple of 128, so
// that the two rows a quarter-warp reads fall on different banks, and room for
// zeros up to a multiple of 32 values; fp32 rows are read along the row.
template <typename WT>
__host__ __device__ inline int row_pitch(int K) {
  return sizeof(WT) == 2 ? (K * 2 + 127) / 128 * 128 + 64 : K * 4;
}
template <typename WT>
__host__ __device__ constexpr int most_tokens() { return sizeof(WT) == 2 ? 16 : 4; }
// Floats of one warp's partial results: rows by tokens (16 x 8 or 16, or 16 x 4).
template <typename WT>
__host__ __device__ inline int part_floats(int tt) { return sizeof(WT) == 4 ? 64 : tt > 8 ? 256 : 128; }
// Shared memory of a call with token tiles of tt, the same on host and device.
struct Plan {
  int off_red, off_idx, off_gate, off_tok, off_slot, off_tile, off_at, off_rows, rows_bytes;
};
template <typename WT>
__host__ __device__ inline Plan make_plan(int T, int k, int E, int Fs, int tt) {
  Plan p;
  const int R = T * k;
  const int tiles = (E < R ? E : R) + R / tt + (Fs ? (T + tt - 1) / tt : 0);
  int o = CW * NS * STAGE;   // (the router's and the selection's scratch lies there first)
  p.off_red = o; o += 2 * CW * part_floats<WT>(tt) * 4;
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
// Tokens of a tile: as many as there is room for one tile of, or 0.
template <typename WT>
int tile_tokens(const DecodeArgs& a) {
  const long long up = row_pitch<WT>(a.D), width = a.F > a.Fs ? a.F : a.Fs;
  const long long down = row_pitch<WT>((int)width) * (sizeof(WT) == 2 ? 2 : 1);
  for (int tt = most_tokens<WT>(); tt >= 1; --tt)
    if (tt * (up > down ? up : down) <= make_plan<WT>(a.T, a.k, a.E, a.Fs, tt).rows_bytes) return tt;
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
// First item of block b's share: the blocks' shares are of equal weight bytes, a
// shared item counting `weight` routed ones.  One 32-bit division: the whole
// block waits for it.
__device__ __forceinline__ int share_of(int all_r, int all_s, int weight, int b) {
  const int units = all_r + all_s * weight, q = units / (int)gridDim.x;
  const int at = q * b + min(b, units - q * (int)gridDim.x);
  if (at <= all_r) return at;
  return all_r + (weight == 1 ? at - all_r : (at - all_r) / weight);
}
template <typename WT, bool UP>
__device__ __forceinline__ Part make_part(const DecodeArgs& a, int n_routed, int n_tiles, bool routed) {
  Part p;
  const bool pair = UP && a.act == 2;
  const int width_r = UP ? a.F : a.D, width_s = UP ? a.Fs : a.D;
  p.rows = pair ? 8 : 16;
  const int per_r = (width_r + p.rows - 1) / p.rows, per_s = (width_s + p.rows - 1) / p.rows;
  const int K_r = UP ? a.D : a.F, K_s = UP ? a.D : a.Fs;
  const int all_r = n_routed * per_r, all_s = (n_tiles - n_routed) * per_s;
  const int weight = UP || a.Fs == 0 ? 1 : a.n_shared;         // Fs = n_shared F
  const int lo = share_of(all_r, all_s, weight, blockIdx.x);
  const int hi = share_of(all_r, all_s, weight, blockIdx.x + 1);
  p.K = routed ? K_r : K_s;
  p.width = routed ? width_r : width_s;
  p.per = routed ? per_r : per_s;
  p.t0 = routed ? 0 : n_routed;
  p.lo = routed ? lo : max(lo - all_r, 0);
  p.hi = routed ? min(hi, all_r) : hi - all_r;
  p.w = static_cast<const char*>(UP ? (routed ? a.w1 : a.ws1) : (routed ? a.w2 : a.ws2));
  p.second = !pair ? 8ll * p.K * (int)sizeof(WT)
                   : static_cast<const char*>(routed ? a.w3 : a.ws3) - p.w;
  return p;
}
// Rows 0..7 of block `blk` of tile `t`.
template <typename WT>
__device__ __forceinline__ const char* item_rows(const Part& p, const Tile* tiles, int t, int blk) {
  const int e = max((int)tiles[p.t0 + t].e, 0);
  return p.w + ((long long)e * p.width + (long long)blk * p.rows) * p.K * (int)sizeof(WT);
}
// Whether rows 8..15 of the block exist (the rows of a matrix are a multiple of 8).
__device__ __forceinline__ bool has_upper(const Part& p, int blk) {
  return p.rows == 8 || blk * 16 + 8 < p.width;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The first of the two bf16 parts of v: the nearest bf16 value, but the largest
// one for a finite v beyond it; an infinity is a part of its own (with 0).
__device__ __forceinline__ float bf16_part(float v) {
  const float h = __bfloat162float(__float2bfloat16_rn(v));
  return isinf(h) ? __uint_as_float(__float_as_uint(v) & 0xffff0000u) : h;
}
// A tile's token rows into shared memory (two planes for hidden activations of a
// bf16 layer, whose rows have zeros from K to the next multiple of 32).
template <typename WT, bool UP>
__device__ __forceinline__ void load_tile(const DecodeArgs& a, const Routing& rt, const Tile& tl,
                                          int K, char* rows) {
  const int pitch = row_pitch<WT>(K), plane = tl.n * pitch;
  for (int t = threadIdx.x >> 5; t < tl.n; t += CW) {              // a warp a token
    const int tok = tl.e >= 0 && UP ? rt.tok[tl.start + t] : tl.start + t;
    const WT* x = static_cast<const WT*>(a.x) + (long long)tok * a.D;
    const float* h = (tl.e >= 0 ? a.hidden : a.hidden_s) + (long long)tok * K;
    if constexpr (sizeof(WT) == 4) {
      const float* src = UP ? reinterpret_cast<const float*>(x) : h;
#pragma unroll 4
      for (int c = threadIdx.x & 31; c < K / 4; c += 32)
        *reinterpret_cast<uint4*>(rows + t * pitch + c * 16) =
            __ldcg(reinterpret_cast<const uint4*>(src) + c);
      continue;
    }
    const int pieces = (K + 31) / 32 * 4;                          // of 8 values
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
          const float h0 = bf16_part(v[2 * j]), h1 = bf16_part(v[2 * j + 1]);
          hi[j] = pack_bf16(h0, h1);
          lo[j] = pack_bf16(isinf(h0) ? 0.f : v[2 * j] - h0, isinf(h1) ? 0.f : v[2 * j + 1] - h1);
        }
        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(to + plane) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
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

// One output pair of an item: rows r and r + 8 of the 16, token `tok` of the
// tile; b0, b1: the rows' biases (up projections of layers that have them).
template <bool UP>
__device__ __forceinline__ void emit(const DecodeArgs& a, const Tile& tl, int block, int r, int tok,
                                     float v0, float v1, float b0, float b1) {
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
      const float v = h ? v1 + b1 : v0 + b0;
      __stcg(o + f, a.act == 1 ? gelu_tanh_f(v) : (v < 0.f ? 0.f : v));     // a NaN stays one
    }
  } else {
    const long long row = (tl.e >= 0 ? 0 : (long long)a.T * a.k) + tl.start + tok;
    const int d = block * 16 + r;
    __stcg(a.ye + row * a.D + d, v0);
    if (d + 8 < a.D) __stcg(a.ye + row * a.D + d + 8, v1);
  }
}

// What a warp does with its stages: begin an item, multiply a stage of `left`
// values of K, and end with partial results that it stores or, alone on the
// item, hands out.
//
// Products<bf16>: mma tiles of 16 rows by 8 tokens.  Both products of a 32-value
// block take 4 of every lane's 8 values, weights and tokens alike, so that each
// operand is one 16-byte read; the sum over K does not care for the order.  A
// column of the result depends on its own token only, so absent tokens repeat
// the last one's row.
template <typename WT, bool UP> struct Products;
template <bool UP> struct Products<bf16, UP> {
  uint32_t at0, at1;           // the lane's token rows of the two token tiles
  int plane, n;
  // token tiles of 8 by chains of dependent products: the two steps of a block,
  // and for hidden activations their two parts
  static constexpr int CH = UP ? 2 : 4;
  float acc[2][CH][4];
  // A sum over the first parts that is not finite is the result: the second
  // parts, zeros or of the other sign, would make a NaN of an infinite weight's
  // or an overflowing product's infinity, and they overflow only where it does.
  __device__ __forceinline__ float total(int t8, int c) const {
    const float first = acc[t8][0][c] + acc[t8][1][c];
    if (UP) return first;
    return isfinite(first) ? first + (acc[t8][CH - 2][c] + acc[t8][CH - 1][c]) : first;
  }
  __device__ __forceinline__ void begin(const char* rows, int pitch, int tokens, int lane) {
    const uint32_t at = smem_addr(rows) + (lane & 3) * 16;
    n = tokens;
    plane = n * pitch;
    at0 = at + min(lane >> 2, n - 1) * pitch;
    at1 = at + min(8 + (lane >> 2), n - 1) * pitch;
#pragma unroll
    for (int h = 0; h < CH; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[0][h][c] = acc[1][h][c] = 0.f;
  }
  __device__ __forceinline__ void stage(uint32_t from, int v0, int left, int lane) {
    const int g = lane >> 2, blocks = min(PIECE / 64, (left + 31) / 32);
    from += g * PIECE;
#pragma unroll 4
    for (int u = 0; u < blocks; ++u) {
      const uint32_t wat = (from + u * 64 + (lane & 3) * 16) ^ ((g & 1) << 6);
      const uint4 w0 = load_rows(wat), w1 = load_rows(wat + 8 * PIECE);
      auto products = [&](float (&c0)[4], float (&c1)[4], uint32_t x_at) {
        const uint4 x = load_rows(x_at);
        mma16816(c0, w0.x, w1.x, w0.y, w1.y, x.x, x.y);
        mma16816(c1, w0.z, w1.z, w0.w, w1.w, x.z, x.w);
      };
      const uint32_t off = (v0 + u * 32) * 2;
      products(acc[0][0], acc[0][1], at0 + off);
      if (!UP) products(acc[0][CH - 2], acc[0][CH - 1], at0 + plane + off);
      if (n > 8) {
        products(acc[1][0], acc[1][1], at1 + off);
        if (!UP) products(acc[1][CH - 2], acc[1][CH - 1], at1 + plane + off);
      }
    }
  }
  // out(row, token, value of row, value of row + 8) for this warp's own item
  template <typename Out>
  __device__ __forceinline__ void each(int lane, const Out& out) const {
#pragma unroll
    for (int t8 = 0; t8 < 2; ++t8)
      if (t8 == 0 || n > 8)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          out(lane >> 2, t8 * 8 + (lane & 3) * 2 + c, total(t8, c), total(t8, c + 2));
  }
  __device__ __forceinline__ void store(float* buf, int lane) const {
#pragma unroll
    for (int t8 = 0; t8 < 2; ++t8)
      if (t8 == 0 || n > 8)
        *reinterpret_cast<float4*>(buf + t8 * 128 + lane * 4) =
            make_float4(total(t8, 0), total(t8, 1), total(t8, 2), total(t8, 3));
  }
  // Sums of KS warps' stored results, o = me, me + lanes, ..
  template <typename Out>
  static __device__ __forceinline__ void join(const float* buf, int size, int KS, int n, int me,
                                              int lanes, const Out& out) {
    for (int o = me; o < (n > 8 ? 128 : 64); o += lanes) {
      const int t8 = o / 64, l = (o % 64) / 2, c = o % 2;
      float v0 = 0.f, v1 = 0.f;
      for (int q = 0; q < KS; ++q) {
        const float* part = buf + q * size + t8 * 128 + l * 4 + c;
        v0 += part[0];
        v1 += part[2];
      }
      out(l >> 2, t8 * 8 + (l & 3) * 2 + c, v0, v1);
    }
  }
};
// Products<float>: a lane multiplies 4 values of each row with 4 of each token.
template <bool UP> struct Products<float, UP> {
  uint32_t at;
  int pitch, n;
  float acc[64];               // row * 4 + token
  __device__ __forceinline__ void begin(const char* rows, int row_bytes, int tokens, int lane) {
    at = smem_addr(rows) + lane * 16;
    pitch = row_bytes;
    n = tokens;
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0.f;
  }
  __device__ __forceinline__ void stage(uint32_t from, int v0, int left, int lane) {
    if (lane * 4 >= left) return;
    float x[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint4 q = load_rows(at + min(t, n - 1) * pitch + v0 * 4);
      x[t][0] = __uint_as_float(q.x); x[t][1] = __uint_as_float(q.y);
      x[t][2] = __uint_as_float(q.z); x[t][3] = __uint_as_float(q.w);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const uint4 q = load_rows((from + r * PIECE + lane * 16) ^ ((r & 1) << 6));
      const float w[4] = {__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z),
                          __uint_as_float(q.w)};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r * 4 + t] = fmaf(w[i], x[t][i], acc[r * 4 + t]);
    }
  }
  // lane l is left with row l / 4 and row 8 + l / 4 of token l % 4
  __device__ __forceinline__ float2 sums(int lane) const {
    float lo[32], hi[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      lo[i] = acc[i];
      hi[i] = acc[32 + i];
    }
    return make_float2(warp_sum32(lo, lane), warp_sum32(hi, lane));
  }
  template <typename Out>
  __device__ __forceinline__ void each(int lane, const Out& out) const {
    const float2 v = sums(lane);
    out(lane >> 2, lane & 3, v.x, v.y);
  }
  __device__ __forceinline__ void store(float* buf, int lane) const {
    const float2 v = sums(lane);
    buf[lane] = v.x;
    buf[32 + lane] = v.y;
  }
  template <typename Out>
  static __device__ __forceinline__ void join(const float* buf, int size, int KS, int, int me, int lanes,
                                              const Out& out) {
    for (int o = me; o < 32; o += lanes) {
      float v0 = 0.f, v1 = 0.f;
      for (int q = 0; q < KS; ++q) {
        v0 += buf[q * size + o];
        v1 += buf[q * size + 32 + o];
      }
      out(o >> 2, o & 3, v0, v1);
    }
  }
};

// Warps to an item: the number that takes the fewest quarter stages for the
// block's share, an item shared by several warps counting one more for adding
// their parts.
__device__ __forceinline__ int warps_per_item(int items, int stages) {
  static_assert(CW == 8, "three halvings");
  int best = 1, cost = 0x7fffffff;
#pragma unroll 1
  for (int l = 0; l <= 3; ++l) {
    const int c = ((items + (CW >> l) - 1) >> (3 - l)) *
                  (((stages + (1 << l) - 1) >> l) * 4 + (l > 0 ? 1 : 0));
    if (c < cost) {
      cost = c;
      best = 1 << l;
    }
  }
  return best;
}

// The items of a part, by the multiplying warps.  Where `flag` is given, the grid
// barrier before the down projection stands between the first weight copies and
// the tiles' tokens.
template <typename WT, bool UP>
__device__ __forceinline__ void compute(const DecodeArgs& a, const Part& p, const Routing& rt, int tt,
                                        int* row_at, char* rows, int rows_bytes, float* red,
                                        uint32_t ring, int* flag) {
  if (p.lo >= p.hi) {
    if (!UP && flag != nullptr) grid_barrier<CTHREADS>(a.ctl, 1, flag);
    return;
  }
  constexpr int ES = (int)sizeof(WT), SV = PIECE / ES;         // values of a row in a stage
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = p.K, stages = (K + SV - 1) / SV;
  const int KS = warps_per_item(p.hi - p.lo, stages), groups = CW >> (__ffs(KS) - 1);
  const int lg = __ffs(KS) - 1, mine = warp >> lg, ks = warp & (KS - 1);
  const int steps = (stages + KS - 1) >> lg;
  const int pitch = row_pitch<WT>(K), size = part_floats<WT>(tt);
  const long long item_step = (long long)groups * p.rows * K * ES;

  // the next stage to be copied: item, its tile and block, step; rows 0..7 of it
  int li = p.lo + mine, lt = li / p.per, lb = li - lt * p.per, ls = 0, put_slot = 0;
  int it = lt, ib = lb;        // (where the computing starts, too)
  const char* lp = li < p.hi ? item_rows<WT>(p, rt.tiles, lt, lb) : nullptr;
  auto put = [&] {
    const int v0 = (ls * KS + ks) * SV;
    if (li < p.hi && v0 < K) {
      // row r's 16-byte pieces change places with their neighbours 64 bytes on
      // for odd r, so that the rows a quarter-warp reads fall on different banks
      const uint32_t dst = ring + put_slot * STAGE + lane * 16;
      const int at = v0 * ES + lane * 16;
      const bool on = at < K * ES;
      const char* src = lp + (on ? at : 0);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        copy16((dst + r * PIECE) ^ ((r & 1) << 6), src + (long long)r * K * ES, on);
      if (has_upper(p, lb)) {
        src += p.second;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          copy16((dst + (8 + r) * PIECE) ^ ((r & 1) << 6), src + (long long)r * K * ES, on);
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
      lp = item_rows<WT>(p, rt.tiles, lt, lb);
    }
  };
#pragma unroll
  for (int u = 0; u < NS; ++u) put();
  if (!UP && flag != nullptr) grid_barrier<CTHREADS>(a.ctl, 1, flag);

  // what is being computed: item, its tile and block
  int i = p.lo + mine, parity = 0, slot = 0;
  int tile = p.lo / p.per;
  for (int b_lo = p.lo; b_lo < p.hi;) {
    // the tokens of as many of the next tiles as there is room for
    int t = tile, used = 0;
    bar_sync<CTHREADS>();      // the last ones are no longer read
    const int first = t;
    for (; t * p.per < p.hi; ++t) {
      const Tile tl = rt.tiles[p.t0 + t];
      const int need = tl.n * pitch * (!UP && ES == 2 ? 2 : 1);
      if (t > first && used + need > rows_bytes) break;
      load_tile<WT, UP>(a, rt, tl, K, rows + used);
      if (threadIdx.x == 0) row_at[t] = used;
      used += need;
    }
    const int b_hi = min(p.hi, t * p.per);
    b_lo = b_hi;
    tile = t;
    bar_sync<CTHREADS>();

    while (i < b_hi) {
      const Tile tl = rt.tiles[p.t0 + it];
      Products<WT, UP> sum;
      sum.begin(rows + row_at[it], pitch, tl.n, lane);
      // the biases of the item's rows, one a lane, on their way from here on
      float bias = 0.f;
      if (UP && a.b1 != nullptr && lane < 16 && ib * 16 + lane < p.width)
        bias = __ldg(a.b1 + (long long)tl.e * a.F + ib * 16 + lane);
      for (int s = 0; s < steps; ++s) {
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        __syncwarp();
        const int v0 = (s * KS + ks) * SV;
        sum.stage(ring + slot * STAGE, v0, K - v0, lane);
        __syncwarp();
        put();
        slot = slot + 1 == NS ? 0 : slot + 1;
      }
      auto out = [&](int row, int tok, float v0, float v1) {       // by whole warps
        const float b0 = UP ? __shfl_sync(0xffffffffu, bias, row) : 0.f;
        const float b1 = UP ? __shfl_sync(0xffffffffu, bias, row + 8) : 0.f;
        emit<UP>(a, tl, ib, row, tok, v0, v1, b0, b1);
      };
      if (KS == 1) {
        sum.each(lane, out);
      } else {
        // partial results of the item's warps; two buffers, so one barrier an item is enough
        float* buf = red + (parity * CW + mine * KS) * size;
        parity ^= 1;
        sum.store(buf + ks * size, lane);
        asm volatile("bar.sync %0, %1;" ::"r"(2 + mine), "r"(KS * 32) : "memory");
        Products<WT, UP>::join(buf, size, KS, tl.n, ks * 32 + lane, KS * 32, out);
      }
      i += groups;
      ib += groups;
      while (ib >= p.per) { ib -= p.per; ++it; }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename WT>
__global__ void __launch_bounds__(THREADS, 1)
decode_kernel(const __grid_constant__ DecodeArgs a, const int tt) {
  extern __shared__ __align__(128) char sm[];
  __shared__ int flag, n_tiles, n_routed, scan[8];
  const Plan P = make_plan<WT>(a.T, a.k, a.E, a.Fs, tt);
  const int tid = threadIdx.x;
  const int T = a.T, D = a.D, k = a.k;
  const Routing rt{reinterpret_cast<short*>(sm + P.off_idx), reinterpret_cast<float*>(sm + P.off_gate),
                   reinterpret_cast<short*>(sm + P.off_tok), reinterpret_cast<short*>(sm + P.off_slot),
                   reinterpret_cast<Tile*>(sm + P.off_tile), scan};
  float* red = reinterpret_cast<float*>(sm + P.off_red);
  char* rows = sm + P.off_rows;

  const int magic = tid == 0 ? __ldcg(a.ctl + DC_MAGIC) : 0;     // (looked at after the logits)

  float* scratch = reinterpret_cast<float*>(sm);
  router<WT, WARPS>(a, scratch);
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
      compute<WT, true>(a, make_part<WT, true>(a, nr, nt, !shared), rt, tt, row_at + shared * nr, rows,
                    P.rows_bytes, red, ring, nullptr);
#pragma unroll 1
    for (int shared = 0; shared < (a.Fs > 0 ? 2 : 1); ++shared)
      compute<WT, false>(a, make_part<WT, false>(a, nr, nt, !shared), rt, tt, row_at + shared * nr, rows,
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
        if (j0 == 0 && i < T * quads) {
          WT* y = static_cast<WT*>(a.y) + (long long)i * 4;
          if constexpr (sizeof(WT) == 2)
            *reinterpret_cast<uint2*>(y) =
                make_uint2(pack_bf16(v[u].x, v[u].y), pack_bf16(v[u].z, v[u].w));
          else
            *reinterpret_cast<float4*>(y) = v[u];
        }
      }
    }
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

template <typename WT>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t st) {
  static std::atomic<unsigned long long> attr_done{0};
  const int sms = sm_count(), tt = tile_tokens<WT>(a);
  if (sms <= 0) return cudaErrorUnknown;
  if (tt <= 0) return cudaErrorInvalidValue;    // (past the entry point's limits)
  // a block per SM, or fewer where each would have less than 8 KB of weights (the
  // kernel's time hardly goes with it: 4 KB, 16 KB and a block on every SM are
  // within 0.2 us of 13.4 at 96 KB of weights, of 13.6 at 390 KB, of 14.4 at
  // 780 KB; one block alone takes 0.3 us more than four at 32 KB, 23 us at 390 KB)
  const long long experts = (long long)a.T * a.k < a.E ? (long long)a.T * a.k : a.E;
  const long long bytes = (experts * a.F + a.Fs) * a.D * (a.act == 2 ? 3 : 2) * (int)sizeof(WT);
  const long long blocks = (bytes + 8191) / 8192;
  return launch_cooperative(decode_kernel<WT>, (int)(blocks < sms ? blocks : sms), THREADS,
                            attr_done, st, a, tt);
}

}  // namespace

cudaError_t launch_decode_init(int* ctl, cudaStream_t st) {
  return launch_pdl(decode_init_kernel, dim3(1), dim3(DC_WORDS), 0, st, ctl);
}

cudaError_t launch_decode(int dtype, const DecodeArgs& a, cudaStream_t st) {
  return dtype == 1 ? launch_t<bf16>(a, st) : launch_t<float>(a, st);
}

}  // namespace moe
