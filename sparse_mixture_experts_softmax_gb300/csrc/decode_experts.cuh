// The expert products of the few-token kernels: items of 16 weight rows, streamed
// through per-warp buffers and multiplied with a tile of tokens (decode.cu has the
// why and the measurements).  Weights are fp32, bf16 or 4-bit ones.
#pragma once

#include "decode_common.cuh"
#include "q4.cuh"

namespace moe {
namespace {

constexpr int WARPS = 16, THREADS = WARPS * 32;

// How a kind of weights is stored: the type of the tokens that it multiplies, the
// bytes of a row's part in a stage (PIECE) and its values, and the bytes of a whole row;
// CW: the warps that multiply (all of them route), NS: the stages of a warp.
// The tokens' rows have zeros up to a multiple of BLOCK values, which is what a lane
// group of the products takes at once.
struct Q4 {};                                   // 4-bit weights (q4.cuh)
struct Q4Eight {};                              // the same, in tiles of at most eight tokens
struct Q4Few {};                                // the same, of a call of at most four tokens
struct Q4Wide {};                               // the same, with room for wide rows
template <typename WT> struct Stored;
template <> struct Stored<float> {
  typedef float Act;
  static constexpr int PIECE = 512, VALUES = 128, STAGE = 16 * PIECE, BLOCK = 1, CW = 8, NS = 2;
  static __host__ __device__ __forceinline__ int row(int K) { return K * 4; }
};
template <> struct Stored<bf16> {
  typedef bf16 Act;
  static constexpr int PIECE = 512, VALUES = 256, STAGE = 16 * PIECE, BLOCK = 32, CW = 8, NS = 2;
  static __host__ __device__ __forceinline__ int row(int K) { return K * 2; }
};
// A stage of 4-bit weights ends with its scales: for each of up to 16 groups (of 32
// inputs), those of the 16 rows.  Widening them takes more than eight warps (one token of
// the large layer 61 us with eight and 53 with sixteen, before the later steps).
template <> struct Stored<Q4> {
  typedef bf16 Act;
  static constexpr int PIECE = 256, VALUES = 512, STAGE = 16 * PIECE + VALUES / 32 * 32, BLOCK = 128,
                       CW = 16, NS = 2;
  static __host__ __device__ __forceinline__ int row(int K) { return K / 2; }
};
template <> struct Stored<Q4Eight> : Stored<Q4> {};
template <> struct Stored<Q4Few> : Stored<Q4> {};
// Half the warps: 80 KB less of buffers and partial results, for calls whose lists leave
// the other forms no room for a row.
template <> struct Stored<Q4Wide> : Stored<Q4> {
  static constexpr int CW = 8;
};
template <typename WT> constexpr bool kBf16Tokens = sizeof(typename Stored<WT>::Act) == 2;
template <typename WT> constexpr bool kQ4 = Stored<WT>::BLOCK == 128;
template <typename WT> constexpr int kCThreads = Stored<WT>::CW * 32;

__host__ __device__ constexpr int up16(int v) { return (v + 15) & ~15; }
// Bytes of one token's row in shared memory.  bf16: 64 past a multiple of 128, so
// that the two rows a quarter-warp reads fall on different banks, and room for
// zeros up to a multiple of BLOCK values; fp32 rows are read along the row.
template <typename WT>
__host__ __device__ constexpr int row_pitch(int K) {
  constexpr int B = Stored<WT>::BLOCK * 2 > 128 ? Stored<WT>::BLOCK * 2 : 128;
  return kBf16Tokens<WT> ? (K * 2 + B - 1) / B * B + 64 : K * 4;
}
template <typename WT>
__host__ __device__ constexpr int most_tokens() { return kBf16Tokens<WT> ? 16 : 4; }
template <> __host__ __device__ constexpr int most_tokens<Q4Eight>() { return 8; }
template <> __host__ __device__ constexpr int most_tokens<Q4Few>() { return 4; }
template <> __host__ __device__ constexpr int most_tokens<Q4Wide>() { return 8; }
// Floats of one warp's partial results: rows by tokens (16 x 8 or 16, or 16 x 4).
template <typename WT>
__host__ __device__ constexpr int part_floats(int tt) { return !kBf16Tokens<WT> ? 64 : tt > 8 ? 256 : 128; }
// Shared memory of a call with token tiles of tt, the same on host and device.
struct Plan {
  int off_red, off_idx, off_gate, off_tok, off_slot, off_tile, off_at, off_rows, rows_bytes;
};
template <typename WT>
__host__ __device__ constexpr Plan make_plan(int T, int k, int E, int Fs, int tt) {
  Plan p{};
  const int R = T * k;
  const int tiles = (E < R ? E : R) + R / tt + (Fs ? (T + tt - 1) / tt : 0);
  // (the router's and the selection's scratch lies there first)
  int o = Stored<WT>::CW * Stored<WT>::NS * Stored<WT>::STAGE;
  p.off_red = o; o += 2 * Stored<WT>::CW * part_floats<WT>(tt) * 4;
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
static_assert((768 + WARPS * 256) * 4 <= Stored<Q4Wide>::CW * Stored<Q4Wide>::NS * Stored<Q4Wide>::STAGE,
              "scratch");
// Bytes of one token's widest row of an operand.
template <typename WT>
__host__ __device__ constexpr long long row_bytes(int D, int width) {
  const long long up = row_pitch<WT>(D), down = (long long)row_pitch<WT>(width) * (kBf16Tokens<WT> ? 2 : 1);
  return up > down ? up : down;
}
// Tokens of a tile: as many as there is room for one tile of, or 0.
template <typename WT>
int tile_tokens(const DecodeArgs& a) {
  const long long row = row_bytes<WT>(a.D, a.F > a.Fs ? a.F : a.Fs);
  for (int tt = most_tokens<WT>(); tt >= 1; --tt)
    if (tt * row <= make_plan<WT>(a.T, a.k, a.E, a.Fs, tt).rows_bytes) return tt;
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
  const char* s;               // 4-bit weights: its scales, the bytes between those of
  long long second_s;          //   an item's two halves,
  int groups, log_g;           //   groups of a row, log2 of a group's inputs
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
  p.second = !pair ? 8ll * Stored<WT>::row(p.K) : static_cast<const char*>(routed ? a.w3 : a.ws3) - p.w;
  if constexpr (kQ4<WT>) {
    p.s = static_cast<const char*>(UP ? (routed ? a.s1 : a.ss1) : (routed ? a.s2 : a.ss2));
    p.second_s = !pair ? 16 : static_cast<const char*>(routed ? a.s3 : a.ss3) - p.s;
    p.log_g = a.log_g;
    p.groups = (p.K + (1 << a.log_g) - 1) >> a.log_g;
  }
  return p;
}
// Rows 0..7 of block `blk` of tile `t`: their weights, and the first group's scales.
template <typename WT>
__device__ __forceinline__ const char* item_rows(const Part& p, const Tile* tiles, int t, int blk) {
  const int e = max((int)tiles[p.t0 + t].e, 0);
  return p.w + ((long long)e * p.width + (long long)blk * p.rows) * Stored<WT>::row(p.K);
}
__device__ __forceinline__ const char* item_scales(const Part& p, const Tile* tiles, int t, int blk) {
  const int e = max((int)tiles[p.t0 + t].e, 0);
  return p.s + ((long long)e * p.groups * p.width + (long long)blk * p.rows) * 2;
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
// Warps to a token's row, as a power of two: all of them for one token, whose row is
// then one round of loads or two.
template <int CW>
__device__ __forceinline__ int warps_a_token(int n) {
  return max(31 - __clz(CW) - (32 - __clz(n - 1)), 0);
}
// A tile's token rows into shared memory (two planes for hidden activations of a
// bf16 layer, whose rows have zeros from K to the next multiple of BLOCK).  Beside
// 4-bit weights, of which a lane reads four words at once, the 16-byte pieces of 128
// values change places, 4 c + j with c + 4 j: the j-th words' inputs of a lane group
// lie next to one another.
template <typename WT, bool UP>
__device__ __forceinline__ void load_tile(const DecodeArgs& a, const Routing& rt, const Tile& tl,
                                          int K, char* rows) {
  typedef typename Stored<WT>::Act Act;
  constexpr int BLOCK = Stored<WT>::BLOCK;
  const int pitch = row_pitch<WT>(K), plane = tl.n * pitch;
  const int lg = warps_a_token<Stored<WT>::CW>(tl.n);
  const int c0 = threadIdx.x & ((32 << lg) - 1), step = 32 << lg;
  for (int t = threadIdx.x >> 5 >> lg; t < tl.n; t += Stored<WT>::CW >> lg) {
    const int tok = tl.e >= 0 && UP ? rt.tok[tl.start + t] : tl.start + t;
    const Act* x = static_cast<const Act*>(a.x) + (long long)tok * a.D;
    const float* h = (tl.e >= 0 ? a.hidden : a.hidden_s) + (long long)tok * K;
    if constexpr (!kBf16Tokens<WT>) {
      const float* src = UP ? reinterpret_cast<const float*>(x) : h;
#pragma unroll 4
      for (int c = c0; c < K / 4; c += step)
        *reinterpret_cast<uint4*>(rows + t * pitch + c * 16) =
            __ldcg(reinterpret_cast<const uint4*>(src) + c);
      continue;
    }
    const int pieces = (K + BLOCK - 1) / BLOCK * (BLOCK / 8);      // of 8 values
#pragma unroll 4
    for (int c = c0; c < pieces; c += step) {
      const int at = kQ4<WT> ? (c & ~15) | (c & 3) << 2 | (c >> 2 & 3) : c;
      char* to = rows + t * pitch + at * 16;
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
// 16 bytes of each of four rows, two rows of a stage of 256-byte pieces apart, where on.
__device__ __forceinline__ void copy16_rows(uint32_t dst, const char* src, long long two_rows, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\tadd.s64 a, %1, %2;\n\t"
      "@p cp.async.cg.shared.global [%0+512], [a], 16;\n\tadd.s64 a, a, %2;\n\t"
      "@p cp.async.cg.shared.global [%0+1024], [a], 16;\n\tadd.s64 a, a, %2;\n\t"
      "@p cp.async.cg.shared.global [%0+1536], [a], 16;\n\t}" ::"r"(dst), "l"(src), "l"(two_rows),
      "r"((int)on)
      : "memory");
}
// 16 bytes, or zeros, where on.
__device__ __forceinline__ void copy16_or0(uint32_t dst, const char* src, bool there, bool on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16, %2;\n\t}" ::"r"(dst), "l"(src), "r"(there ? 16 : 0),
      "r"((int)on)
      : "memory");
}
__device__ __forceinline__ uint4 load_rows(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t load_scale(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
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
// MmaProducts: mma tiles of 16 rows by 8 tokens.  With bf16 weights both products of a
// 32-value block take 4 of every lane's 8 values, weights and tokens alike, so that each
// operand is one 16-byte read; the sum over K does not care for the order.  A
// column of the result depends on its own token only, so absent tokens repeat
// the last one's row.  FEW: of up to four tokens' hidden activations, the first parts are
// columns 0 to 3 of the one tile and the second parts columns 4 to 7: half the products and
// reads (one token of the large layer 45 -> 41 us).
template <typename WT, bool UP> struct Products;
template <bool UP, bool Q4W, int MOST> struct MmaProducts {
  static constexpr bool FEW = MOST <= 4;
  uint32_t at0, at1;           // the lane's token rows of the two token tiles
  int plane, n;
  // token tiles of 8 by chains of dependent products: the two steps of a block,
  // and for hidden activations their two parts
  static constexpr int T8 = MOST > 8 ? 2 : 1, CH = UP || FEW ? 2 : 4;
  float acc[T8][CH][4];
  // A sum over the first parts that is not finite is the result: the second
  // parts, zeros or of the other sign, would make a NaN of an infinite weight's
  // or an overflowing product's infinity, and they overflow only where it does.
  __device__ __forceinline__ float total(int t8, int c) const {
    const float first = acc[t8][0][c] + acc[t8][1][c];
    const float second = UP ? 0.f : FEW ? __shfl_xor_sync(0xffffffffu, first, 2)
                                        : acc[t8][CH - 2][c] + acc[t8][CH - 1][c];
    const float sum = UP || !isfinite(first) ? first : first + second;
    return Q4W ? Q4_UNSCALE * sum : sum;
  }
  __device__ __forceinline__ void begin(const Part&, const char* rows, int pitch, int tokens, int lane) {
    const uint32_t at = smem_addr(rows) + (lane & 3) * 16;
    n = tokens;
    plane = n * pitch;
    at0 = at + min(FEW && !UP ? lane >> 2 & 3 : lane >> 2, n - 1) * pitch +
          (FEW && !UP && lane >= 16 ? plane : 0);
    at1 = at + min(8 + (lane >> 2), n - 1) * pitch;
#pragma unroll
    for (int t = 0; t < T8; ++t)
#pragma unroll
      for (int h = 0; h < CH; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[t][h][c] = 0.f;
  }
  // out(row, token, value of row, value of row + 8) for this warp's own item
  template <typename Out>
  __device__ __forceinline__ void each(int lane, const Out& out) const {
#pragma unroll
    for (int t8 = 0; t8 < T8; ++t8)
      if (t8 == 0 || n > 8)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          out(lane >> 2, t8 * 8 + (lane & 3) * 2 + c, total(t8, c), total(t8, c + 2));
  }
  __device__ __forceinline__ void store(float* buf, int lane) const {
#pragma unroll
    for (int t8 = 0; t8 < T8; ++t8)
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
template <bool UP> struct Products<bf16, UP> : MmaProducts<UP, false, most_tokens<bf16>()> {
  static constexpr int PIECE = Stored<bf16>::PIECE;
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
      products(this->acc[0][0], this->acc[0][1], this->at0 + off);
      if (!UP) products(this->acc[0][this->CH - 2], this->acc[0][this->CH - 1], this->at0 + this->plane + off);
      if (this->n > 8) {
        products(this->acc[1][0], this->acc[1][1], this->at1 + off);
        if (!UP) products(this->acc[1][this->CH - 2], this->acc[1][this->CH - 1], this->at1 + this->plane + off);
      }
    }
  }
};
// 4-bit weights: a lane reads 32 inputs' codes of its two rows at once, in which the
// scale does not change, and multiplies word by word.  The four lanes of a row take
// 128 inputs in turn, lane c words 4 c to 4 c + 3.
template <bool UP, int MOST> struct Q4Products : MmaProducts<UP, true, MOST> {
  static constexpr bool FEW = MOST <= 4;
  static constexpr int T8 = MOST > 8 ? 2 : 1;
  static constexpr int PIECE = Stored<Q4>::PIECE;
  static_assert(PIECE == 256, "four blocks of 128 inputs");
  uint32_t code_at, scale_at, scale_step;      // the lane's, in a stage; from one block to the next
  __device__ __forceinline__ void begin(const Part& p, const char* rows, int pitch, int tokens, int lane) {
    MmaProducts<UP, true, MOST>::begin(p, rows, pitch, tokens, lane);
    const int g = lane >> 2, c = lane & 3;
    code_at = g * PIECE + ((c * 16) ^ ((g & 1) << 6));
    scale_at = 16 * PIECE + g * 2 + (c * 32 >> p.log_g) * 32;
    scale_step = 128 * 32 >> p.log_g;
  }
  template <bool FAST, int TT>
  __device__ __forceinline__ void block(uint32_t codes, uint32_t scales, const uint32_t (&x)[2], bool on) {
    const uint4 w0 = load_rows(codes), w1 = load_rows(codes + 8 * PIECE);
    uint4 r[2][4];
    q4_runs<FAST>(w0, w1, on ? load_scale(scales) : 0u, on ? load_scale(scales + 16) : 0u, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 a = r[0][j], b = r[1][j];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int h = 0; h < (UP || FEW ? 1 : 2); ++h) {
          const uint4 v = load_rows(x[t] + (h ? this->plane : 0) + j * 64);
          mma16816(this->acc[t][2 * h], a.x, b.x, a.y, b.y, v.x, v.y);
          mma16816(this->acc[t][2 * h + 1], a.z, b.z, a.w, b.w, v.z, v.w);
        }
    }
  }
  // Past a row's end lie codes of any value, which meet zeros of x.  Where their group's scale
  // may be an infinity or a NaN (never the short way's) it is taken as a zero there.
  template <bool FAST, int TT>
  __device__ __forceinline__ void blocks(uint32_t from, int v0, int end, int left, int lane) {
    uint32_t x[2] = {this->at0 + v0 * 2, this->at1 + v0 * 2};
    uint32_t scales = from + scale_at;
    const uint32_t codes = from + code_at;       // (a stage starts at a multiple of 256 bytes)
#pragma unroll 1
    for (int u = 0; u < end; u += 64) {
      block<FAST, TT>(codes ^ u, scales, x, FAST || u * 2 + (lane & 3) * 32 < left);
      scales += scale_step;
      x[0] += 256;
      x[1] += 256;
    }
  }
  // (whether all of the stage's scales take the fast way is looked at once)
  __device__ __forceinline__ void stage(uint32_t from, int v0, int left, int lane) {
    const int end = min(PIECE, (left + 127) / 128 * 64);
    uint32_t ok = 0x80008000u;
    if (lane < (int)(scale_step >> 2)) {         // (a stage's groups are scale_step / 8, of 32 bytes)
      const uint4 s = load_rows(from + 16 * PIECE + lane * 16);
      ok &= q4_fast(s.x) & q4_fast(s.y) & q4_fast(s.z) & q4_fast(s.w);
    }
    if (__all_sync(0xffffffffu, ok == 0x80008000u)) {
      if (T8 > 1 && this->n > 8) blocks<true, T8>(from, v0, end, left, lane);
      else blocks<true, 1>(from, v0, end, left, lane);
    } else {
      blocks<false, T8>(from, v0, end, left, lane);
    }
  }
};
template <bool UP> struct Products<Q4, UP> : Q4Products<UP, most_tokens<Q4>()> {};
template <bool UP> struct Products<Q4Eight, UP> : Q4Products<UP, most_tokens<Q4Eight>()> {};
template <bool UP> struct Products<Q4Few, UP> : Q4Products<UP, most_tokens<Q4Few>()> {};
template <bool UP> struct Products<Q4Wide, UP> : Q4Products<UP, most_tokens<Q4Wide>()> {};
// Products<float>: a lane multiplies 4 values of each row with 4 of each token.
template <bool UP> struct Products<float, UP> {
  uint32_t at;
  int pitch, n;
  float acc[64];               // row * 4 + token
  __device__ __forceinline__ void begin(const Part&, const char* rows, int row_bytes, int tokens, int lane) {
    at = smem_addr(rows) + lane * 16;
    pitch = row_bytes;
    n = tokens;
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0.f;
  }
  static constexpr int PIECE = Stored<float>::PIECE;
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
template <int CW>
__device__ __forceinline__ int warps_per_item(int items, int stages) {
  static_assert(CW == 8 || CW == 16, "halvings");
  constexpr int L = CW == 8 ? 3 : 4;
  int best = 1, cost = 0x7fffffff;
#pragma unroll 1
  for (int l = 0; l <= L; ++l) {
    const int c = ((items + (CW >> l) - 1) >> (L - l)) *
                  (((stages + (1 << l) - 1) >> l) * 4 + (l > 0 ? 1 : 0));
    if (c < cost) {
      cost = c;
      best = 1 << l;
    }
  }
  return best;
}

// The layer's own tokens and results: routed tiles and the shared branch's.  Where `flag`
// is given, the grid barrier before the down projection stands between the first weight
// copies and the tiles' tokens.
template <typename WT, bool UP> struct LayerJob {
  const DecodeArgs& a;
  const Routing& rt;
  int* flag;
  __device__ __forceinline__ void wait_tokens() const {
    if (!UP && flag != nullptr) grid_barrier<kCThreads<WT>>(a.ctl, 1, flag);
  }
  __device__ __forceinline__ void load(const Tile& tl, int K, char* rows) const {
    load_tile<WT, UP>(a, rt, tl, K, rows);
  }
  // the bias of row `lane` of an item
  __device__ __forceinline__ float bias(const Part& p, const Tile& tl, int block, int lane) const {
    float b = 0.f;
    if (UP && a.b1 != nullptr && lane < 16 && block * 16 + lane < p.width)
      b = __ldg(a.b1 + (long long)tl.e * a.F + block * 16 + lane);
    return b;
  }
  __device__ __forceinline__ void out(const Part&, const Tile& tl, int block, int row, int tok, float v0,
                                      float v1, float b0, float b1) const {
    emit<UP>(a, tl, block, row, tok, v0, v1, b0, b1);
  }
};

// The items of a part, by the multiplying warps.
template <typename WT, bool UP, typename Job>
__device__ __forceinline__ void compute(const Job& job, const Part& p, const Tile* tiles, int tt,
                                        int* row_at, char* rows, int rows_bytes, float* red,
                                        uint32_t ring) {
  if (p.lo >= p.hi) {
    job.wait_tokens();
    return;
  }
  constexpr int CW = Stored<WT>::CW, NS = Stored<WT>::NS, CTHREADS = kCThreads<WT>;
  constexpr int PIECE = Stored<WT>::PIECE, STAGE = Stored<WT>::STAGE;
  constexpr int SV = Stored<WT>::VALUES;                       // values of a row in a stage
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = p.K, stages = (K + SV - 1) / SV;
  const int KS = warps_per_item<CW>(p.hi - p.lo, stages), groups = CW >> (__ffs(KS) - 1);
  const int lg = __ffs(KS) - 1, mine = warp >> lg, ks = warp & (KS - 1);
  const int steps = (stages + KS - 1) >> lg;
  const int pitch = row_pitch<WT>(K), size = part_floats<WT>(tt);
  const int row = Stored<WT>::row(K);
  const long long item_step = (long long)groups * p.rows * row;

  // the next stage to be copied: item, its tile and block, step; rows 0..7 of it
  int li = p.lo + mine, lt = li / p.per, lb = li - lt * p.per, ls = 0, put_slot = 0;
  int it = lt, ib = lb;        // (where the computing starts, too)
  const char *lp = nullptr, *sp = nullptr;     // (4-bit weights: this lane's, of the next stage)
  // where it copies codes to, the row's bytes from there on, and groups from its own on
  const uint32_t q4_to = (ring + (lane >> 4) * PIECE + (lane & 15) * 16) ^ (lane >> 4 << 6);
  const bool q4_scales = lane < 2 * (SV >> p.log_g);
  const long long q4_sp_step = 2ll * KS * (SV >> p.log_g) * p.width;
  int q4_left = 0, q4_groups = 0;
  bool q4_upper = false;
  auto begin_item = [&] {
    lp = item_rows<WT>(p, tiles, lt, lb);
    if constexpr (kQ4<WT>) {
      const int at = ks * PIECE + (lane & 15) * 16, g = ks * (SV >> p.log_g) + (lane >> 1);
      lp += (lane >> 4) * row + at;
      sp = item_scales(p, tiles, lt, lb) + 2ll * g * p.width + (lane & 1) * p.second_s;
      q4_left = row - at;
      q4_groups = p.groups - g;
      q4_upper = has_upper(p, lb);
    }
  };
  if constexpr (kQ4<WT>) {
    if (li < p.hi) begin_item();
  } else {
    lp = li < p.hi ? item_rows<WT>(p, tiles, lt, lb) : nullptr;
  }
  auto put = [&] {
    const int v0 = kQ4<WT> ? 0 : (ls * KS + ks) * SV;
    if (li < p.hi && v0 < K) {     // (4-bit weights: q4_left and q4_groups tell where the row ends)
      // row r's 16-byte pieces change places with their neighbours 64 bytes on
      // for odd r, so that the rows a quarter-warp reads fall on different banks
      if constexpr (kQ4<WT>) {
        // two rows at a time, then the scales: lane 2 g + h has group g's of half h.
        // What lies in the place of codes past the row's end are codes, which meet
        // zeros of x; the scales of groups past it are zeros.
        const bool on = q4_left > 0;
        const uint32_t slot_at = put_slot * STAGE;
        copy16_rows(q4_to + slot_at, lp, 2 * row, on);
        copy16_rows(q4_to + slot_at + 8 * PIECE, lp + p.second, 2 * row, on && q4_upper);
        const bool there = q4_groups > 0 && (q4_upper || !(lane & 1));
        copy16_or0(ring + slot_at + 16 * PIECE + lane * 16, there ? sp : p.s, there, q4_scales);
        lp += KS * PIECE;
        sp += q4_sp_step;
        q4_left -= KS * PIECE;
        q4_groups -= KS * (SV >> p.log_g);
      } else {
        const uint32_t dst = ring + put_slot * STAGE + lane * 16;
        constexpr int ES = PIECE / SV;
        const int at = v0 * ES + lane * 16;
        const bool on = at < K * ES;
        const char* src = lp + (on ? at : 0);
#pragma unroll
        for (int r = 0; r < 8; ++r) copy16((dst + r * PIECE) ^ ((r & 1) << 6), src + (long long)r * K * ES, on);
        if (has_upper(p, lb)) {
          src += p.second;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            copy16((dst + (8 + r) * PIECE) ^ ((r & 1) << 6), src + (long long)r * K * ES, on);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    put_slot = put_slot + 1 == NS ? 0 : put_slot + 1;
    if (++ls < steps) return;
    ls = 0;
    li += groups;
    lb += groups;
    if (kQ4<WT>) {
      if (li >= p.hi) return;
      while (lb >= p.per) { lb -= p.per; ++lt; }
      begin_item();
      return;
    }
    lp += item_step;
    if (lb >= p.per && li < p.hi) {
      do { lb -= p.per; ++lt; } while (lb >= p.per);
      lp = item_rows<WT>(p, tiles, lt, lb);
    }
  };
#pragma unroll
  for (int u = 0; u < NS; ++u) put();
  job.wait_tokens();

  // what is being computed: item, its tile and block
  int i = p.lo + mine, parity = 0, slot = 0;
  int tile = p.lo / p.per;
  for (int b_lo = p.lo; b_lo < p.hi;) {
    // the tokens of as many of the next tiles as there is room for
    int t = tile, used = 0;
    bar_sync<CTHREADS>();      // the last ones are no longer read
    const int first = t;
    for (; t * p.per < p.hi; ++t) {
      const Tile tl = tiles[p.t0 + t];
      const int need = tl.n * pitch * (!UP && kBf16Tokens<WT> ? 2 : 1);
      if (t > first && used + need > rows_bytes) break;
      job.load(tl, K, rows + used);
      if (threadIdx.x == 0) row_at[t] = used;
      used += need;
    }
    const int b_hi = min(p.hi, t * p.per);
    b_lo = b_hi;
    tile = t;
    bar_sync<CTHREADS>();

    while (i < b_hi) {
      const Tile tl = tiles[p.t0 + it];
      Products<WT, UP> sum;
      sum.begin(p, rows + row_at[it], pitch, tl.n, lane);
      // the biases of the item's rows, one a lane, on their way from here on
      const float bias = job.bias(p, tl, ib, lane);
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
        job.out(p, tl, ib, row, tok, v0, v1, b0, b1);
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

}  // namespace
}  // namespace moe
