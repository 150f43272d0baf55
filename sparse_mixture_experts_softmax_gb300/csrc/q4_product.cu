// The matrix product grouped by expert with 4-bit weights, for few rows, and the choice
// between this kernel and the one for many (q4_gemm.cu).
//
// A few rows of an expert are bound by reading its weights once, and a single matrix has
// to be spread over all SMs: the few-token layer's way (decode_experts.cuh), 16 rows of
// a matrix times up to 16 rows of x an item, items of equal bytes dealt to the blocks,
// the warps of a block sharing an item's inputs where it has few items.
#include <limits.h>

#include "decode_experts.cuh"
#include "q4.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int CW_ = Stored<Q4>::CW;
static_assert(CW_ == WARPS, "all warps multiply");
constexpr int MAX_ROWS = 4096;               // of a call (their tiles lie in shared memory)
struct RowsPlan {
  int off_red, off_tile, off_at, off_rows, rows_bytes, max_tiles;
};
__host__ __device__ inline RowsPlan rows_plan(int R, int E, int tt) {
  RowsPlan P;
  P.max_tiles = (E < R ? E : R) + R / tt;
  int o = CW_ * Stored<Q4>::NS * Stored<Q4>::STAGE;
  P.off_red = o; o += 2 * CW_ * part_floats<Q4>(tt) * 4;
  P.off_tile = o; o += up16(P.max_tiles * 8);
  P.off_at = o; o += up16(P.max_tiles * 4);
  P.off_rows = o;
  P.rows_bytes = SMEM_MAX - o;
  return P;
}

// Tokens straight from x, results straight to c.
struct RowsJob {
  const Q4Product& p;
  __device__ __forceinline__ void wait_tokens() const {}
  __device__ __forceinline__ void load(const Tile& tl, int K, char* rows) const {
    const int pitch = row_pitch<Q4>(K), pieces = (K + 127) / 128 * 16;       // of 8 values
    const int lg = warps_a_token<CW_>(tl.n), step = 32 << lg;
    for (int t = threadIdx.x >> 5 >> lg; t < tl.n; t += CW_ >> lg) {
      const bf16* x = static_cast<const bf16*>(p.x) + (long long)(tl.start + t) * K;
#pragma unroll 4
      for (int c = threadIdx.x & (step - 1); c < pieces; c += step) {
        const int at = (c & ~15) | (c & 3) << 2 | (c >> 2 & 3);             // (as load_tile has it)
        *reinterpret_cast<uint4*>(rows + t * pitch + at * 16) =
            c * 8 < K ? __ldg(reinterpret_cast<const uint4*>(x + c * 8)) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  __device__ __forceinline__ float bias(const Part& pt, const Tile& tl, int block, int lane) const {
    if (p.bias == nullptr || lane >= 16 || block * 16 + lane >= pt.width) return 0.f;
    return __ldg(p.bias + (long long)tl.e * p.N + block * 16 + lane);
  }
  __device__ __forceinline__ void out(const Part& pt, const Tile& tl, int block, int row, int tok, float v0,
                                      float v1, float b0, float b1) const {
    if (tok >= tl.n) return;
    bf16* c = static_cast<bf16*>(p.c) + (long long)(tl.start + tok) * p.N + block * pt.rows + row;
    if (p.act == 2) {
      *c = __float2bfloat16_rn(silu_f(v0) * v1);
      return;
    }
    c[0] = __float2bfloat16_rn(act(v0 + b0));
    if (block * 16 + 8 < pt.width) c[8] = __float2bfloat16_rn(act(v1 + b1));
  }
  __device__ __forceinline__ float act(float v) const {
    if (p.act == 1) return gelu_tanh_f(v);
    return p.act == 0 && v < 0.f ? 0.f : v;      // a NaN stays one
  }
};

__global__ void __launch_bounds__(THREADS, 1)
q4_rows_kernel(const __grid_constant__ Q4Product p, const int tt) {
  extern __shared__ __align__(256) char sm[];
  __shared__ int n_tiles;
  int* scan = reinterpret_cast<int*>(sm);          // (where the weights' buffers lie later)
  int* offs = scan + 64;                           // [E + 1]
  const RowsPlan P = rows_plan(p.R, p.E, tt);
  Tile* tiles = reinterpret_cast<Tile*>(sm + P.off_tile);
  const int e = threadIdx.x;
  pdl_begin();
  const int lo = clamped_offset(p.offsets, p.E, p.R, scan);
  if (e <= p.E) offs[e] = lo;
  __syncthreads();
  const int rows = e < p.E ? offs[e + 1] - lo : 0, mine = (rows + tt - 1) / tt;
  const int behind = q4_block_scan<false>(mine, scan + 32);
  for (int i = 0; i < mine; ++i)
    tiles[behind - mine + i] = Tile{(short)e, (short)min(tt, rows - i * tt), lo + i * tt};
  if (e == THREADS - 1) n_tiles = behind;
  __syncthreads();

  Part pt;
  const bool pair = p.act == 2;
  pt.rows = pair ? 8 : 16;
  pt.K = p.K;
  pt.width = p.N;
  pt.per = (p.N + pt.rows - 1) / pt.rows;
  pt.t0 = 0;
  const long long items = (long long)n_tiles * pt.per;
  pt.lo = (int)(items * blockIdx.x / gridDim.x);
  pt.hi = (int)(items * (blockIdx.x + 1) / gridDim.x);
  pt.w = static_cast<const char*>(p.codes);
  pt.s = static_cast<const char*>(p.scales);
  pt.second = !pair ? 8ll * Stored<Q4>::row(p.K) : static_cast<const char*>(p.codes3) - pt.w;
  pt.second_s = !pair ? 16 : static_cast<const char*>(p.scales3) - pt.s;
  pt.log_g = p.G == 32 ? 5 : p.G == 64 ? 6 : 7;
  pt.groups = (p.K + p.G - 1) / p.G;
  const uint32_t ring = smem_addr(sm) + (threadIdx.x >> 5) * Stored<Q4>::NS * Stored<Q4>::STAGE;
  compute<Q4, true>(RowsJob{p}, pt, tiles, tt, reinterpret_cast<int*>(sm + P.off_at), sm + P.off_rows,
                    P.rows_bytes, reinterpret_cast<float*>(sm + P.off_red), ring);
}

// Rows of a tile: as many as there is room for one tile of, or 0.
int tile_rows(const Q4Product& p) {
  const long long pitch = row_pitch<Q4>(p.K);
  for (int tt = most_tokens<Q4>(); tt >= 1; --tt)
    if (tt * pitch <= rows_plan(p.R, p.E, tt).rows_bytes) return tt;
  return 0;
}

cudaError_t launch_q4_rows(const Q4Product& p, int tt, cudaStream_t st) {
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t err = ensure_dynamic_smem(q4_rows_kernel, SMEM_MAX, attr_done);
  if (err != cudaSuccess) return err;
  const int n = tc::sm_count();
  // a block an SM, or fewer where each would have less than 8 KB of weights and less than
  // eight items (1000 rows of 64 x 32, 1 KB of weights: 83 us on one block, 12 on the 32
  // that the items ask for; 333 rows of 1000 x 480 21 on 30 blocks, 13 on all)
  const long long experts = p.E < p.R ? p.E : p.R, mats = p.act == 2 ? 2 : 1;
  const long long by_bytes = (experts * p.N * (p.K / 2) * mats + 8191) / 8192;
  const long long by_items = ((experts + p.R / tt) * p.N * mats + 127) / 128;
  const long long blocks = by_bytes > by_items ? by_bytes : by_items;
  return launch_pdl(q4_rows_kernel, dim3((unsigned)(blocks < n ? blocks : n)), dim3(THREADS), SMEM_MAX,
                    st, p, tt);
}

}  // namespace

cudaError_t launch_q4_product(const Q4Product& p, cudaStream_t st) {
  const int tt = p.R <= MAX_ROWS && !p.stall ? tile_rows(p) : 0;
  if (tt == 0) return launch_q4_gemm(p, st);
  // Every row tile reads its expert's matrix again, most of it from L2, and widens it
  // again; the other kernel does so once for up to 160 rows, but its tiles of 128 outputs
  // leave SMs without work where there are few, and a tile's chain along K then takes 2 us for
  // 1024 inputs.  Its tensor maps cost the host 1.3 us more.  So the few-row kernel is taken where
  // experts have three quarters of a tile's rows or less in the mean, or where all its tiles'
  // weights are no more than 8 MB (either way below the host's time for a call, 8 and 9.4 us) or
  // 1.5 K^2 bytes.  Measured, few and many (us, from a graph, rows dealt evenly): 128 experts of
  // 4096 inputs and 2 x 2048 outputs, 1, 4, 5, 8 and 16 rows an expert 190, 200, 201, 381, 569 and
  // 250, 252, 252, 254, 258; 16 of 2048 inputs and 2 x 2048 outputs, 8, 12 and 16 rows 20, 25, 41 and
  // 23, 23, 23; one matrix of 2048 x 8192 (outputs, inputs), 16, 32 and 48 rows 12.5, 18.9, 27.5 and
  // 20.9, 21.1, 21.5; of 4096 x 4096, 16, 32 and 64 rows 9.1, 12.4, 18.8 and 12.5, 12.8, 13.5; of
  // 2048 x 2048, 16, 32, 48 and 64 rows 6.6, 8.2, 7.7, 11.7 and 8.3, 8.4, 8.7, 9.0; of 1024 x 1024, 32,
  // 128, 256 and 512 rows 6.0, 7.6, 9.5, 11.9 and 6.3, 7.6, 7.6, 7.7.  Call after call through Python:
  // 8 experts of 480 inputs and 1000 outputs, 42 and 80 rows an expert 8.3, 11.0 and 9.5, 9.4; one
  // matrix of 1024 x 1024, 64 and 256 rows 7.8, 10.3 and 9.0, 9.4.  Left behind: weights of 24 MB in
  // place of 8 (1000 rows of 1000 x 480 11.3 and 7.1).
  // The host does not see where the rows are: 128, 256 and 640 rows of the 128 experts, all of
  // them on four, take the few-row kernel's 42, 71 and 146 us, where the other's are 13, 14 and 18.
  const long long tiles = (p.E < p.R ? p.E : p.R) + p.R / tt;
  const long long bytes = tiles * p.N * (p.K / 2) * (p.act == 2 ? 2 : 1);
  const bool few = 4ll * p.R <= 3ll * tt * p.E || bytes <= (8ll << 20) || 2 * bytes <= 3ll * p.K * p.K;
  if (!few || tiles * ((p.N + 7) / 8) > INT_MAX) return launch_q4_gemm(p, st);
  return launch_q4_rows(p, tt, st);
}

}  // namespace moe
