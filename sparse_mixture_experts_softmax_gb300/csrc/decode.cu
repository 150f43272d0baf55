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
//
// 4-bit layers widen each weight to bf16 in front of the same products, which then counts
// more than HBM: all sixteen warps multiply, each with stages of 256 bytes (512 inputs) of
// 16 rows, tiles are of up to 8 tokens, and calls of up to four tokens have a kernel of
// their own (Q4Few); where rows are wide, eight warps with larger tiles (wide_rows).  Measured,
// the large layer: 64 tokens (1.78 GB of codes and scales, groups of 32) 361 to 377 us, 4.7 to
// 4.9 TB/s; one token (106 MB with the router's weights, groups of 128) 41 us, of which 7 go to
// the logits and the selection and 4 to barriers and the last pass.  Left behind: eight warps 61
// and 599 us (one and 64 tokens); stages of 128 bytes 64 tokens 519 (the instructions to copy a
// stage are the same as for 256); the four-token form chosen for every tile within one kernel 43
// and 400 (its registers spill); W2's first rows copied to L2 ahead 47 and 394, against 45 and 392
// then; a stage's loop unrolled four times the same times and 30 KB more code.
#include "../../include/moe_block.h"
#include "decode_experts.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

template <typename WT>
__global__ void __launch_bounds__(THREADS, 1)
decode_kernel(const __grid_constant__ DecodeArgs a, const int tt) {
  extern __shared__ __align__(256) char sm[];
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
  router<typename Stored<WT>::Act, WARPS>(a, scratch);
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
  if (warp < Stored<WT>::CW) {
    const uint32_t ring = smem_addr(sm) + warp * Stored<WT>::NS * Stored<WT>::STAGE;
#pragma unroll 1
    for (int shared = 0; shared < (a.Fs > 0 ? 2 : 1); ++shared)
      compute<WT, true>(LayerJob<WT, true>{a, rt, nullptr}, make_part<WT, true>(a, nr, nt, !shared),
                        rt.tiles, tt, row_at + shared * nr, rows, P.rows_bytes, red, ring);
#pragma unroll 1
    for (int shared = 0; shared < (a.Fs > 0 ? 2 : 1); ++shared)
      compute<WT, false>(LayerJob<WT, false>{a, rt, shared ? nullptr : &flag},
                         make_part<WT, false>(a, nr, nt, !shared), rt.tiles, tt, row_at + shared * nr,
                         rows, P.rows_bytes, red, ring);
    grid_barrier<kCThreads<WT>>(a.ctl, 2, &flag);
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
          typename Stored<WT>::Act* y = static_cast<typename Stored<WT>::Act*>(a.y) + (long long)i * 4;
          if constexpr (kBf16Tokens<WT>)
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

// A tile of one token has room whatever the entry points let through: the lists of the
// most tokens, of 32 choices among 256 experts, beside the widest rows.
template <typename WT>
constexpr bool always_fits(int T) {
  return row_bytes<WT>(MOE_DECODE_MAX_ROW_BYTES / (int)sizeof(typename Stored<WT>::Act), MOE_DECODE_MAX_F) <=
         make_plan<WT>(T, 32, 256, MOE_DECODE_MAX_F, 1).rows_bytes;
}
static_assert(always_fits<float>(MOE_DECODE_MAX_TOKENS) && always_fits<bf16>(MOE_DECODE_MAX_TOKENS) &&
              always_fits<Q4Wide>(MOE_DECODE_MAX_TOKENS) && always_fits<Q4Few>(most_tokens<Q4Few>()), "limits");

template <typename WT>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t st) {
  static std::atomic<unsigned long long> attr_done{0};
  const int sms = tc::sm_count(), tt = tile_tokens<WT>(a);
  if (tt <= 0) return cudaErrorInvalidValue;    // (past the entry points' limits)
  // a block per SM, or fewer where each would have less than 8 KB of weights (the
  // kernel's time hardly goes with it: 4 KB, 16 KB and a block on every SM are
  // within 0.2 us of 13.4 at 96 KB of weights, of 13.6 at 390 KB, of 14.4 at
  // 780 KB; one block alone takes 0.3 us more than four at 32 KB, 23 us at 390 KB)
  const long long experts = (long long)a.T * a.k < a.E ? (long long)a.T * a.k : a.E;
  const long long bytes = (experts * a.F + a.Fs) * (a.act == 2 ? 3 : 2) * (long long)Stored<WT>::row(a.D);
  const long long blocks = (bytes + 8191) / 8192;
  return launch_cooperative(decode_kernel<WT>, (int)(blocks < sms ? blocks : sms), THREADS,
                            attr_done, st, a, tt);
}

// Whether a call of 4-bit weights goes by half the warps.  Their tiles have more tokens where
// rows are wide, so that an expert's weights are read and widened fewer times, but a reading
// takes up to 1.2 times as long: they are chosen where the readings, tokens dealt evenly, are
// less than 1 / 1.2, or where the others have no room for a row at all (64 tokens' 32 choices
// among 256 experts beside rows of more than 18 KB).  Measured, 16 and 8 warps (us, from a
// graph; D = 4096 where not stated): 8 experts, k = 2, F = 8192, T = 5, 8, 16, 32, 64: 92, 130, 212,
// 364, 1211 and 106, 128, 172, 278, 460; F = 4096: 55, 72, 86, 123, 249 and 61, 80, 88, 105, 161; F =
// 2816: 40, 54, 68, 95, 147 and 44, 60, 67, 91, 125; D = 16384, F = 512, T = 5, 16, 64: 43, 80, 366 and
// 46, 72, 167; 64 experts, k = 8, F = 4096, T = 16, 64: 334, 947 and 358, 565; F = 1408 and four shared
// experts: 224, 702 and 197, 397; 16 experts, k = 4, D = F = 2048, T = 64: 87 and 95; the large layer,
// T = 16, 64: 215, 359 and 258, 420.
bool wide_rows(const DecodeArgs& a) {
  const long long R = (long long)a.T * a.k, experts = R < a.E ? R : a.E;
  const long long eight = tile_tokens<Q4Eight>(a), wide = tile_tokens<Q4Wide>(a);
  auto readings = [&](long long tt) {          // times tt
    const long long routed = experts * tt > R ? experts * tt : R, shared = a.T > tt ? a.T : tt;
    return routed + (a.Fs > 0 ? a.n_shared * shared : 0);
  };
  return 5 * wide * readings(eight) > 6 * eight * readings(wide);
}

}  // namespace

cudaError_t launch_decode_init(int* ctl, cudaStream_t st) {
  return launch_pdl(decode_init_kernel, dim3(1), dim3(DC_WORDS), 0, st, ctl);
}

cudaError_t launch_decode(int kind, const DecodeArgs& a, cudaStream_t st) {
  // 4-bit weights, one token of the large layer: 41 us by Q4Few's kernel, 45 by tiles of up
  // to 16 tokens.  More tokens, tiles of up to 16 and of up to 8 (us; registers for 16 spill, and
  // a second tile's weights come from L2): the large layer, 64 tokens 389 and 374; 64 experts of
  // 1024 and 704, k = 6, 16 and 64 tokens 38.5, 55.1 and 36.1, 45.0; 16 of 1024 and 1024, k = 4, 48
  // tokens 42.1 and 35.1; 8 of 512 and 1024, k = 2, 5 and 64 tokens 18.5, 30.4 and 17.6, 26.6.
  if (kind == DECODE_Q4 && a.T <= most_tokens<Q4Few>()) return launch_t<Q4Few>(a, st);
  if (kind == DECODE_Q4) return wide_rows(a) ? launch_t<Q4Wide>(a, st) : launch_t<Q4Eight>(a, st);
  return kind == DECODE_BF16 ? launch_t<bf16>(a, st) : launch_t<float>(a, st);
}

}  // namespace moe
