// The routing half of the few-token MoE layer's kernel: bounded waits, the grid
// barrier, the router's logits and the selection.
//
// A block runs most of this once and from a cold instruction cache, where the
// weights that stream through L2 leave nothing of the last call's code: the
// larger pieces are functions of their own, not inlined at every use (one token
// of the large layer: 90 -> 79 us).
#pragma once

#include <float.h>

#include "common.cuh"
#include "decode.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int SMEM_MAX = 226 * 1024;   // dynamic part of 227 KB
constexpr unsigned long long WAIT_NS = 2000000000ull;

// ---- waits: every one is bounded, and an expired one ends the kernel in order
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// A barrier of the block's first NTHREADS threads.
template <int NTHREADS>
__device__ __forceinline__ void bar_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(NTHREADS) : "memory");
}
// One of the kernel's grid barriers, for the first NTHREADS threads of every
// block.  Each has a counter of its own, zero on entry; the last block to leave
// the kernel zeroes them for the next call.  Returns false when the wait expired
// (uniform over those threads).
template <int NTHREADS>
__device__ __forceinline__ bool grid_barrier(int* ctl, int which, int* flag) {
  bar_sync<NTHREADS>();
  if (gridDim.x == 1) return *flag == 0;
  if (threadIdx.x == 0) {
    int* bar = ctl + DC_BAR + which;
    // release and acquire on the counter order the block's accesses (the block's
    // barrier carries them to and from this thread); a full fence costs more
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(bar) : "memory");
    int seen = 0;
    unsigned long long t0 = 0;
    while (true) {
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(bar) : "memory");
      if (seen >= (int)gridDim.x) break;
      const unsigned long long t = now_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > WAIT_NS) {
        ctl[DC_STATUS] = DEV_STATUS_TIMEOUT;
        *flag = 1;
        break;
      }
    }
  }
  bar_sync<NTHREADS>();
  return *flag == 0;
}

// Sums 32 values over the warp at once: lane l gets the whole sum of v[l].
// (31 exchanges; one at a time they would take 160.)
__device__ __forceinline__ float warp_sum32(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

// Logits of the units (EB experts, TB tokens) that fall to this block, one unit
// at a time by its NW warps.  The layer multiplies with W_g in its own type, as
// its training forward does; bf16 products are exact in fp32, a thread's chain
// is a few terms long and the rest is a tree, so that a near-tie of two experts
// is as narrow as fp32 allows.  red: NW * 32 floats of shared memory.
template <typename WT, int EB, int TB, int NW>
__device__ __noinline__ void router_logits(const DecodeArgs& a, float* red) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = a.T, D = a.D, E = a.E;
  const int ntt = (T + TB - 1) / TB, neb = (E + EB - 1) / EB;
  const WT* x = static_cast<const WT*>(a.x);
  for (int u = blockIdx.x; u < neb * ntt; u += gridDim.x) {
    const int e0 = (u / ntt) * EB, t0 = (u % ntt) * TB, nt = min(TB, T - t0), ne = min(EB, E - e0);
    float s[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = 0.f;
    for (int d = tid * 4; d < D; d += NW * 128) {
      float w[EB][4];
#pragma unroll
      for (int e = 0; e < EB; ++e) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(
            a.w_gate + (long long)(e0 + min(e, ne - 1)) * D + d));
        w[e][0] = q.x; w[e][1] = q.y; w[e][2] = q.z; w[e][3] = q.w;
        if constexpr (sizeof(WT) == 2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[e][i] = to_f(from_f<bf16>(w[e][i]));
        }
      }
      // absent tokens repeat the last one: a branch here would make the loads
      // wait for one another
      float v[TB][4];
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const WT* px = x + (long long)(t0 + min(t, nt - 1)) * D + d;
        if constexpr (sizeof(WT) == 2) {
          const uint2 q = __ldg(reinterpret_cast<const uint2*>(px));
          v[t][0] = __uint_as_float(q.x << 16); v[t][1] = __uint_as_float(q.x & 0xffff0000u);
          v[t][2] = __uint_as_float(q.y << 16); v[t][3] = __uint_as_float(q.y & 0xffff0000u);
        } else {
          const float4 q = __ldg(reinterpret_cast<const float4*>(px));
          v[t][0] = q.x; v[t][1] = q.y; v[t][2] = q.z; v[t][3] = q.w;
        }
      }
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int e = 0; e < EB; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[e * 8 + t] = fmaf(w[e][i], v[t][i], s[e * 8 + t]);
    }
    if (EB * TB == 1) {
      const float v = warp_sum(s[0]);
      if (lane == 0) red[warp * 32] = v;
    } else {
      red[warp * 32 + lane] = warp_sum32(s, lane);
    }
    __syncthreads();
    if (tid < EB * 8) {
      const int e = tid / 8, t = tid % 8;
      if (e < ne && t < nt) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += red[w * 32 + tid];
        if (a.logit_bias != nullptr) v += a.logit_bias[e0 + e];
        __stcg(a.logits + (long long)(t0 + t) * E + e0 + e, v);
      }
    }
    __syncthreads();
  }
}

template <typename WT, int NW>
__device__ __forceinline__ void router(const DecodeArgs& a, float* red) {
  if (a.T == 1) router_logits<WT, 1, 1, NW>(a, red);
  else if (a.E * ((a.T + 7) / 8) > 2 * (int)gridDim.x) router_logits<WT, 4, 8, NW>(a, red);
  else router_logits<WT, 1, 8, NW>(a, red);
}

// Selection keys as whole numbers in the order of the selection: a larger key
// first, NaN after every number; 0 is left for what may not be chosen.  Equal
// ones go to the smaller id.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {     // of a number's key
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// Token t's scores, kept groups, k experts and gates by one warp; a lane holds
// the experts lane + 32 c, c < NC.  Each of the k picks is two whole-number
// reductions: the largest key, then the smallest id that has it.  (Two or four
// tokens side by side in a warp cost more in cold code than they save.)  row: E
// floats of shared memory of the warp's own; mask: see select_all.
template <int NC>
__device__ __noinline__ void select_token(const DecodeArgs& a, int t, float* row, short* idx,
                                          float* gate, uint32_t* mask, int lane) {
  const int E = a.E, k = a.k;
  float s[NC], cb[NC];
  uint32_t key[NC];
  const float* lg = a.logits + (long long)t * E;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 32 * c;
    s[c] = e < E ? __ldcg(lg + e) : -INFINITY;
    cb[c] = a.corr_bias != nullptr && e < E ? __ldg(a.corr_bias + e) : 0.f;
  }
  if (a.score == 0) {
    float m = -FLT_MAX, z = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) m = fmaxf(m, s[c]);
    m = key_value(__reduce_max_sync(0xffffffffu, order_key(m)));
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      s[c] = lane + 32 * c < E ? expf(s[c] - m) : 0.f;
      z += s[c];
    }
    const float inv = 1.0f / warp_sum(z);
#pragma unroll
    for (int c = 0; c < NC; ++c) s[c] *= inv;
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) s[c] = sigmoidf_(s[c]);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = lane + 32 * c;
    const float kv = a.corr_bias != nullptr ? s[c] + cb[c] : s[c];
    key[c] = e < E ? order_key(kv) : 0u;
    if (e < E) row[e] = kv;
  }
  __syncwarp();
  if (a.n_groups > 1) {
    const int NG = a.n_groups, per = E / NG;
    uint32_t gk = 0u;
    if (lane < NG) {
      float m1 = -INFINITY, m2 = -INFINITY;
      for (int e0 = 0; e0 < per; e0 += 8) {
        float v[8];            // eight reads at a time, not one after the other
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = e0 + i < per ? row[lane * per + e0 + i] : -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m2 = v[i] > m1 ? m1 : (v[i] > m2 ? v[i] : m2);
          m1 = v[i] > m1 ? v[i] : m1;
        }
      }
      gk = order_key((per == 1 || a.group_score == 1) ? m1 : m1 + m2);
    }
    uint32_t keep = 0u;
    for (int r = 0; r < a.topk_groups; ++r) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, gk);
      const int g = __ffs(__ballot_sync(0xffffffffu, lane < NG && gk == best)) - 1;
      keep |= 1u << g;
      if (lane == g) gk = 0u;
    }
    const float inv = 1.0f / (float)per;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = lane + 32 * c, g = (int)(((float)e + 0.5f) * inv);   // e / per, exact below 2^8
      if (e < E && !((keep >> g) & 1u)) key[c] = 0u;
    }
    __syncwarp();
  }
  // the scores take the keys' place: a pick looks its own up at the end
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (lane + 32 * c < E) row[lane + 32 * c] = s[c];
  __syncwarp();
  int pick = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint32_t top = 0u;
    int at = 0x7fffffff;
#pragma unroll
    for (int c = NC - 1; c >= 0; --c)
      if (key[c] >= top && key[c] != 0u) { top = key[c]; at = lane + 32 * c; }
    const uint32_t best = __reduce_max_sync(0xffffffffu, top);
    const int e = __reduce_min_sync(0xffffffffu, top == best ? at : 0x7fffffff);
    if (lane == j) pick = e;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (lane + 32 * c == e) key[c] = 0u;
  }
  const float mine = lane < k ? row[pick] : 0.f;
  const float sum = warp_sum(mine);
  if (lane < k) {
    idx[t * k + lane] = (short)pick;
    gate[t * k + lane] = mine / sum;
    if (mask != nullptr)
      atomicOr(mask + 2 * pick + (t >> 5), 1u << (t & 31));   // whole numbers: any order
  }
  __syncwarp();
}

struct Tile {
  short e, n;         // expert (-1: the shared branch), tokens
  int start;          // first slot (first token for the shared branch)
};
// The routing of a call in shared memory.
struct Routing {
  short* idx;         // [T, k]
  float* gate;        // [T, k]
  short* tok;         // [R] slot -> token; slots are expert-major, tokens ascending
  short* slot;        // [T, k] -> slot, or -1 (dropped by the capacity)
  Tile* tiles;        // token tiles of the chosen experts, then of the shared branch
  int* scan;          // 8 words of scratch
};

// Selection and the expert-major lists, by NW warps (every block for itself:
// cheaper than another grid barrier).  An expert's tokens are a mask of at most
// 64 bits, so that its count, its slots' order and the capacity's cut are
// population counts.  TT: tokens of a tile; scratch: 768 + NW E words.
template <int NW>
__device__ __forceinline__ void select_all(const DecodeArgs& a, const Routing& r, int TT,
                                           float* scratch, int* n_routed, int* n_tiles) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = a.T, E = a.E, k = a.k, R = T * k;
  uint32_t* mask = reinterpret_cast<uint32_t*>(scratch);      // [256][2]
  int* base_of = reinterpret_cast<int*>(scratch) + 512;       // [256]
  float* row = scratch + 768 + warp * E;
  if (T == 1) {
    // one token: its picks are the lists (an expert keeps at least one row), and
    // the two barriers and the scans below would cost as much as the picking
    if (warp == 0) {
      if (E <= 64) select_token<2>(a, 0, row, r.idx, r.gate, nullptr, lane);
      else if (E <= 128) select_token<4>(a, 0, row, r.idx, r.gate, nullptr, lane);
      else select_token<8>(a, 0, row, r.idx, r.gate, nullptr, lane);
      if (lane < k) {
        r.tiles[lane] = Tile{r.idx[lane], 1, lane};
        r.tok[lane] = 0;
        r.slot[lane] = (short)lane;
        if (blockIdx.x == 0) {
          if (a.idx != nullptr) a.idx[lane] = r.idx[lane];
          if (a.gate != nullptr) a.gate[lane] = r.gate[lane];
        }
      }
      if (lane == 0) {
        *n_routed = k;
        *n_tiles = k + (a.Fs > 0 ? 1 : 0);
        if (a.Fs > 0) r.tiles[k] = Tile{(short)-1, 1, 0};
      }
    }
    __syncthreads();
    return;
  }
  for (int i = tid; i < 512; i += NW * 32) mask[i] = 0u;
  __syncthreads();
  for (int t = warp; t < T; t += NW) {
    if (E <= 32) select_token<1>(a, t, row, r.idx, r.gate, mask, lane);
    else if (E <= 64) select_token<2>(a, t, row, r.idx, r.gate, mask, lane);
    else if (E <= 128) select_token<4>(a, t, row, r.idx, r.gate, mask, lane);
    else select_token<8>(a, t, row, r.idx, r.gate, mask, lane);
  }
  __syncthreads();
  // expert tid's first slot and tile: one scan over the experts' kept counts (at
  // most 2048 in all) and, 16 bits up, their tiles
  int mine = 0, both = 0, incl = 0;
  if (warp < 8) {
    mine = min(__popc(mask[2 * tid]) + __popc(mask[2 * tid + 1]), a.cap);
    both = mine + ((mine + TT - 1) / TT << 16);
    incl = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) r.scan[warp] = incl;
  }
  __syncthreads();
  if (warp < 8) {
    int before = incl - both, total_t = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const int v = r.scan[w];
      if (w < warp) before += v;
      total_t += v >> 16;
    }
    const int base = before & 0xffff;
    int tile = before >> 16;
    base_of[tid] = base;
    for (int i = 0; i < mine; i += TT)
      r.tiles[tile++] = Tile{(short)tid, (short)min(TT, mine - i), base + i};
    const int nsh = a.Fs > 0 ? (T + TT - 1) / TT : 0;
    if (tid < nsh)
      r.tiles[total_t + tid] = Tile{(short)-1, (short)min(TT, T - tid * TT), tid * TT};
    if (tid == 0) {
      *n_routed = total_t;
      *n_tiles = total_t + nsh;
    }
  }
  __syncthreads();
  for (int i = tid; i < R; i += NW * 32) {
    const int e = r.idx[i], t = i / k;
    const uint32_t below = (1u << (t & 31)) - 1u;
    const int place = t < 32 ? __popc(mask[2 * e] & below)
                             : __popc(mask[2 * e]) + __popc(mask[2 * e + 1] & below);
    const int s = base_of[e] + place;
    const bool kept = place < a.cap;
    r.slot[i] = kept ? (short)s : (short)-1;
    if (kept) r.tok[s] = (short)t;
    if (blockIdx.x == 0) {
      if (a.idx != nullptr) a.idx[i] = e;
      if (a.gate != nullptr) a.gate[i] = r.gate[i];
    }
  }
  __syncthreads();
}

// The last block out zeroes the barriers' counters for the next call.
__device__ __forceinline__ void leave(int* ctl) {
  if (gridDim.x == 1) return;
  if (atomicAdd(ctl + DC_EXIT, 1) == (int)gridDim.x - 1) {
    ctl[DC_BAR] = 0;
    ctl[DC_BAR + 1] = 0;
    ctl[DC_BAR + 2] = 0;
    __threadfence();
    ctl[DC_EXIT] = 0;
  }
}

// Launches `kernel` with one block per SM at most, all resident together (its
// blocks wait on one another).
template <typename... KArgs, typename... Args>
cudaError_t launch_cooperative(void (*kernel)(KArgs...), int blocks, int threads,
                               std::atomic<unsigned long long>& attr_done, cudaStream_t st,
                               const Args&... args) {
  cudaError_t e = ensure_dynamic_smem(kernel, SMEM_MAX, attr_done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = SMEM_MAX;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace moe
