// Tokens by expert, and the weighted sum of the experts' rows.
#pragma once

#include <stdint.h>

#include "cluster.cuh"
#include "common.cuh"
#include "fp8_rows.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// Dispatch: a stable counting sort of the choices by expert, in one launch of
// one cluster, whose CTAs take consecutive runs of the choices: each counts its
// run, they add up one another's counts through distributed shared memory, and
// each places its own entries, 256 a warp at a time, ranked among equals by a
// match over the warp's lanes and the counts of the warps before.  No workspace
// and no order that could change.
// ---------------------------------------------------------------------------
constexpr int kDispThreads = 1024, kDispWarps = 32;
constexpr int kDispMaxExperts = 1024;
constexpr int kDispIter = 8;                                   // times 32 choices a warp and round
constexpr int kDispRound = kDispWarps * kDispIter * 32;        // choices a CTA places at a time
constexpr int kDispMaxCtas = 8;

struct DispatchArgs {
  const int* idx;
  int n, top_k, experts;   // n choices
  int* offsets;
  int* rows;
  int* slots;
};

// Inclusive scan over the block's 1,024 threads.
__device__ __forceinline__ int disp_scan(int v, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += x;
  }
  return v + (warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
}

// Dynamic shared memory: uint16 counts [kDispWarps][experts].
static __global__ void __launch_bounds__(kDispThreads)
    dispatch_kernel(const __grid_constant__ DispatchArgs a) {
  extern __shared__ __align__(16) uint16_t disp_counts[];
  __shared__ int s_total[kDispMaxExperts];   // this CTA's choices of each expert
  __shared__ int s_next[kDispMaxExperts];    // where its next one goes
  __shared__ int s_warp[kDispWarps];
  __shared__ int s_end;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, E = a.experts;
  const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
  const int per = ((a.n + ctas - 1) / ctas + 31) / 32 * 32;
  const int i0 = min(a.n, rank * per), i1 = min(a.n, i0 + per);
  s_total[t] = 0;
  __syncthreads();
  for (int i = i0 + t; i < i1; i += kDispThreads) {
    const int e = __ldg(a.idx + i);
    if ((unsigned)e < (unsigned)E) atomicAdd(&s_total[e], 1);
  }
  cluster_sync();
  int all = 0, before = 0;
  if (t < E) {
    const uint32_t mine = smem_addr(&s_total[t]);
    for (int c = 0; c < ctas; ++c) {
      const int v = ld_cluster_s32(cluster_map(mine, c));
      if (c < rank) before += v;
      all += v;
    }
  }
  const int end = disp_scan(all, s_warp);
  s_next[t] = end - all + before;
  if (rank == 0) {
    if (t < E) a.offsets[t] = end - all;
    if (t == E - 1) a.offsets[E] = end;
  }
  if (t == E - 1) s_end = end;
  __syncthreads();
  // past the last entry, where choices name no expert
  for (int i = s_end + rank * kDispThreads + t; i < a.n; i += ctas * kDispThreads) a.rows[i] = -1;

  uint16_t* mine = disp_counts + warp * E;
  for (int r0 = i0; r0 < i1; r0 += kDispRound) {
    for (int e = lane; e < E; e += 32) mine[e] = 0;
    __syncwarp();
    const int w0 = r0 + warp * (kDispIter * 32);
    int expert[kDispIter], at[kDispIter];
#pragma unroll
    for (int k = 0; k < kDispIter; ++k) {
      const int i = w0 + 32 * k + lane;
      expert[k] = i < i1 ? __ldg(a.idx + i) : -1;
      if ((unsigned)expert[k] >= (unsigned)E) expert[k] = -1;
    }
#pragma unroll
    for (int k = 0; k < kDispIter; ++k) {
      const unsigned same = __match_any_sync(0xffffffffu, expert[k]);
      const int before_me = __popc(same & ((1u << lane) - 1));
      int seen = 0;
      if (expert[k] >= 0) seen = mine[expert[k]];
      __syncwarp();
      if (expert[k] >= 0 && before_me == 0) mine[expert[k]] = (uint16_t)(seen + __popc(same));
      __syncwarp();
      at[k] = seen + before_me;
    }
    __syncthreads();
    // the warps' counts to where each warp's first one goes, relative to s_next
    if (t < E) {
      int sum = 0;
      for (int w = 0; w < kDispWarps; ++w) {
        const int v = disp_counts[w * E + t];
        disp_counts[w * E + t] = (uint16_t)sum;
        sum += v;
      }
      s_total[t] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDispIter; ++k) {
      const int i = w0 + 32 * k + lane;
      if (i >= i1) continue;
      int slot = -1;
      if (expert[k] >= 0) {
        slot = s_next[expert[k]] + mine[expert[k]] + at[k];
        a.rows[slot] = i / a.top_k;
      }
      a.slots[i] = slot;
    }
    __syncthreads();
    if (t < E) s_next[t] += s_total[t];
    __syncthreads();
  }
  cluster_sync();   // no CTA leaves while another may still read its counts
}

// ---------------------------------------------------------------------------
// Combine: a thread's 8 columns of a token, the experts' rows loaded ahead of
// their sums, which are taken in the order of j.
// ---------------------------------------------------------------------------
constexpr int kCombThreads = 128;

struct CombineArgs {
  const void* y;
  long long ys;
  const float* w;
  const int* slots;
  const void* res;   // or null
  long long rs;
  void* out;
  long long os;
  int tokens, top_k, y_rows, d, f16;
};

template <bool F32>
static __global__ void __launch_bounds__(kCombThreads)
    combine_kernel(const __grid_constant__ CombineArgs a) {
  const int c = 8 * (blockIdx.x * kCombThreads + threadIdx.x);
  if (c >= a.d) return;
  for (int t = blockIdx.y; t < a.tokens; t += gridDim.y) {
    float sum[8];
    if (a.res) {
      raw8_to_float<F32>(load_raw8<F32>(a.res, t * a.rs + c), a.f16, sum);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = 0.f;
    }
    const long long first = (long long)t * a.top_k;
    constexpr int AHEAD = 8;
    for (int k0 = 0; k0 < a.top_k; k0 += AHEAD) {
      Raw8<F32> r[AHEAD];
      float w[AHEAD];
      bool ok[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int slot = k0 + k < a.top_k ? __ldg(a.slots + first + k0 + k) : -1;
        ok[k] = (unsigned)slot < (unsigned)a.y_rows;
        if (ok[k]) {
          r[k] = load_raw8<F32>(a.y, slot * a.ys + c);
          w[k] = __ldg(a.w + first + k0 + k);
        }
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (!ok[k]) continue;
        float v[8];
        raw8_to_float<F32>(r[k], a.f16, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = fmaf(w[k], v[j], sum[j]);
      }
    }
    store8<F32>(a.out, t * a.os + c, a.f16, sum);
  }
}

}  // namespace moe
