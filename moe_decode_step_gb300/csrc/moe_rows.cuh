// Tokens by expert, and the weighted sum of the experts' rows.
#pragma once

#include <stdint.h>

#include "cluster.cuh"
#include "common.cuh"
#include "fp8_rows.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// Dispatch: a stable counting sort of the choices by expert, in one launch of
// clusters of up to 16 CTAs.  The CTAs of a cluster take consecutive runs of the
// choices, count them and add up one another's counts through distributed shared
// memory.  Long calls have several clusters, which all count everything and each
// place their part of every run.  To place choices, a CTA takes 32 x WARPS x ITER a
// round: a choice's place among its warp's is found by ballots over the bits of the
// expert (a match of the lanes takes an SM 60 cycles: with it and one cluster a
// prompt of 32,768 tokens took 27 us, 19 without) and a count a warp and expert; the
// round's entries are put in order in shared memory first, so that an expert's go out
// side by side.  No workspace, and no order that could change.  Latency bounds it.
// Measured on the device: 64 rows of 16 of 896 6.0 us, 32,768 rows of 8 of 256 11.5.
// ---------------------------------------------------------------------------
constexpr int kDispThreads = 1024, kDispWarps = 32;
constexpr int kDispMaxExperts = 1024;
constexpr int kDispMaxCtas = 16;
constexpr int kDispMaxClusters = 4;   // (8 of 16 CTAs do not fit side by side: 20 us)
template <int WARPS, int ITER>
constexpr int disp_smem(int experts) {
  return WARPS * experts * 2 + WARPS * 32 * ITER * (4 + 2);
}

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
  __syncthreads();
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

// Dynamic shared memory: uint16 counts [WARPS][experts], then a round's tokens
// (int) and experts (uint16) in order.
template <int WARPS, int ITER>
static __global__ void __launch_bounds__(kDispThreads)
    dispatch_kernel(const __grid_constant__ DispatchArgs a) {
  extern __shared__ __align__(16) uint16_t disp_counts[];
  __shared__ int s_total[kDispMaxExperts];   // the run's choices of each expert
  __shared__ int s_early[kDispMaxExperts];   // those before this cluster's part
  __shared__ int s_next[kDispMaxExperts];    // where its next one goes
  __shared__ int s_base[kDispMaxExperts];    // the same less its place in the round
  __shared__ int s_warp[kDispWarps];
  __shared__ int s_end;
  constexpr int ROUND = 32 * WARPS * ITER;
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, E = a.experts;
  int* s_token = reinterpret_cast<int*>(disp_counts + WARPS * E);
  uint16_t* s_expert = reinterpret_cast<uint16_t*>(s_token + ROUND);
  uint16_t* mine = disp_counts + warp * E;
  const int ctas = (int)cluster_size(), rank = (int)cluster_rank();
  const int clusters = gridDim.x / ctas, cluster = blockIdx.x / ctas;
  const int per = ((a.n + ctas - 1) / ctas + 31) / 32 * 32;
  const int i0 = min(a.n, rank * per), i1 = min(a.n, i0 + per);
  const int part = (per + clusters - 1) / clusters;
  const int p0 = min(i1, i0 + cluster * part), p1 = min(i1, p0 + part);
  const int bits = 32 - __clz(E - 1);       // of every expert
  const bool once = clusters == 1 && per <= ROUND;   // (alike in every CTA)
  int expert[ITER], at[ITER];

  // this round's choices: their places among their warp's of the same expert, and
  // what the warps before have of each
  auto rank_round = [&](int r0) {
    if (warp < WARPS) {
      const int w0 = r0 + warp * (ITER * 32);
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        const int i = w0 + 32 * k + lane;
        expert[k] = i < p1 ? __ldg(a.idx + i) : -1;
        if ((unsigned)expert[k] >= (unsigned)E) expert[k] = -1;
      }
      for (int e = lane; e < E; e += 32) mine[e] = 0;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        const bool in = expert[k] >= 0;
        unsigned same = __ballot_sync(0xffffffffu, in);
#pragma unroll 5
        for (int b = 0; b < bits; ++b) {
          const bool one = (expert[k] >> b) & 1;
          const unsigned ones = __ballot_sync(0xffffffffu, one);
          same &= one ? ones : ~ones;
        }
        const int before = __popc(same & ((1u << lane) - 1));
        int seen = 0;
        if (in) seen = mine[expert[k]];
        __syncwarp();
        if (in && before == 0) mine[expert[k]] = (uint16_t)(seen + __popc(same));
        __syncwarp();
        at[k] = seen + before;
      }
    }
    __syncthreads();
    int sum = 0;
    if (t < E) {
#pragma unroll 8
      for (int w = 0; w < WARPS; ++w) {
        const int v = disp_counts[w * E + t];
        disp_counts[w * E + t] = (uint16_t)sum;
        sum += v;
      }
    }
    return sum;   // of expert t in this round
  };

  int own = 0;
  s_early[t] = 0;
  if (once) {
    own = rank_round(i0);
    s_total[t] = own;
  } else {
    s_total[t] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = i0 + t; i < i1; i += kDispThreads) {
      const int e = __ldg(a.idx + i);
      if ((unsigned)e < (unsigned)E) {
        atomicAdd(&s_total[e], 1);
        if (i < p0) atomicAdd(&s_early[e], 1);
      }
    }
  }
  cluster_sync();
  int all = 0, before = s_early[t];
  if (t < E) {
    const uint32_t here = smem_addr(&s_total[t]);
    int v[kDispMaxCtas];
#pragma unroll
    for (int c = 0; c < kDispMaxCtas; ++c)
      v[c] = c < ctas ? ld_cluster_s32(cluster_map(here, c)) : 0;
#pragma unroll
    for (int c = 0; c < kDispMaxCtas; ++c) {
      if (c < rank) before += v[c];
      all += v[c];
    }
  }
  const int end = disp_scan(all, s_warp);
  s_next[t] = end - all + before;
  if (blockIdx.x == 0) {
    if (t < E) a.offsets[t] = end - all;
    if (t == E - 1) a.offsets[E] = end;
  }
  if (t == E - 1) s_end = end;
  cluster_sync();   // every CTA has read the counts (and s_end, s_next are written)
  // past the last entry, where choices name no expert
  for (int i = s_end + blockIdx.x * kDispThreads + t; i < a.n; i += gridDim.x * kDispThreads)
    a.rows[i] = -1;

  for (int r0 = p0; r0 < p1; r0 += ROUND) {
    if (!once) own = rank_round(r0);
    const int first = disp_scan(own, s_warp) - own;   // its place in the round
    if (t < E) {
      s_base[t] = s_next[t] - first;
#pragma unroll 8
      for (int w = 0; w < WARPS; ++w) disp_counts[w * E + t] += (uint16_t)first;
    }
    if (t == E - 1) s_end = first + own;   // entries of this round
    __syncthreads();
    if (warp < WARPS) {
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        const int i = r0 + warp * (ITER * 32) + 32 * k + lane;
        if (i >= p1) continue;
        int slot = -1;
        if (expert[k] >= 0) {
          const int p = mine[expert[k]] + at[k];
          slot = s_base[expert[k]] + p;
          s_token[p] = (int)((unsigned)i / (unsigned)a.top_k);
          s_expert[p] = (uint16_t)expert[k];
        }
        a.slots[i] = slot;
      }
    }
    __syncthreads();
    for (int p = t; p < s_end; p += kDispThreads) a.rows[s_base[s_expert[p]] + p] = s_token[p];
    if (t < E) s_next[t] += own;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Combine: a thread's 8 columns of a token, the experts' rows loaded ahead of
// their sums, which are taken in the order of j.  HBM bounds it: 8 rows of each of
// 4,096 tokens, 7,168 columns, in 88 us, 6.7 TB/s.
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
  pdl_wait_prerequisites();
  pdl_launch_dependents();
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
