// Expert routing from logits: one warp per row, expert lane + 32 i in
// register i.
#pragma once

#include "kv_cache.cuh"
#include "topk.cuh"

namespace moe {

constexpr int kRouteWarps = 4;

struct RouteArgs {
  const void* logits;
  long long row_stride, rows;
  const float* bias;
  int32_t* idx;
  float* w;
  int dtype, E, k, softmax, groups, topk_groups, group_top, renorm;
  float scale;
};

// Order-preserving image of a score, NaN below everything (0; -infinity maps above it).
__device__ __forceinline__ uint32_t route_key(float v) {
  return v == v ? float_order_bits(v) : 0u;
}

__device__ __forceinline__ float route_load(const RouteArgs& a, long long row, int e) {
  const long long i = row * a.row_stride + e;
  if (a.dtype == MOE_DTYPE_F32) return static_cast<const float*>(a.logits)[i];
  const uint16_t u = static_cast<const uint16_t*>(a.logits)[i];
  return a.dtype == MOE_DTYPE_F16 ? f16_lo(u) : bf16_bits_to_f32(u);
}

// N: registers a lane (E <= 32 N).
template <int N>
static __global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * kRouteWarps + warp;
  __shared__ float s_sel[kRouteWarps][N * 32];
  if (row >= a.rows) return;
  float s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    s[i] = e < a.E ? route_load(a, row, e) : -INFINITY;
  }
  if (a.softmax) {
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, s[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = expf(s[i] - m);
      z += s[i];
    }
    z = warp_sum(z);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = z == 0.f ? 0.f : s[i] / z;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = topk_score(s[i]);
  }
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < a.E ? route_key(s[i] + (a.bias ? __ldg(a.bias + e) : 0.f)) : 0u;
  }
  unsigned allowed = 0xffffffffu;
  const int size = a.E / a.groups;
  if (a.groups > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E) s_sel[warp][e] = s[i] + (a.bias ? __ldg(a.bias + e) : 0.f);
    }
    __syncwarp();
    uint32_t gk = 0;
    if (lane < a.groups) {
      float b1 = -INFINITY, b2 = -INFINITY;
      for (int j = 0; j < size; ++j) {
        float v = s_sel[warp][lane * size + j];
        if (v != v) v = -INFINITY;
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      gk = float_order_bits(a.group_top == 2 && size > 1 ? b1 + b2 : b1);
    }
    int rank = 0;   // groups before this one
    for (int g = 0; g < a.groups; ++g) {
      const uint32_t o = __shfl_sync(0xffffffffu, gk, g);
      rank += o > gk || (o == gk && g < lane);
    }
    allowed = __ballot_sync(0xffffffffu, lane < a.groups && rank < a.topk_groups);
  }
  // the k best, one at a time: the warp's largest key, then its lowest expert
  unsigned taken = 0;   // registers of this lane already out
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    if (e >= a.E || !((allowed >> (e / size)) & 1u || a.groups == 1)) taken |= 1u << i;
  }
  float mine = 0.f, sum = 0.f;
  int mine_e = 0;
  for (int j = 0; j < a.k; ++j) {
    uint32_t bk = 0;
    int be = 0x7FFFFFFF;
#pragma unroll
    for (int i = N - 1; i >= 0; --i) {
      if (!((taken >> i) & 1u) && (key[i] >= bk)) {
        bk = key[i];
        be = lane + 32 * i;
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
    const int e = __reduce_min_sync(0xffffffffu, bk == top ? be : 0x7FFFFFFF);
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (lane + 32 * i == e) {
        taken |= 1u << i;
        v = s[i];
      }
    }
    v = __shfl_sync(0xffffffffu, v, e & 31);
    sum += v;
    if (lane == j) {
      mine = v;
      mine_e = e;
    }
  }
  if (lane < a.k) {
    a.idx[row * a.k + lane] = mine_e;
    a.w[row * a.k + lane] =
        a.scale * (a.renorm ? (sum == 0.f ? 0.f : mine / sum) : mine);
  }
}

}  // namespace moe
