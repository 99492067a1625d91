// Expert routing from logits: one warp per row.
//
// A row is E logits read once and k indices and weights written, a few hundred
// instructions against E * 4 bytes, so issue slots bound long calls and the
// chain of k selections short ones.  Lane l holds experts 4l .. 4l + 3 of every
// 128 (one 16-byte load; rows that do not allow it: expert l of every 32), and
// of these only its two best in order: a selection is then the warp's largest
// head (redux) and the lowest expert among equals (redux), after which one lane
// moves up; a lane whose two are gone looks through the rest again, once a row
// or so.  Selection compares the scores that are written: the k of them are
// computed again, by the same operations, from the logits (the layer's own
// router does the same, so both pick the same experts).  Groups whose size is
// a power of two find their two best by shuffles, others through shared memory.
// Measured: 32,768 rows of 256 experts, 8 of the 4 best of 8 groups: 32.8 us,
// 1.1 TB/s; issue slots bound it (85% busy, 951 instructions a row; approximate
// exponentials and reciprocals 30.2 us, but neighbours changed places where
// their scores differ by less than a few 1e-7).  64 rows of 896, 16 best: 14 to
// 17 us a call, most of it the host's time.
#pragma once

#include "kv_cache.cuh"
#include "topk.cuh"

namespace moe {

constexpr int kRouteWarps = 8;

struct RouteArgs {
  const void* logits;
  long long row_stride, rows;
  const float* bias;
  int32_t* idx;
  float* w;
  int dtype, E, k, softmax, groups, topk_groups, group_top, renorm;
  float scale;
};

// Order-preserving image of a score: NaN 1, everything else above; 0 is left
// for experts that are out.
__device__ __forceinline__ uint32_t route_key(float v) {
  return v == v ? float_order_bits(v) : 1u;
}

__device__ __forceinline__ float route_load(const RouteArgs& a, long long row, int e) {
  const long long i = row * a.row_stride + e;
  if (a.dtype == MOE_DTYPE_F32) return __ldg(static_cast<const float*>(a.logits) + i);
  const uint16_t u = __ldg(static_cast<const uint16_t*>(a.logits) + i);
  return a.dtype == MOE_DTYPE_F16 ? f16_lo(u) : bf16_bits_to_f32(u);
}

// The two best of (a1, a2) and (b1, b2).
__device__ __forceinline__ void route_merge2(uint32_t& a1, uint32_t& a2, uint32_t b1,
                                             uint32_t b2) {
  a2 = max(min(a1, b1), max(a2, b2));
  a1 = max(a1, b1);
}
// The score of a key; -inf for NaN and for experts that are out.
__device__ __forceinline__ float route_score(uint32_t key) {
  return key > 1u ? __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key) : -INFINITY;
}

// CH: chunks of 32 V experts a row has at most; V: experts of a chunk a lane.
template <int CH, int V>
static __global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
  constexpr int N = CH * V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * kRouteWarps + warp;
  if (row >= a.rows) return;
  auto expert = [&](int i) { return 32 * V * (i / V) + V * lane + i % V; };

  // ---- scores ----
  float s[N];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = 32 * V * c + V * lane;
    if (V == 4 && e + 3 < a.E) {
      const long long at = row * a.row_stride + e;
      if (a.dtype == MOE_DTYPE_F32) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at));
        s[V * c] = f.x;
        s[V * c + 1 % V] = f.y;
        s[V * c + 2 % V] = f.z;
        s[V * c + 3 % V] = f.w;
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + at));
        const float2 f = unpack16(u.x, a.dtype == MOE_DTYPE_F16);
        const float2 g = unpack16(u.y, a.dtype == MOE_DTYPE_F16);
        s[V * c] = f.x;
        s[V * c + 1 % V] = f.y;
        s[V * c + 2 % V] = g.x;
        s[V * c + 3 % V] = g.y;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) s[V * c + v] = e + v < a.E ? route_load(a, row, e + v) : -INFINITY;
    }
  }
  float m = 0.f, inv = 0.f;
  if (a.softmax) {
    float z = 0.f;
    m = -INFINITY;
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
    inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __fmul_rn(s[i], inv);   // rounded, as it is written
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = topk_score(s[i]);
  }
  if (a.bias) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = 32 * V * c + V * lane;
      if (V == 4 && e + 3 < a.E) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(a.bias + e));
        s[V * c] += f.x;
        s[V * c + 1 % V] += f.y;
        s[V * c + 2 % V] += f.z;
        s[V * c + 3 % V] += f.w;
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (e + v < a.E) s[V * c + v] += __ldg(a.bias + e + v);
      }
    }
  }
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = route_key(s[i]);
  if (a.E != 32 * N) {
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = expert(i) < a.E ? key[i] : 0u;
  }

  // ---- groups ----
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    const bool two = a.group_top == 2 && size > 1;
    float score = -INFINITY;   // lane g: of group g
    const bool pow2 = V == 4 && (size & (size - 1)) == 0 && size >= 4 && size <= 128;
    if (pow2) {
      const int per = size >> 2;                       // lanes a group
      const int from = lane * size;                    // group `lane`'s first expert
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint32_t* x = key + V * c;
        uint32_t t1 = max(x[0], x[1 % V]), t2 = min(x[0], x[1 % V]);
        route_merge2(t1, t2, max(x[2 % V], x[3 % V]), min(x[2 % V], x[3 % V]));
        for (int o = 1; o < per; o <<= 1) {
          const uint32_t o1 = __shfl_xor_sync(0xffffffffu, t1, o);
          const uint32_t o2 = __shfl_xor_sync(0xffffffffu, t2, o);
          route_merge2(t1, t2, o1, o2);
        }
        const float f1 = route_score(t1);
        const float g =
            __shfl_sync(0xffffffffu, two ? f1 + route_score(t2) : f1, (from >> 2) & 31);
        if (lane < a.groups && (from >> 7) == c) score = g;
      }
    } else {
      extern __shared__ uint32_t route_smem[];
      uint32_t* sel = route_smem + warp * N * 32;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (expert(i) < a.E) sel[expert(i)] = key[i];
      __syncwarp();
      if (lane < a.groups) {
        uint32_t t1 = 0u, t2 = 0u;
        for (int j = 0; j < size; ++j) route_merge2(t1, t2, sel[lane * size + j], 0u);
        score = two ? route_score(t1) + route_score(t2) : route_score(t1);
      }
    }
    const uint32_t gk = lane < a.groups ? route_key(score) : 0u;
    int rank = 0;   // groups before this one
#pragma unroll 8
    for (int g = 0; g < a.groups; ++g) {
      const uint32_t o = __shfl_sync(0xffffffffu, gk, g);
      rank += o > gk || (o == gk && g < lane);
    }
    const unsigned in = __ballot_sync(0xffffffffu, lane < a.groups && rank < a.topk_groups);
    if (pow2) {
      const int shift = 31 - __clz(size);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const bool keep = (in >> (((32 * V * c + V * lane) >> shift) & 31)) & 1u;
#pragma unroll
        for (int v = 0; v < V; ++v) key[V * c + v] = keep ? key[V * c + v] : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (expert(i) < a.E && !((in >> (expert(i) / size)) & 1u)) key[i] = 0u;
    }
  }

  // ---- the k best ----
  uint32_t b1 = 0u, b2 = 0u;   // the lane's best two left, and which experts
  int e1 = 0, e2 = 0;          // (less V * lane)
#pragma unroll
  for (int i = 0; i < N; ++i) {   // ascending experts: the first of equals stays ahead
    const uint32_t x = key[i];
    const bool first = x > b1, second = x > b2;
    const int e = 32 * V * (i / V) + i % V;
    b2 = first ? b1 : second ? x : b2;
    e2 = first ? e1 : second ? e : e2;
    b1 = first ? x : b1;
    e1 = first ? e : e1;
  }
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, b1);
    const int ex = e1 + V * lane;
    const int e = __reduce_min_sync(0xffffffffu, b1 == top ? ex : 0x7FFFFFFF);
    mine = lane == j ? e : mine;
    if (ex == e && b1 == top) {
      const int last = e1;
      b1 = b2;
      e1 = e2;
      b2 = 0u;
      if (b1 == 0u) {   // the best of those after the one just taken
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int n = 32 * V * (i / V) + i % V;
          if ((key[i] < top || (key[i] == top && n > last)) && key[i] > b1) {
            b1 = key[i];
            e1 = n;
          }
        }
      }
    }
  }

  // ---- weights of the selected, from their logits ----
  float v = 0.f;
  if (lane < a.k) {
    const float x = route_load(a, row, mine);
    v = a.softmax ? __fmul_rn(expf(x - m), inv) : topk_score(x);
  }
  const float sum = warp_sum(v);
  if (lane < a.k) {
    a.idx[row * a.k + lane] = mine;
    a.w[row * a.k + lane] = a.scale * (a.renorm ? (sum == 0.f ? 0.f : v / sum) : v);
  }
}

}  // namespace moe
