// Attention over the 8-bit cache.
#pragma once

#include "kv_cache.cuh"

namespace moe {

struct AttnArgs {
  KvView c;
  const uint16_t* q;
  long long q_ts, q_hs;
  uint16_t* out;
  long long o_ts, o_hs;
  float* lse;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  const int* q_start;
  int f16, rows, n_tokens, heads, group, max_blocks, causal, window;
  float scale_log2;   // scale * log2(e)
};

// One row's queries: tokens [tok, tok + n), seq cached tokens.
struct AttnRow {
  int tok, n, seq;
};

__device__ __forceinline__ AttnRow attn_row(const AttnArgs& a, int r) {
  AttnRow w;
  w.tok = min(max(a.q_start[r], 0), a.n_tokens);
  w.n = min(max(a.q_start[r + 1], w.tok), a.n_tokens) - w.tok;
  const long long cap = (long long)a.max_blocks << a.c.bs_log2;
  w.seq = (int)min((long long)max(a.seq_lens[r], 0), cap);
  return w;
}

// Keys [lo, hi) that query i of the row sees.
__device__ __forceinline__ void attn_seen(const AttnArgs& a, const AttnRow& w, int i, int& lo,
                                          int& hi) {
  const int p = w.seq - w.n + i;
  hi = a.causal ? max(0, min(w.seq, p + 1)) : w.seq;
  lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
}

// The simple kernel: one warp per (token, query head), a lane per key for the
// scores, the lanes across the head dimension for the sum of values.  Grid:
// (tokens, heads / warps).
constexpr int kAttnSimpleWarps = 4;

template <int D>
static __global__ void __launch_bounds__(32 * kAttnSimpleWarps) kv_attention_simple(
    const AttnArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = blockIdx.x, h = blockIdx.y * kAttnSimpleWarps + warp;
  __shared__ float s_q[kAttnSimpleWarps][D];
  if (h >= a.heads) return;
  // the row whose tokens hold this one: the last with q_start <= tok
  int lo_r = 0, hi_r = a.rows;
  while (hi_r - lo_r > 1) {
    const int mid = (lo_r + hi_r) >> 1;
    if (a.q_start[mid] <= tok) lo_r = mid;
    else hi_r = mid;
  }
  const AttnRow w = attn_row(a, lo_r);
  if (tok < w.tok || tok >= w.tok + w.n) return;
  int lo, hi;
  attn_seen(a, w, tok - w.tok, lo, hi);
  const uint16_t* q = a.q + tok * a.q_ts + h * a.q_hs;
  for (int j = lane; j < D; j += 32)
    s_q[warp][j] = a.f16 ? f16_lo(q[j]) : bf16_bits_to_f32(q[j]);
  __syncwarp();
  const int kh = h / a.group, bs = 1 << a.c.bs_log2;
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int j0 = lo & ~31; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    int id = -1;
    if (j >= lo && j < hi) {
      id = a.table[lo_r * a.table_stride + (j >> a.c.bs_log2)];
      if (id < 0 || id >= a.c.n_blocks) id = -1;
    }
    if (id >= 0) {
      const uint8_t* kp = a.c.k + id * a.c.bstride + kh * a.c.hstride + (j & (bs - 1)) * a.c.tstride;
      float acc = 0.f;
      for (int d = 0; d < D; d += 4) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(kp + d);
        const uint32_t x = e4m3x2_to_f16x2(u & 0xFFFFu), y = e4m3x2_to_f16x2(u >> 16);
        acc = fmaf(s_q[warp][d], f16_lo(x), acc);
        acc = fmaf(s_q[warp][d + 1], f16_hi(x), acc);
        acc = fmaf(s_q[warp][d + 2], f16_lo(y), acc);
        acc = fmaf(s_q[warp][d + 3], f16_hi(y), acc);
      }
      s = acc * (a.scale_log2 * pow2f(kv_exp(a.c.ks[id * a.c.sstride + kh])));
    }
    const bool seen = id >= 0;
    const float mx = fmaxf(m, warp_max(s));
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float down = exp2f(m - ref);
    const float p = seen ? exp2f(s - ref) : 0.f;
    m = mx;
    l = l * down + warp_sum(p);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= down;
    for (int t = 0; t < 32; ++t) {
      const int tid = __shfl_sync(0xffffffffu, id, t);
      if (tid < 0) continue;   // not seen: its value does not enter
      const float pv = __shfl_sync(0xffffffffu, p, t) *
                       pow2f(kv_exp(a.c.vs[tid * a.c.sstride + kh]));
      const uint8_t* vp = a.c.v + tid * a.c.bstride + kh * a.c.hstride +
                          ((j0 + t) & (bs - 1)) * a.c.tstride;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        o[i] = fmaf(pv, f16_lo(e4m3x2_to_f16x2(vp[lane + 32 * i])), o[i]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // NaN stays NaN
  uint16_t* out = a.out + tok * a.o_ts + h * a.o_hs;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    out[lane + 32 * i] = (uint16_t)pack16(o[i] * inv, 0.f, a.f16);
  if (a.lse && lane == 0) a.lse[(long long)tok * a.heads + h] =
      l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace moe
