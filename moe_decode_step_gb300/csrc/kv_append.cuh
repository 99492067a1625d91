// New keys and values into the 8-bit cache.
//
// The tokens a step writes into one block share its scale, so the unit of
// work is a group: the consecutive tokens of one block, found at its first
// token (the leader: the slot before it lies in another block).  A warp takes
// one group of one head and one side: the largest magnitude, the exponent,
// then the codes; where the block held tokens and its exponent grows, their
// codes are rounded to the new scale first.
#pragma once

#include "kv_cache.cuh"

namespace moe {

constexpr int kAppendWarps = 8;
constexpr int kAppendChunk = 16;   // slots whose leaders one CTA looks after

struct AppendArgs {
  KvView c;
  const uint16_t* src[2];
  long long ts[2], hs[2];   // elements
  int f16;
  const int* slot;
  int n_tokens;
};

__device__ __forceinline__ int append_block_of(const AppendArgs& a, int slot) {
  return slot >= 0 && (slot >> a.c.bs_log2) < a.c.n_blocks ? slot >> a.c.bs_log2 : -1;
}

// One warp: tokens [t0, t0 + n) of head h, side s (0 K, 1 V) into block b
// from offset off.
template <int D>
__device__ __forceinline__ void append_group(const AppendArgs& a, int s, int h, int b, int off,
                                             int t0, int n, int lane) {
  constexpr int LPT = D / 8;          // lanes a token (16 bytes each)
  constexpr int TPW = 32 / LPT;       // tokens a pass
  const int sub = lane / LPT, part = lane % LPT;
  const uint16_t* src = a.src[s] + h * a.hs[s] + part * 8;
  uint8_t* dst = (s ? a.c.v : a.c.k) + b * a.c.bstride + h * a.c.hstride + part * 8;
  uint8_t* sp = (s ? a.c.vs : a.c.ks) + b * a.c.sstride + h;
  float amax = 0.f;
  for (int i = sub; i < n; i += TPW) {
    const uint4 w = *reinterpret_cast<const uint4*>(src + (t0 + i) * a.ts[s]);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack16(u[j], a.f16);
      const float x = fabsf(f.x), y = fabsf(f.y);
      if (x <= 3.4028235e38f) amax = fmaxf(amax, x);   // finite values only
      if (y <= 3.4028235e38f) amax = fmaxf(amax, y);
    }
  }
  int e = kv_block_exp(warp_max(amax));
  if (off > 0) {
    const int old = kv_exp(*sp);
    if (old >= e) {
      e = old;
    } else {
      const float down = pow2f(old - e);
      for (int i = sub; i < off; i += TPW) {
        uint2* p = reinterpret_cast<uint2*>(dst + i * a.c.tstride);
        uint2 v = *p;
        uint32_t r[2] = {v.x, v.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t lo, hi;
          e4m3x4_to_f16x2(r[j], lo, hi);
          r[j] = f32x2_to_e4m3x2(f16_lo(lo) * down, f16_hi(lo) * down) |
                 f32x2_to_e4m3x2(f16_lo(hi) * down, f16_hi(hi) * down) << 16;
        }
        *p = make_uint2(r[0], r[1]);
      }
    }
  }
  __syncwarp();
  if (lane == 0) *sp = (uint8_t)(e + 127);
  const float inv = pow2f(-e);
  for (int i = sub; i < n; i += TPW) {
    const uint4 w = *reinterpret_cast<const uint4*>(src + (t0 + i) * a.ts[s]);
    const float2 f0 = unpack16(w.x, a.f16), f1 = unpack16(w.y, a.f16), f2 = unpack16(w.z, a.f16),
                 f3 = unpack16(w.w, a.f16);
    const uint32_t lo = f32x2_to_e4m3x2(f0.x * inv, f0.y * inv) |
                        f32x2_to_e4m3x2(f1.x * inv, f1.y * inv) << 16;
    const uint32_t hi = f32x2_to_e4m3x2(f2.x * inv, f2.y * inv) |
                        f32x2_to_e4m3x2(f3.x * inv, f3.y * inv) << 16;
    *reinterpret_cast<uint2*>(dst + (off + i) * a.c.tstride) = make_uint2(lo, hi);
  }
}

template <int D>
static __global__ void __launch_bounds__(32 * kAppendWarps) kv_append_kernel(const AppendArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * kAppendChunk;
  const int h = blockIdx.y >> 1, s = blockIdx.y & 1;
  // leaders among this chunk's slots (every warp finds them for itself)
  const int t = t0 + lane;
  int mine = -1, slot = -1;
  if (lane < kAppendChunk && t < a.n_tokens) {
    slot = a.slot[t];
    mine = append_block_of(a, slot);
    if (mine >= 0 && t > 0 && append_block_of(a, a.slot[t - 1]) == mine) mine = -1;
  }
  unsigned leaders = __ballot_sync(0xffffffffu, mine >= 0);
  for (int k = 0; leaders; ++k, leaders &= leaders - 1) {
    if (k % kAppendWarps != warp) continue;
    const int l = __ffs(leaders) - 1;
    const int b = __shfl_sync(0xffffffffu, mine, l);
    const int off = __shfl_sync(0xffffffffu, slot, l) & ((1 << a.c.bs_log2) - 1);
    // the group's length: tokens after the leader in the same block
    const int room = min((1 << a.c.bs_log2) - off, a.n_tokens - (t0 + l));
    int n = 0;
    while (n < room) {
      const int i = n + lane;
      const bool in = i < room && append_block_of(a, a.slot[t0 + l + i]) == b;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (m != 0xffffffffu) {
        n += __ffs(~m) - 1;
        break;
      }
      n += 32;
    }
    append_group<D>(a, s, h, b, off, t0 + l, min(n, room), lane);
  }
}

}  // namespace moe
