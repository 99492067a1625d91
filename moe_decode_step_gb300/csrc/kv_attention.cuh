// Attention over the 8-bit cache: arguments, masks and the kernel for few
// query rows per KV head.
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
  float* partial;     // two slots per CTA
  int* desc;          // per CTA: the split tile it begins
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
  lo = a.window > 0 ? (int)max(0ll, (long long)p - a.window + 1) : 0;
}

// ---------------------------------------------------------------------------
// Few query rows per KV head (decode, short verify steps): mma.sync
// ---------------------------------------------------------------------------
// The rows of one KV head (query i, head of the group: row i * group + head)
// form tiles of 16, the M of one m16n8k16.  A call reads every visible byte of
// the cache once per tile and does 4 * 16 * D operations on its 2 * D bytes a
// token: at 16 rows 32 operations a byte, far below the tensor cores' balance,
// so HBM bounds it and the layout serves the loads.
//
// Work: strips of 32 tokens of (row of the batch, KV head, tile), ordered in
// that order; CTA i takes strips [i * per, (i + 1) * per), so that ragged
// lengths leave every SM the same bytes.  Inside a CTA the strips go round
// the warps, each with its own running maximum and sums, joined in shared
// memory at the end of a tile; a tile cut by a CTA boundary leaves partial
// sums in the workspace, which the second kernel joins in CTA order (results
// do not depend on timing).
//
// Loads: each thread copies (cp.async) exactly the 16-byte pieces that it
// feeds to its own MMAs, into a ring of its own in shared memory, so a strip
// needs no barrier at all; the ring only deepens the loads in flight (D = 128:
// 8 warps x 2 strips x 8 KB = 128 KB an SM; 1 us of latency at 6.7 TB/s needs
// 44 KB).  The contraction order of either product is free, so the pieces
// need no shuffling: in each half of a strip (16 tokens) lane (g, t) = (lane /
// 4, lane % 4) holds, for the scores, 16 consecutive dims (from 16 t, and from
// 64 + 16 t) of keys g and g + 8, and for the values CH = D / 8 consecutive
// dims (from CH g) of tokens 2t, 2t + 1, 2t + 8, 2t + 9, byte-transposed in
// registers.  Codes become f16 exactly (cvt.rn.f16x2.e4m3x2); queries enter
// as f16 scaled per row by a power of two, which keeps all of bf16's 8 bits.
// What bounds the kernel beside HBM is instruction issue (a strip of 8 KB is
// 64 MMAs, 128 conversions and about as much again of everything else), so a
// strip is two halves long: one maximum, one vote and twice the independent
// MMAs for 32 tokens.
//
// Scales: a half lies in one block, so one exponent ek scales its scores and
// one ev its values.  With t = score * log2(e) + ev the weights 2^(t - M), M
// the running maximum of t, are the values' true relative sizes: in (0, 1],
// which f16 holds, whatever the spread of the block scales.  The
// denominator takes the same weights times 2^-ev in fp32 (|ev| <= 60 keeps
// them inside its range).
constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;

template <int D>
struct DecShape {
  static constexpr int CH = D / 8;                 // value dims a lane holds per token
  static constexpr int KP = D / 32;                // 16-byte key pieces a lane and half (2 keys)
  static constexpr int VP = 4 * CH / 16;           // the same for values (4 tokens)
  static constexpr int HALF = 32 * 16 * (KP + VP); // bytes of one warp's half strip
  static constexpr int STAGES = D == 64 ? 6 : 3;
  static constexpr int RS = D + 8;                 // row stride of the join buffer (floats)
  // ring, join buffer (4 rows a round), m, l and factor of every warp's rows,
  // m, l and score factor of the tile's, queries
  static constexpr int SMEM = kDecWarps * (STAGES * 2 * HALF + 4 * RS * 4 + 3 * 16 * 4) +
                              3 * 16 * 4 + 16 * D * 2;
};

// One slot of partial sums: O [16][D] in the join buffer's column order, then
// M [16] and l [16].
template <int D>
constexpr int kDecSlot = 16 * D + 32;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? BYTES : 0;   // 0: the destination is zero-filled, src is not read
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row's share of the work: M tiles of 16 rows, S strips each, from strip s0.
struct DecRow {
  AttnRow w;
  int M, S, s0;
};

__device__ __forceinline__ DecRow dec_row(const AttnArgs& a, int r) {
  DecRow x;
  x.w = attn_row(a, r);
  x.M = (int)(((long long)x.w.n * a.group + 15) >> 4);
  int lo, hi, unused;
  attn_seen(a, x.w, 0, lo, unused);
  attn_seen(a, x.w, x.w.n - 1, unused, hi);
  x.s0 = lo >> 5;
  x.S = max(1, ((hi + 31) >> 5) - x.s0);   // a tile that sees nothing still writes its zeros
  return x;
}

__device__ __forceinline__ long long dec_units(const AttnArgs& a, const DecRow& x) {
  return (long long)a.c.heads * x.M * x.S;
}

// Position in the strip order: strip s of tile m of KV head h of row r.
struct DecCursor {
  int r, h, m, s;
  DecRow x;
};

// To the next tile.
__device__ __forceinline__ void dec_next_tile(const AttnArgs& a, DecCursor& c) {
  c.s = 0;
  if (++c.m < c.x.M) return;
  c.m = 0;
  if (++c.h < a.c.heads) return;
  c.h = 0;
  do {
    if (++c.r >= a.rows) return;
    c.x = dec_row(a, c.r);
  } while (c.x.M == 0);
}

// This CTA's strips [u0, u0 + n) and its cursor at u0; every thread calls.
// Also `per`.  The sums over the rows are made by every CTA for itself.
__device__ __forceinline__ void dec_schedule(const AttnArgs& a, long long& u0, long long& n,
                                             long long& per, DecCursor& cur) {
  __shared__ long long s_sum[kDecWarps];
  __shared__ long long s_left;
  __shared__ int s_row;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int chunk = (a.rows + kDecThreads - 1) / kDecThreads;
  const int r0 = min(a.rows, t * chunk), r1 = min(a.rows, r0 + chunk);
  long long sum = 0;
  for (int r = r0; r < r1; ++r) sum += dec_units(a, dec_row(a, r));
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  long long total = 0, base = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w == warp) base = total;
    total += s_sum[w];
  }
  per = max((total + gridDim.x - 1) / gridDim.x, (long long)kDecWarps);
  u0 = per * blockIdx.x;
  n = min(per, total - u0);
  long long before = base + inc - sum;
  if (n > 0 && u0 >= before && u0 < before + sum) {
    int r = r0;
    for (;; ++r) {
      const long long k = dec_units(a, dec_row(a, r));
      if (u0 < before + k) break;
      before += k;
    }
    s_row = r;
    s_left = u0 - before;
  }
  __syncthreads();
  if (n <= 0) return;
  cur.r = s_row;
  cur.x = dec_row(a, cur.r);
  const long long left = s_left;
  cur.s = (int)(left % cur.x.S);
  const int hm = (int)(left / cur.x.S);
  cur.m = hm % cur.x.M;
  cur.h = hm / cur.x.M;
}

// What one warp loads ahead.  Block ids and scales are two dependent misses to
// HBM a half strip; they are asked for in batches of 16 strips, lane i for the
// i-th half of the batch, a whole batch before the first of them is used.
struct DecLoader {
  int r;              // the lane's position in the strip order: row,
  long long idx;      // strip of the row
  DecRow x;
  long long left;     // strips of the CTA from the lane's on
  // the half of the current batch: bytes from the cache's start, tokens cached
  long long at;
  int cached;
  uint32_t sc_now, sc_before;   // its scales, and those of the batch before:
                                // ek + 128 | ev + 128 << 8 | block exists << 16
  // the half of the next batch
  int id, head, offset, next_cached;
  uint32_t sk, sv;
  int k;              // strips fetched
  uint32_t slot;      // ring slot of the next one
};

__device__ __forceinline__ void dec_lane_lookup(const AttnArgs& a, DecLoader& l, int lane) {
  l.id = -1;
  l.head = l.offset = l.next_cached = 0;
  if (l.left <= 0) return;
  const int s = (int)(l.idx % l.x.S);
  l.head = (int)(l.idx / l.x.S) / l.x.M;
  const int p0 = ((l.x.s0 + s) << 5) + ((lane & 1) << 4);
  l.next_cached = min(max(l.x.w.seq - p0, 0), 16);
  if (l.next_cached) l.id = __ldg(a.table + l.r * a.table_stride + (p0 >> a.c.bs_log2));
  l.offset = p0 & ((1 << a.c.bs_log2) - 1);
}
__device__ __forceinline__ void dec_lane_advance(const AttnArgs& a, DecLoader& l, int n) {
  l.left -= n;
  if (l.left <= 0) return;
  l.idx += n;
  for (;;) {
    const long long units = dec_units(a, l.x);
    if (l.idx < units) return;
    l.idx -= units;
    l.x = dec_row(a, ++l.r);
  }
}
__device__ __forceinline__ void dec_lane_scales(const AttnArgs& a, DecLoader& l) {
  if (l.id >= a.c.n_blocks) l.id = -1;
  const long long at = (long long)max(l.id, 0) * a.c.sstride + l.head;
  l.sk = __ldg(a.c.ks + at);
  l.sv = __ldg(a.c.vs + at);
}
// The next batch becomes the current one (but for its scales).
__device__ __forceinline__ void dec_lane_take(const AttnArgs& a, DecLoader& l) {
  l.cached = l.id >= 0 ? l.next_cached : 0;
  l.at = (long long)max(l.id, 0) * a.c.bstride + (long long)l.head * a.c.hstride +
         (long long)l.offset * a.c.tstride;
}
__device__ __forceinline__ uint32_t dec_pack_scales(bool exists, uint32_t sk, uint32_t sv) {
  return (uint32_t)(kv_exp(sk) + 128) | (uint32_t)(kv_exp(sv) + 128) << 8 |
         (exists ? 1u << 16 : 0u);
}

// Byte offsets of a lane's pieces in a half: keys g, g + 8 and tokens 2t, 2t + 8.
struct DecOffsets {
  long long k0, k1, v0, v1;
};

template <int D>
__device__ __forceinline__ void dec_fetch(const AttnArgs& a, DecLoader& l, const DecOffsets& f,
                                          int strips, uint32_t ring, int lane) {
  using Sh = DecShape<D>;
  if (l.k < strips) {
    const int b = l.k & 15;
    if (b == 0 && l.k > 0) {
      dec_lane_take(a, l);
      l.sc_before = l.sc_now;
      l.sc_now = dec_pack_scales(l.id >= 0, l.sk, l.sv);
      dec_lane_advance(a, l, 16 * kDecWarps);
      dec_lane_lookup(a, l, lane);
    } else if (b == 8) {
      dec_lane_scales(a, l);
    }
    const long long ts = a.c.tstride;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int cached = __shfl_sync(0xffffffffu, l.cached, 2 * b + half);
      const long long at = __shfl_sync(0xffffffffu, l.at, 2 * b + half);
      const uint8_t* kp = a.c.k + at;
      const uint8_t* vp = a.c.v + at;
      const uint32_t dst = ring + l.slot * (2 * Sh::HALF) + half * Sh::HALF + lane * 16;
      const int g = lane >> 2, t = lane & 3;
      const uint8_t* src[6] = {kp + f.k0, kp + f.k1, vp + f.v0, vp + f.v0 + ts, vp + f.v1,
                               vp + f.v1 + ts};
      const int tok[6] = {g, g + 8, 2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
      if (cached == 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            cp_async<16>(dst + (i * (D / 64) + c) * 512, src[i] + c * 64, true);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) cp_async<16>(dst + (Sh::KP + i) * 512, src[2 + i], true);
          else cp_async<8>(dst + (Sh::KP + (i >> 1)) * 512 + (i & 1) * 8, src[2 + i], true);
        }
      } else {   // a row's end: what is not cached is zero-filled and not read
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            cp_async<16>(dst + (i * (D / 64) + c) * 512,
                         tok[i] < cached ? src[i] + c * 64 : a.c.k, tok[i] < cached);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = tok[2 + i] < cached;
          const uint8_t* p = in ? src[2 + i] : a.c.v;
          if constexpr (D == 128) cp_async<16>(dst + (Sh::KP + i) * 512, p, in);
          else cp_async<8>(dst + (Sh::KP + (i >> 1)) * 512 + (i & 1) * 8, p, in);
        }
      }
    }
    ++l.k;
    l.slot = l.slot + 1 == Sh::STAGES ? 0 : l.slot + 1;
  }
  cp_async_commit();
}

// Packed scales of a half of the warp's strip k, at most a ring behind the fetches.
__device__ __forceinline__ uint32_t dec_scales(const DecLoader& l, int k, int half) {
  const uint32_t v = (k >> 4) == ((l.k - 1) >> 4) ? l.sc_now : l.sc_before;
  return __shfl_sync(0xffffffffu, v, 2 * (k & 15) + half);
}

// E4M3 NaN codes of a word zeroed; `any` picks up whether there were some.
__device__ __forceinline__ uint32_t drop_nan4(uint32_t w, uint32_t& any) {
  const uint32_t m = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  any |= m;
  return w & ~m;
}

// Rows of the tile: row j is query i = (16 m + j) / group of the batch row,
// query head h * group + (16 m + j) % group.
__device__ __forceinline__ bool dec_tile_row(const AttnArgs& a, const DecCursor& c, int j, int& i,
                                             int& head) {
  const long long rho = (long long)c.m * 16 + j;
  i = (int)(rho / a.group);
  head = c.h * a.group + (int)(rho - (long long)i * a.group);
  return i < c.x.w.n;
}

// Natural logarithm of the denominator from its reference (log2) and sum.
__device__ __forceinline__ float attn_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}
// 1 / l; 0 where nothing was seen, NaN where the sum is.
__device__ __forceinline__ float attn_inverse(float l) { return l > 0.f ? 1.f / l : l; }
// 2^(m - ref) with both -infinity (nothing seen) giving 1.
__device__ __forceinline__ float attn_factor(float m, float ref) {
  return m == -INFINITY ? (ref == -INFINITY ? 1.f : 0.f) : exp2_approx(m - ref);
}

template <int D>
static __global__ void __launch_bounds__(kDecThreads, 1) kv_attention_decode(const AttnArgs a) {
  using Sh = DecShape<D>;
  constexpr int CH = Sh::CH, KS = D / 16;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  float* s_join = reinterpret_cast<float*>(dec_smem + kDecWarps * Sh::STAGES * 2 * Sh::HALF);
  float* s_m = s_join + kDecWarps * 4 * Sh::RS;    // [warp][16]
  float* s_l = s_m + kDecWarps * 16;
  float* s_f = s_l + kDecWarps * 16;
  float* s_tm = s_f + kDecWarps * 16;              // [16] of the tile
  float* s_tl = s_tm + 16;
  float* s_fac = s_tl + 16;                        // score factors, later the lse
  uint16_t* s_q = reinterpret_cast<uint16_t*>(s_fac + 16);   // [16][D]; the output too
  const uint32_t ring = smem_addr(dec_smem) + warp * Sh::STAGES * 2 * Sh::HALF;
  const uint8_t* ringp = dec_smem + warp * Sh::STAGES * 2 * Sh::HALF;

  pdl_launch_dependents();
  long long u0, n_units, per;
  DecCursor cur;
  dec_schedule(a, u0, n_units, per, cur);
  if (threadIdx.x == 0) a.desc[4 * blockIdx.x] = 0;
  if (n_units <= 0) return;

  DecLoader ld;
  ld.r = cur.r;
  ld.x = cur.x;
  ld.idx = ((long long)cur.h * cur.x.M + cur.m) * cur.x.S + cur.s;
  ld.left = n_units;
  ld.k = 0;
  ld.slot = 0;
  ld.sc_before = 0;
  dec_lane_advance(a, ld, warp + kDecWarps * (lane >> 1));
  dec_lane_lookup(a, ld, lane);
  dec_lane_scales(a, ld);
  dec_lane_take(a, ld);
  const bool exists = ld.id >= 0;
  const uint32_t sk0 = ld.sk, sv0 = ld.sv;
  const DecOffsets off = {g * a.c.tstride + t * 16, (g + 8) * a.c.tstride + t * 16,
                          2 * t * a.c.tstride + g * CH, (2 * t + 8) * a.c.tstride + g * CH};
  const int strips = (int)((n_units - warp + kDecWarps - 1) / kDecWarps);
#pragma unroll 1
  for (int i = 0; i < Sh::STAGES - 1; ++i) dec_fetch<D>(a, ld, off, strips, ring, lane);
  ld.sc_now = dec_pack_scales(exists, sk0, sv0);
  dec_lane_advance(a, ld, 16 * kDecWarps);
  dec_lane_lookup(a, ld, lane);
  int done = 0;                 // strips of the warp consumed
  int slot_in = 0;              // ring slot of the next one

  long long u = 0;              // strips done by the CTA, in its own order
  int next = warp;              // this warp's next strip, relative to the tile's first
  int part = 0;                 // tiles begun
  while (u < n_units) {
    const int nseg = (int)min((long long)(cur.x.S - cur.s), n_units - u);
    const int real = (int)min(16ll, (long long)cur.x.w.n * a.group - 16ll * cur.m);
    // ---- queries of the tile: f16 times 2^-shift, in shared memory; the
    // scale's sign goes with them, so that the factors are positive ----
    for (int j = warp; j < 16; j += kDecWarps) {
      int i, head;
      float v[D / 32];
      float mx = 0.f;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) v[k] = 0.f;
      if (dec_tile_row(a, cur, j, i, head)) {
        const uint16_t* q = a.q + (long long)(cur.x.w.tok + i) * a.q_ts + head * a.q_hs;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const float2 f =
              unpack16(*reinterpret_cast<const uint32_t*>(q + 2 * lane + 64 * k), a.f16);
          v[2 * k] = f.x;
          v[2 * k + 1] = f.y;
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      mx = warp_max(mx);
      // the row's largest value in [2^13, 2^14): f16's exponents reach 2^-38 of it
      const int be = (int)(__float_as_uint(mx) >> 23);
      const int sh = be == 0 || be == 255 ? 0 : min(max(be - 140, -120), 120);
      const float down =
          a.scale_log2 == 0.f ? 0.f : (a.scale_log2 < 0.f ? -pow2f(-sh) : pow2f(-sh));
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
        *reinterpret_cast<uint32_t*>(s_q + j * D + 2 * lane + 64 * k) =
            pack_f16x2(v[2 * k] * down, v[2 * k + 1] * down);
      if (lane == 0) s_fac[j] = fabsf(a.scale_log2) * pow2f(sh);
    }
    __syncthreads();
    uint32_t qf[KS][4];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = (k >> 2) * 64 + t * 16 + (k & 3) * 4;
      const uint2 x = *reinterpret_cast<const uint2*>(s_q + g * D + d);
      const uint2 y = *reinterpret_cast<const uint2*>(s_q + (g + 8) * D + d);
      qf[k][0] = x.x;
      qf[k][1] = y.x;
      qf[k][2] = x.y;
      qf[k][3] = y.y;
    }
    const float fac0 = s_fac[g], fac1 = s_fac[g + 8];
    // what the lane's two rows see, and what every and any row of the tile sees
    int i0, i1, hd, lo0, hi0, lo1, hi1, lo_all, hi_all, lo_any, hi_any;
    if (!dec_tile_row(a, cur, g, i0, hd)) i0 = cur.x.w.n - 1;
    if (!dec_tile_row(a, cur, g + 8, i1, hd)) i1 = cur.x.w.n - 1;
    attn_seen(a, cur.x.w, i0, lo0, hi0);
    attn_seen(a, cur.x.w, i1, lo1, hi1);
    dec_tile_row(a, cur, 0, i0, hd);
    if (!dec_tile_row(a, cur, 15, i1, hd)) i1 = cur.x.w.n - 1;
    attn_seen(a, cur.x.w, i0, lo_any, hi_all);
    attn_seen(a, cur.x.w, i1, lo_all, hi_any);

    float o[CH][4];
#pragma unroll
    for (int j = 0; j < CH; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

#pragma unroll 1
    for (; next < nseg; next += kDecWarps) {
      dec_fetch<D>(a, ld, off, strips, ring, lane);
      cp_async_wait<Sh::STAGES - 1>();
      const uint32_t meta0 = dec_scales(ld, done, 0), meta1 = dec_scales(ld, done, 1);
      ++done;
      __syncwarp();
      const uint8_t* base = ringp + slot_in * (2 * Sh::HALF);
      const uint8_t* sp = base + lane * 16;
      const int p0 = (cur.x.s0 + cur.s + next) << 5;
      slot_in = slot_in + 1 == Sh::STAGES ? 0 : slot_in + 1;
      if (!((meta0 | meta1) >> 16) || p0 >= hi_any || p0 + 32 <= lo_any) continue;
      // ---- scores ----
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = *reinterpret_cast<const uint4*>(sp + (i >> 1) * Sh::HALF +
                                                 ((i & 1) * (D / 64) + c) * 512);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t* q = qf[4 * c + k];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            e4m3x4_to_f16x2(k == 0 ? w[i].x : k == 1 ? w[i].y : k == 2 ? w[i].z : w[i].w, b0, b1);
            mma_f16_16816(s[i], q[0], q[1], q[2], q[3], b0, b1);
          }
        }
      }
      // ---- weights ----
      const float ke0 = pow2f((int)(meta0 & 0xFFu) - 128), ke1 = pow2f((int)(meta1 & 0xFFu) - 128);
      const int ev0 = (int)((meta0 >> 8) & 0xFFu) - 128, ev1 = (int)((meta1 >> 8) & 0xFFu) - 128;
      const float f00 = fac0 * ke0, f01 = fac0 * ke1, f10 = fac1 * ke0, f11 = fac1 * ke1;
      const bool masked =
          p0 + 32 > hi_all || p0 < lo_all || !((meta0 & meta1) >> 16);
      if (masked) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int j = p0 + 8 * i + 2 * t + c;
            const bool there = (i < 2 ? meta0 : meta1) >> 16;
            if (!there || j < lo0 || j >= hi0) s[i][c] = -INFINITY;
            if (!there || j < lo1 || j >= hi1) s[i][2 + c] = -INFINITY;
          }
      }
      // (a factor that underflowed to 0 makes NaN of -infinity, which fmaxf drops)
      float x0 = fmaxf(fmaf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])), f00, (float)ev0),
                       fmaf(fmaxf(fmaxf(s[2][0], s[2][1]), fmaxf(s[3][0], s[3][1])), f01, (float)ev1));
      float x1 = fmaxf(fmaf(fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3])), f10, (float)ev0),
                       fmaf(fmaxf(fmaxf(s[2][2], s[2][3]), fmaxf(s[3][2], s[3][3])), f11, (float)ev1));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
      if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float d0 = attn_factor(m0, n0), d1 = attn_factor(m1, n1);
        m0 = n0;
        m1 = n1;
        l0 *= d0;
        l1 *= d1;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          o[j][0] *= d0;
          o[j][1] *= d0;
          o[j][2] *= d1;
          o[j][3] *= d1;
        }
      }
      const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
      const float c00 = (float)ev0 - r0, c01 = (float)ev1 - r0, c10 = (float)ev0 - r1,
                  c11 = (float)ev1 - r1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i][0] = exp2_approx(fmaf(s[i][0], i < 2 ? f00 : f01, i < 2 ? c00 : c01));
        s[i][1] = exp2_approx(fmaf(s[i][1], i < 2 ? f00 : f01, i < 2 ? c00 : c01));
        s[i][2] = exp2_approx(fmaf(s[i][2], i < 2 ? f10 : f11, i < 2 ? c10 : c11));
        s[i][3] = exp2_approx(fmaf(s[i][3], i < 2 ? f10 : f11, i < 2 ? c10 : c11));
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int j = p0 + 8 * i + 2 * t + c;
            const bool there = (i < 2 ? meta0 : meta1) >> 16;
            if (!there || j < lo0 || j >= hi0) s[i][c] = 0.f;
            if (!there || j < lo1 || j >= hi1) s[i][2 + c] = 0.f;
          }
      }
      const float un0 = pow2f(-ev0), un1 = pow2f(-ev1);
      l0 = fmaf(un0, (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]), l0);
      l1 = fmaf(un0, (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]), l1);
      l0 = fmaf(un1, (s[2][0] + s[2][1]) + (s[3][0] + s[3][1]), l0);
      l1 = fmaf(un1, (s[2][2] + s[2][3]) + (s[3][2] + s[3][3]), l1);
      // ---- values ----
      uint32_t nan = 0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float(*ss)[4] = s + 2 * half;
        const uint32_t pa0 = pack_f16x2(ss[0][0], ss[0][1]), pa1 = pack_f16x2(ss[0][2], ss[0][3]);
        const uint32_t pa2 = pack_f16x2(ss[1][0], ss[1][1]), pa3 = pack_f16x2(ss[1][2], ss[1][3]);
        const uint8_t* hp = sp + half * Sh::HALF;
        uint32_t vw[4][CH / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(hp + (Sh::KP + i) * 512);
            vw[i][0] = w.x;
            vw[i][1] = w.y;
            vw[i][2] = w.z;
            vw[i][3] = w.w;
          } else {
            const uint2 w =
                *reinterpret_cast<const uint2*>(hp + (Sh::KP + (i >> 1)) * 512 + (i & 1) * 8);
            vw[i][0] = w.x;
            vw[i][1] = w.y;
          }
        }
        if (masked) {
          // a weight of 0 does not keep a NaN value out of the sums: NaN codes
          // leave the product here and are given back to the rows that see them
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < CH / 4; ++c) vw[i][c] = drop_nan4(vw[i][c], nan);
        }
#pragma unroll
        for (int c = 0; c < CH / 4; ++c) {
          uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
          e4m3x4_to_f16x2(__byte_perm(vw[0][c], vw[1][c], 0x5140), a0, a1);
          e4m3x4_to_f16x2(__byte_perm(vw[2][c], vw[3][c], 0x5140), b0, b1);
          e4m3x4_to_f16x2(__byte_perm(vw[0][c], vw[1][c], 0x7362), a2, a3);
          e4m3x4_to_f16x2(__byte_perm(vw[2][c], vw[3][c], 0x7362), b2, b3);
          mma_f16_16816(o[4 * c], pa0, pa1, pa2, pa3, a0, b0);
          mma_f16_16816(o[4 * c + 1], pa0, pa1, pa2, pa3, a1, b1);
          mma_f16_16816(o[4 * c + 2], pa0, pa1, pa2, pa3, a2, b2);
          mma_f16_16816(o[4 * c + 3], pa0, pa1, pa2, pa3, a3, b3);
        }
      }
      if (masked && __any_sync(0xffffffffu, nan != 0)) {
        // columns 2t, 2t + 1 of value tile j are dims CH (2t) + j, CH (2t + 1) + j:
        // lanes 8t + tt and 8t + 4 + tt hold them for token pair tt
        const float qnan = __int_as_float(0x7FFFFFFF);
#pragma unroll 1
        for (int tok = 0; tok < 32; ++tok) {
          const int tt = (tok & 7) >> 1, i = (tok & 1) + 2 * ((tok >> 3) & 1), j = p0 + tok;
          const bool there = ((tok < 16 ? meta0 : meta1) >> 16) != 0;
          const bool see0 = there && j >= lo0 && j < hi0, see1 = there && j >= lo1 && j < hi1;
          const uint8_t* hp = base + (tok >> 4) * Sh::HALF;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int src = 8 * t + 4 * c + tt;
            const uint8_t* p = D == 128 ? hp + (Sh::KP + i) * 512 + src * 16
                                        : hp + (Sh::KP + (i >> 1)) * 512 + src * 16 + (i & 1) * 8;
#pragma unroll
            for (int jj = 0; jj < CH; ++jj) {
              if ((p[jj] & 0x7F) != 0x7F) continue;
              if (see0) o[jj][c] = qnan;
              if (see1) o[jj][2 + c] = qnan;
            }
          }
        }
        __syncwarp();
      }
    }
    next -= nseg;

    // ---- join the warps' sums, four rows a round ----
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (t == 0) {
      s_m[warp * 16 + g] = m0;
      s_m[warp * 16 + g + 8] = m1;
      s_l[warp * 16 + g] = l0;
      s_l[warp * 16 + g + 8] = l1;
    }
    __syncthreads();
    if (threadIdx.x < kDecWarps * 16) {
      const int row = threadIdx.x & 15;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, s_m[w * 16 + row]);
      s_f[threadIdx.x] = attn_factor(s_m[threadIdx.x], m);
      if (threadIdx.x < 16) {
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w)
          l = fmaf(s_l[w * 16 + row], attn_factor(s_m[w * 16 + row], m), l);
        s_tm[row] = m;
        s_tl[row] = l;
      }
    }
    __syncthreads();
    const bool whole = cur.s == 0 && nseg == cur.x.S;
    float* slot = a.partial + (2ll * blockIdx.x + (part > 0)) * kDecSlot<D>;
    const float d0 = s_f[warp * 16 + g], d1 = s_f[warp * 16 + g + 8];
#pragma unroll
    for (int round = 0; round < 4; ++round) {
      if (4 * round >= real) break;
      float* dst = s_join + (warp * 4 + (g & 3)) * Sh::RS + 2 * t;
      if ((g >> 2) == (round & 1)) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
          *reinterpret_cast<float2*>(dst + j * 8) =
              round < 2 ? make_float2(o[j][0] * d0, o[j][1] * d0)
                        : make_float2(o[j][2] * d1, o[j][3] * d1);
      }
      __syncthreads();
      for (int e = threadIdx.x; e < 2 * D; e += kDecThreads) {
        const int r = e / (D / 2), row = 4 * round + r, col = (e % (D / 2)) * 2;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(s_join + (w * 4 + r) * Sh::RS + col);
          sum.x += v.x;
          sum.y += v.y;
        }
        if (whole) {
          const float inv = attn_inverse(s_tl[row]);
          uint16_t* so = s_q + row * D + (col >> 3);
          so[(col & 7) * CH] = (uint16_t)pack16(sum.x * inv, 0.f, a.f16);
          so[((col & 7) + 1) * CH] = (uint16_t)pack16(sum.y * inv, 0.f, a.f16);
        } else {
          *reinterpret_cast<float2*>(slot + row * D + col) = sum;
        }
      }
      __syncthreads();
    }
    if (whole) {
      for (int e = threadIdx.x; e < real * (D / 8); e += kDecThreads) {
        const int row = e / (D / 8), d = (e % (D / 8)) * 8;
        int i, head;
        dec_tile_row(a, cur, row, i, head);
        const long long tok = cur.x.w.tok + i;
        *reinterpret_cast<uint4*>(a.out + tok * a.o_ts + head * a.o_hs + d) =
            *reinterpret_cast<const uint4*>(s_q + row * D + d);
        if (d == 0 && a.lse) a.lse[tok * a.heads + head] = attn_lse(s_tm[row], s_tl[row]);
      }
      __syncthreads();   // the queries of the next tile go into s_q
    } else {
      if (threadIdx.x < 16) {
        slot[16 * D + threadIdx.x] = s_tm[threadIdx.x];
        slot[16 * D + 16 + threadIdx.x] = s_tl[threadIdx.x];
      }
      if (cur.s == 0 && threadIdx.x == 0) {
        // this CTA begins a tile that later CTAs go on with
        const long long end = u0 + u + cur.x.S;   // the tile's end in strips of the call
        int* d = a.desc + 4 * blockIdx.x;
        d[1] = part > 0;
        d[2] = cur.r;
        d[3] = cur.h * cur.x.M + cur.m;
        d[0] = (int)((end - 1) / per) - (int)blockIdx.x + 1;
      }
    }
    u += nseg;
    ++part;
    if (u < n_units) dec_next_tile(a, cur);
  }
  cp_async_wait<0>();
}

// Join of the tiles cut by CTA boundaries: block (i, j) takes rows j, j +
// gridDim.y, ... of the tile that CTA i began, if any.  The partial sums of
// CTAs i, i + 1, ... go round groups of D threads, four loads in flight each,
// and the groups' sums are added in order.
constexpr int kJoinThreads = 512;
constexpr int kJoinMax = 1024;   // CTAs of the first kernel

template <int D>
static __global__ void __launch_bounds__(kJoinThreads) kv_attention_join(const AttnArgs a) {
  constexpr int NG = kJoinThreads / D;
  __shared__ float s_w[kJoinMax];
  __shared__ float s_red[kJoinThreads];
  const int t = threadIdx.x;
  pdl_wait_prerequisites();
  const int4 d = *reinterpret_cast<const int4*>(a.desc + 4 * blockIdx.x);
  const int n = d.x;
  if (n == 0) return;
  DecCursor c;
  c.r = d.z;
  c.x = dec_row(a, c.r);
  c.h = d.w / c.x.M;
  c.m = d.w - c.h * c.x.M;
  // piece k: the tile's slot in CTA i + k (its first one, but for the beginning)
  const float* first = a.partial + (2ll * blockIdx.x + d.y) * kDecSlot<D>;
  const float* rest = a.partial + 2ll * blockIdx.x * kDecSlot<D>;
  const int col = t % D, grp = t / D, dim = (col & 7) * (D / 8) + (col >> 3);
  for (int row = blockIdx.y; row < 16; row += gridDim.y) {
    int i, head;
    if (!dec_tile_row(a, c, row, i, head)) break;
    float m = -INFINITY;
    for (int k = t; k < n; k += kJoinThreads) {
      const float* p = k == 0 ? first : rest + 2ll * k * kDecSlot<D>;
      const float v = p[16 * D + row];
      s_w[k] = v;
      m = fmaxf(m, v);
    }
    m = warp_max(m);
    if ((t & 31) == 0) s_red[t >> 5] = m;
    __syncthreads();
    m = s_red[t & 15];
    m = warp_max(m);
    float l = 0.f;
    for (int k = t; k < n; k += kJoinThreads) {
      const float* p = k == 0 ? first : rest + 2ll * k * kDecSlot<D>;
      const float f = attn_factor(s_w[k], m);
      s_w[k] = f;
      l = fmaf(p[16 * D + 16 + row], f, l);
    }
    l = warp_sum(l);
    __syncthreads();
    if ((t & 31) == 0) s_red[t >> 5] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) l += s_red[w];
    float sum = 0.f;
#pragma unroll 4
    for (int k = grp; k < n; k += NG) {
      const float* p = k == 0 ? first : rest + 2ll * k * kDecSlot<D>;
      sum = fmaf(p[row * D + col], s_w[k], sum);
    }
    __syncthreads();
    s_red[t] = sum;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int w = 1; w < NG; ++w) sum += s_red[w * D + col];
      const long long tok = c.x.w.tok + i;
      a.out[tok * a.o_ts + head * a.o_hs + dim] =
          (uint16_t)pack16(sum * attn_inverse(l), 0.f, a.f16);
      if (a.lse && t == 0) a.lse[tok * a.heads + head] = attn_lse(m, l);
    }
    __syncthreads();
  }
}

}  // namespace moe
