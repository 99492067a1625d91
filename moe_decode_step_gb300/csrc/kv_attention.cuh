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
  float* partial;     // slots of partial sums
  unsigned* arrived;  // four per CTA, zero when the kernel starts
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
// form tiles of 8 or 16 rows, one or two n-tiles of m16n8k16 products whose M
// is 16 tokens (scores, transposed) or 16 dims (values): with the rows on the
// short side 8 rows cost half of what they would as M, in MMAs, registers and
// exponentials.  A call reads every visible byte of the cache once per tile
// and does 4 * 16 * D operations on the 2 * D bytes of a token at 16 rows: 32
// operations a byte, far below the tensor cores' balance, so HBM bounds it
// and the layout serves the loads.
//
// Work: strips of 32 tokens of (row of the batch, KV head, tile), ordered in
// that order; CTA i takes strips [i * per, (i + 1) * per) and each of its
// warps an equal run of them, whatever the rows' lengths.  A warp works by
// itself: it writes the tiles that lie inside its run and keeps partial sums
// of the one or two that its ends cut.  When its warps are done the CTA joins
// them once, in strip order; of a tile that CTA ends cut, the CTA that arrives
// last (a counter; nobody waits) joins the CTAs' sums in their order, in two
// levels where they are more than 16: results do not depend on timing.  (With
// the strips dealt round the warps and joined at the end of every tile, a tile
// cost about 6 us of barriers and refilling; a second kernel for the CTAs'
// sums 10 to 15 us against 4 inside.)
// One CTA an SM, one share each: the SMs of full GPCs stream more slowly (at
// 1.2 GB 40 of them took 230 us where the others took 200), but up to three
// waves of smaller CTAs, two an SM, lost more in starts and joins (290 us
// against 256).
// Measured (codes and scales per time): 64 rows of 2,047 to 16,383 tokens, 8
// KV heads of 128, 8 rows a head: 258 us, 4.7 TB/s, 70% of a copy's rate; one
// row of 262,142 tokens, 2 KV heads, 16 rows a head: 57 us, 2.4 TB/s; 32 rows
// in a window of 1,024, 32 KV heads of 64: 42 us, 3.1 TB/s.  Of the short
// ones 10 us are the start (2), the joins (2 + 3 + 3) and cold code.
//
// Loads: each thread copies (cp.async) exactly the 16-byte pieces that it
// feeds to its own MMAs, into a ring of its own in shared memory, so a strip
// needs no barrier at all; the ring only deepens the loads in flight (D = 128:
// 12 warps x 8 KB = 96 KB an SM; 1 us of latency at 6.7 TB/s needs 44 KB).
// The contraction order of either product is free, so the pieces need no
// shuffling: in each half of a strip (16 tokens) lane (g, t) = (lane / 4, lane
// % 4) holds, for the scores, 16 consecutive dims (from 16 t, and from 64 + 16
// t) of keys g and g + 8, and for the values CH = D / 8 consecutive dims (from
// CH g) of tokens 2t, 2t + 1, 2t + 8, 2t + 9, byte-transposed in registers.
// Codes become f16 exactly (cvt.rn.f16x2.e4m3x2); queries enter as f16 scaled
// per row by a power of two, which keeps all of bf16's 8 bits.  The scores'
// fragments become the weights' by movmatrix.
// What bounds the kernel beside HBM is latency in the chain scores - maximum -
// weights - values, hidden by 12 to 16 warps an SM, and instruction issue
// (128 conversions a strip of 8 KB, 32 MMAs per n-tile), so a strip is two
// halves long: one maximum and one vote for 32 tokens.
//
// Scales: a half lies in one block, so one exponent ek scales its scores and
// one ev its values.  With t = score * log2(e) + ev the weights 2^(t - M) are
// the values' true relative sizes, whatever the spread of the block scales.
// M is the running maximum of t less kDecLead: the largest weight is 2^13, so
// that f16 keeps all its bits down to 2^-27 of it, and what many keys far
// behind a leading one add up to is not rounded away.  The denominator takes
// the same weights times 2^-ev in fp32; blocks of ev below kKvExpLow (zeros, or
// values below 2^-19) take theirs with 2^(kKvExpLow - ev) more, which the
// second product's do not have.
constexpr float kDecLead = 13.f;

template <int D, int NT>   // NT: n-tiles of 8 rows in a tile
struct DecShape {
  static constexpr int ROWS = 8 * NT;
  static constexpr int CH = D / 8;                 // value dims a lane holds per token
  static constexpr int KP = D / 32;                // 16-byte key pieces a lane and half (2 keys)
  static constexpr int VP = 4 * CH / 16;           // the same for values (4 tokens)
  static constexpr int HALF = 32 * 16 * (KP + VP); // bytes of one warp's half strip
  static constexpr int WARPS = NT == 1 ? (D == 128 ? 12 : 16) : (D == 128 ? 8 : 12);
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int STAGES = 196608 / (WARPS * 2 * HALF);
  static constexpr int RING = STAGES * 2 * HALF;   // a warp's
  static constexpr int SMEM = WARPS * RING;
  // one slot of partial sums: O [ROWS][D] in dec_dim's column order, then m
  // [ROWS] and l [ROWS].  A warp's last piece goes into its ring, its first
  // one (if it has two) into a slot of the workspace, as do the CTA's sums
  // of the tiles that its ends cut: one begun before it, one by it.
  static constexpr int SLOT = ROWS * D + 2 * ROWS;
  static constexpr int SLOTS = WARPS + 2;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid,
                                         uint64_t policy) {
  const int n = valid ? BYTES : 0;   // 0: the destination is zero-filled, src is not read
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2, %3;" ::"r"(
                     dst),
                 "l"(src), "r"(n), "l"(policy)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], 8, %2, %3;" ::"r"(dst),
                 "l"(src), "r"(n), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Transpose of an 8 x 8 matrix of 16-bit elements held as MMA fragments.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// A row's share of the work: M tiles of TILE rows, S strips each, from strip s0.
struct DecRow {
  AttnRow w;
  int M, S, s0;
};

template <int TILE>
__device__ __forceinline__ DecRow dec_row(const AttnArgs& a, int r) {
  DecRow x;
  x.w = attn_row(a, r);
  x.M = (int)(((long long)x.w.n * a.group + TILE - 1) / TILE);
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
template <int TILE>
__device__ __forceinline__ void dec_next_tile(const AttnArgs& a, DecCursor& c) {
  c.s = 0;
  if (++c.m < c.x.M) return;
  c.m = 0;
  if (++c.h < a.c.heads) return;
  c.h = 0;
  do {
    if (++c.r >= a.rows) return;
    c.x = dec_row<TILE>(a, c.r);
  } while (c.x.M == 0);
}

// Exclusive prefix over the CTA's threads, and the total; every thread calls.
template <int WARPS>
__device__ __forceinline__ long long dec_scan(long long v, long long& total) {
  __shared__ long long s_sum[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  long long base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w == warp) base = total;
    total += s_sum[w];
  }
  return base + inc - v;
}

// A CTA's share: n strips from the cursor on, u0 the first in the order of all.
// Either `per` strips a CTA before cuts are moved, or (per 0) the CTAs c0 ..
// c0 + ctas - 1 share the one tile that this CTA works on.
struct DecShare {
  long long u0, n, per;
  int c0, ctas;
  DecCursor cur;
};

// Equal shares cut tiles anywhere, and a tile cut by a CTA's end costs that CTA
// a second tile's joins, some 5 us.  So few tiles are split each on its own, if
// no CTA then has more than kDecSlack strips over the equal share, and many
// tiles of no more strips than that stay whole, if the equal share is four
// times as much.  Against equal shares: 2 tiles of 8,192 strips 57 us (70), 64
// of 128 strips 37.5 (39.6), 64 of 47 strips 27.3 (31.4), 1,024 of 33 strips
// 45.7 (47.7).
constexpr int kDecSlack = 40;

// Every thread calls.  The sums over the rows are made by every CTA for itself.
template <int TILE, int WARPS>
__device__ __forceinline__ void dec_schedule(const AttnArgs& a, DecShare& sh) {
  __shared__ long long s_left, s_cut[2];
  __shared__ int s_row;
  const int t = threadIdx.x;
  const int chunk = (a.rows + (32 * WARPS) - 1) / (32 * WARPS);
  const int r0 = min(a.rows, t * chunk), r1 = min(a.rows, r0 + chunk);
  long long sum = 0, tiles = 0, total, n_tiles;
  bool large = false;
  for (int r = r0; r < r1; ++r) {
    const DecRow x = dec_row<TILE>(a, r);
    sum += dec_units(a, x);
    tiles += (long long)a.c.heads * x.M;
    large |= x.S > kDecSlack;
  }
  long long before = dec_scan<WARPS>(sum, total);
  dec_scan<WARPS>(tiles, n_tiles);
  const long long even = max((total + gridDim.x - 1) / gridDim.x, (long long)WARPS);
  // the tiles' CTAs, ceil(S / most) each, are at most total / most + n_tiles
  const long long spare = (long long)gridDim.x - n_tiles;
  const long long most = spare > 0 ? max((total + spare - 1) / spare, (long long)WARPS) : 0;
  const bool apart = spare > 0 && most <= even + kDecSlack;
  long long at = even * blockIdx.x;   // in strips, or in CTAs
  long long n = min(even, total - at);
  if (!apart && !__syncthreads_or(large) && even >= 4 * kDecSlack) {
    // whole tiles: those that begin in the CTA's equal share
    if (t < 2) s_cut[t] = total;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long x = at + k * even;
      long long y = before;
      if (x >= total || x < before || x >= before + sum) continue;
      for (int r = r0;; ++r) {
        const DecRow w = dec_row<TILE>(a, r);
        const long long units = dec_units(a, w);
        if (x < y + units) {
          s_cut[k] = y + (x - y + w.S - 1) / w.S * w.S;
          break;
        }
        y += units;
      }
    }
    __syncthreads();
    at = s_cut[0];
    n = s_cut[1] - at;
  } else if (apart) {
    sum = 0;
    for (int r = r0; r < r1; ++r) {
      const DecRow x = dec_row<TILE>(a, r);
      sum += (long long)a.c.heads * x.M * ((x.S + most - 1) / most);
    }
    before = dec_scan<WARPS>(sum, total);
    at = blockIdx.x;
  }
  sh.per = apart ? 0 : even;
  sh.u0 = apart ? 0 : at;
  sh.n = apart ? (at < total ? 1 : 0) : n;
  if (sh.n > 0 && at >= before && at < before + sum) {
    int r = r0;
    for (;; ++r) {
      const DecRow x = dec_row<TILE>(a, r);
      const long long k =
          apart ? (long long)a.c.heads * x.M * ((x.S + most - 1) / most) : dec_units(a, x);
      if (at < before + k) break;
      before += k;
    }
    s_row = r;
    s_left = at - before;
  }
  __syncthreads();
  if (sh.n <= 0) return;
  DecCursor& cur = sh.cur;
  cur.r = s_row;
  cur.x = dec_row<TILE>(a, cur.r);
  const int S = cur.x.S, parts = apart ? (int)((S + most - 1) / most) : S;
  const int hm = (int)(s_left / parts), part = (int)(s_left - (long long)hm * parts);
  cur.m = hm % cur.x.M;
  cur.h = hm / cur.x.M;
  cur.s = part;
  if (apart) {
    cur.s = (int)((long long)S * part / parts);
    sh.n = (long long)S * (part + 1) / parts - cur.s;
    sh.c0 = blockIdx.x - part;
    sh.ctas = parts;
  }
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
template <int TILE>
__device__ __forceinline__ void dec_lane_advance(const AttnArgs& a, DecLoader& l, long long n) {
  l.left -= n;
  if (l.left <= 0) return;
  l.idx += n;
  for (;;) {
    const long long units = dec_units(a, l.x);
    if (l.idx < units) return;
    l.idx -= units;
    l.x = dec_row<TILE>(a, ++l.r);
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
// The codes are read once: first out of L2, which keeps the kernel's own cold
// code and the partial sums there.
struct DecOffsets {
  long long k0, k1, v0, v1;
  uint64_t policy;
};

template <int D, int NT>
__device__ __forceinline__ void dec_fetch(const AttnArgs& a, DecLoader& l, const DecOffsets& f,
                                          int strips, uint32_t ring, int lane) {
  using Sh = DecShape<D, NT>;
  if (l.k < strips) {
    const int b = l.k & 15;
    if (b == 0 && l.k > 0) {
      dec_lane_take(a, l);
      l.sc_before = l.sc_now;
      l.sc_now = dec_pack_scales(l.id >= 0, l.sk, l.sv);
      dec_lane_advance<Sh::ROWS>(a, l, 16);
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
            cp_async<16>(dst + (i * (D / 64) + c) * 512, src[i] + c * 64, true, f.policy);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) cp_async<16>(dst + (Sh::KP + i) * 512, src[2 + i], true, f.policy);
          else cp_async<8>(dst + (Sh::KP + (i >> 1)) * 512 + (i & 1) * 8, src[2 + i], true, f.policy);
        }
      } else {   // a row's end: what is not cached is zero-filled and not read
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            cp_async<16>(dst + (i * (D / 64) + c) * 512,
                         tok[i] < cached ? src[i] + c * 64 : a.c.k, tok[i] < cached, f.policy);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = tok[2 + i] < cached;
          const uint8_t* p = in ? src[2 + i] : a.c.v;
          if constexpr (D == 128) cp_async<16>(dst + (Sh::KP + i) * 512, p, in, f.policy);
          else cp_async<8>(dst + (Sh::KP + (i >> 1)) * 512 + (i & 1) * 8, p, in, f.policy);
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

// Rows of the tile: row j is query i = (TILE m + j) / group of the batch row,
// query head h * group + (TILE m + j) % group.
template <int TILE>
__device__ __forceinline__ bool dec_tile_row(const AttnArgs& a, const DecCursor& c, int j, int& i,
                                             int& head) {
  const unsigned rho = (unsigned)c.m * TILE + j;   // tokens * heads < 2^31
  i = (int)(rho / (unsigned)a.group);
  head = c.h * a.group + (int)(rho - (unsigned)i * (unsigned)a.group);
  return i < c.x.w.n;
}

// Dim of a column in the partial sums' order: column 16 j + 2 g + e is dim
// CH g + 2 j + e (a lane's pairs adjacent, a warp's store contiguous).
template <int D>
__device__ __forceinline__ int dec_dim(int col) {
  return ((col >> 1) & 7) * (D / 8) + 2 * (col >> 4) + (col & 1);
}

// Natural logarithm of the denominator from its reference (log2) and sum.
__device__ __forceinline__ float attn_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}
// 1 / l; 0 where nothing was seen, NaN where the sum is.
__device__ __forceinline__ float attn_inverse(float l) { return l > 0.f ? 1.f / l : l; }
// Scores past this are so far apart in fp32 (2^-2 and more) that t - M rounded
// once is no weight any more: t is rounded first, as M was, and t - M is exact.
constexpr float kAttnLarge = 4194304.f;   // 2^22
// 2^((m - ref) / 2) with both -infinity (nothing seen) giving 1.  Sums of the
// values take its square; the denominator takes it twice: between blocks of
// exponents -60 and 60 the square may underflow where the denominator counts.
__device__ __forceinline__ float attn_half_factor(float m, float ref) {
  return m == -INFINITY ? (ref == -INFINITY ? 1.f : 0.f) : exp2_approx(0.5f * (m - ref));
}

// Partial sums of a piece of a tile.
struct DecPiece {
  int state;       // 0: none, else 1 | begins its tile << 1 | ends it << 2
  int h, m, tok, n, S;
  long long at;    // the tile's first strip, relative to the CTA's
};

// Partial sums to be joined: up to 32 pieces of one tile, those in `mask`,
// into the output (dst null) or the slot `dst`, which may be one of theirs.
// Piece k is in the workspace at base + k * stride (+ extra for k = 0), or, for
// a CTA's own pieces (ring set), pieces 2w at base + w * stride and 2w + 1 at
// ring + w * ring_stride.
struct DecJob {
  const float* base;
  float* dst;
  const float* ring;
  long long stride, extra;
  int ring_stride;
  unsigned mask;
  int h, m, tok, n;
};

// Where the joined rows go: the call's arguments, in shared memory.
struct DecOut {
  uint16_t* out;
  float* lse;
  long long o_ts, o_hs;
  int heads, f16;
  unsigned group;
};

// Groups `item`, item + step, ... of R rows of `jobs` jobs, the first rows of
// all of them first; a warp a group, V columns a lane.  Small and not inlined:
// the code runs a few times per launch, mostly fetched cold, and everything it
// reads but the pieces is in shared memory.  What other CTAs wrote is read at
// L2, B pieces of R rows at once and without branches between: a round trip is
// 0.7 us, and what follows it as long again.  (128 rows of a tcgen05 tile, R 2
// and B 8: 20 us for two tiles of four pieces.)
// (ORDERED: the pieces' columns are the dims themselves.)
template <int D, int ROWS, bool ORDERED = false>
__device__ __noinline__ void dec_join(const DecOut* to, const DecJob* job, int jobs, int item,
                                      int step) {
  constexpr int V = D / 32, R = ROWS > 16 ? 4 : ROWS > 8 ? 2 : 1, B = 16 / R;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (; item < jobs * (ROWS / R); item += step) {
    const DecJob& b = job[item % jobs];
    const int row = item / jobs * R;
    const unsigned rho = (unsigned)b.m * ROWS + row;   // as in dec_tile_row
    if ((int)(rho / to->group) >= b.n) continue;
    const float* ring = b.ring;
    const int sh = ring ? 1 : 0;                       // workspace piece k has mask bit k << sh
    const unsigned mask = b.mask, far = ring ? mask & 0x55555555u : mask;
    const int last = far ? (31 - __clz(far)) >> sh : 0;
    float mk[R], lk[R];
#pragma unroll
    for (int x = 0; x < R; ++x) {
      mk[x] = -INFINITY;
      lk[x] = 0.f;
      if ((mask >> lane) & 1u) {
        if (ring && (lane & 1)) {
          const float* ml = ring + (lane >> 1) * b.ring_stride + ROWS * D + row + x;
          mk[x] = ml[0];
          lk[x] = ml[ROWS];
        } else {
          const float* ml = b.base + (lane >> sh) * b.stride + (lane == 0 ? b.extra : 0) +
                            ROWS * D + row + x;
          mk[x] = __ldcg(ml);
          lk[x] = __ldcg(ml + ROWS);
        }
      }
    }
    float acc[R][V], tm[R], f[R], tl[R];
#pragma unroll 1
    for (int k = 0; k <= last; k += B) {
      float2 v[R][B][V / 2];
#pragma unroll
      for (int u = 0; u < B; ++u) {   // what is not there has weight 0
        const bool in = (far >> ((k + u) << sh)) & 1u;
        const float* src = b.base + (k + u) * b.stride + (k + u == 0 ? b.extra : 0) + row * D +
                           V * lane;
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
          for (int n = 0; n < V / 2; ++n)
            v[x][u][n] = in ? __ldcg(reinterpret_cast<const float2*>(src + x * D + 2 * n))
                            : make_float2(0.f, 0.f);
      }
      if (k == 0) {
#pragma unroll
        for (int x = 0; x < R; ++x) tm[x] = warp_max(mk[x]);
#pragma unroll
        for (int x = 0; x < R; ++x) {
          const float h =
              mk[x] == -INFINITY && lk[x] == 0.f ? 0.f : attn_half_factor(mk[x], tm[x]);
          f[x] = h * h;
          tl[x] = warp_sum(lk[x] * h * h);
#pragma unroll
          for (int n = 0; n < V; ++n) acc[x][n] = 0.f;
        }
        if (ring) {
#pragma unroll 4
          for (int p = 0; p < 16; ++p) {
            const float* src = ring + p * b.ring_stride + row * D + V * lane;
#pragma unroll
            for (int x = 0; x < R; ++x) {
              const float fk = __shfl_sync(0xffffffffu, f[x], 2 * p + 1);
              if (!((mask >> (2 * p + 1)) & 1u)) continue;
#pragma unroll
              for (int n = 0; n < V; ++n) acc[x][n] = fmaf(src[x * D + n], fk, acc[x][n]);
            }
          }
        }
      }
#pragma unroll
      for (int x = 0; x < R; ++x)
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const float fk = __shfl_sync(0xffffffffu, f[x], ((k + u) << sh) & 31);
#pragma unroll
          for (int n = 0; n < V / 2; ++n) {
            acc[x][2 * n] = fmaf(v[x][u][n].x, fk, acc[x][2 * n]);
            acc[x][2 * n + 1] = fmaf(v[x][u][n].y, fk, acc[x][2 * n + 1]);
          }
        }
    }
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const int i = (int)((rho + x) / to->group);
      if (i >= b.n) break;
      if (!b.dst) {
        const float inv = attn_inverse(tl[x]);
        const long long tok = b.tok + i;
        const int head = b.h * (int)to->group + (int)(rho + x - (unsigned)i * to->group);
        uint16_t* out = to->out + tok * to->o_ts + head * to->o_hs;
#pragma unroll
        for (int n = 0; n < V; n += 2)
          *reinterpret_cast<uint32_t*>(
              out + (ORDERED ? V * lane + n : dec_dim<D>(V * lane + n))) =
              pack16(acc[x][n] * inv, acc[x][n + 1] * inv, to->f16);
        if (lane == 0 && to->lse) to->lse[tok * to->heads + head] = attn_lse(tm[x], tl[x]);
      } else {
        float* dst = b.dst + (row + x) * D + V * lane;
#pragma unroll
        for (int n = 0; n < V; n += 2)
          *reinterpret_cast<float2*>(dst + n) = make_float2(acc[x][n], acc[x][n + 1]);
        if (lane == 0) {
          b.dst[ROWS * D + row + x] = tm[x];
          b.dst[ROWS * D + ROWS + row + x] = tl[x];
        }
      }
    }
  }
}

constexpr int kDecGroup = 16;                          // CTAs joined at once
constexpr int kDecMaxCtas = kDecGroup * kDecGroup;     // in two levels

// The sums of tiles that the CTA's own ends cut are in its slots (p0: of a
// tile begun before, p1: of one that it begins; null: none), at `base` + the
// CTA * STRIDE (+ SLOT for the CTA that begins the tile): count them, and
// whoever comes last joins.  Level 0: the CTAs of one group; level 1: the
// groups, each in its first CTA's slot.  Both tiles are counted before either
// is joined: others may wait for this CTA's sums.  Every thread calls.
template <int D, int ROWS, int WARPS, int STRIDE, int SLOT, bool ORDERED>
__device__ __forceinline__ void dec_join_ctas(const AttnArgs& a, float* base,
                                              const DecShare& share, const DecPiece* p0,
                                              const DecPiece* p1, const DecOut* to, DecJob* job) {
  __shared__ int s_jobs;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const DecPiece* p = lane == 0 ? p0 : p1;
  bool open = lane < 2 && p;
  int c0 = share.c0, n = share.ctas;
  if (warp == 0 && open && share.per) {
    const long long tile = share.u0 + p->at;
    c0 = (int)(tile / share.per);
    n = (int)((tile + p->S - 1) / share.per) - c0 + 1;
  }
#pragma unroll 1
  for (int level = 0; level < 2; ++level) {
    __syncthreads();
    if (warp == 0) {
      const int groups = (n + kDecGroup - 1) / kDecGroup;
      const int grp = level ? 0 : ((int)blockIdx.x - c0) / kDecGroup;
      const int count = level ? groups : min(kDecGroup, n - grp * kDecGroup);
      bool won = false;
      if (open) {
        // counters of CTA c: the tile it begins, that tile's first group, and
        // the later group of a tile begun before that starts with c
        unsigned* counter = a.arrived + 4 * (c0 + grp * kDecGroup) + (level ? 0 : grp ? 2 : 1);
        __threadfence();
        won = atomicAdd(counter, 1u) == (unsigned)count - 1;
        __threadfence();
      }
      const unsigned m = __ballot_sync(0xffffffffu, won);
      if (won) {
        float* from = base + (long long)(c0 + grp * kDecGroup) * STRIDE;
        const int extra = grp > 0 ? 0 : SLOT;
        const bool final = level == 1 || groups == 1;
        job[__popc(m & ((1u << lane) - 1))] = {
            from, final ? nullptr : from + extra, nullptr,
            (long long)(level ? kDecGroup : 1) * STRIDE, extra, 0, ~0u >> (32 - count),
            p->h, p->m, p->tok, p->n};
      }
      open = won && groups > 1;
      if (lane == 0) s_jobs = __popc(m);
    }
    __syncthreads();
    if (s_jobs == 0) return;
    dec_join<D, ROWS, ORDERED>(to, job, s_jobs, warp, WARPS);
  }
}

template <int D, int NT>
static __global__ void __launch_bounds__(DecShape<D, NT>::THREADS, 1)
    kv_attention_decode(const AttnArgs a) {
  using Sh = DecShape<D, NT>;
  constexpr int CH = Sh::CH, KS = D / 16, ROWS = Sh::ROWS, W = Sh::WARPS;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  __shared__ DecPiece s_piece[2 * W];
  __shared__ DecOut s_out;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_addr(dec_smem) + warp * Sh::RING;
  uint8_t* ringp = dec_smem + warp * Sh::RING;
  float* slots = a.partial + (long long)blockIdx.x * Sh::SLOTS * Sh::SLOT;

  DecShare share;
  dec_schedule<ROWS, W>(a, share);
  const long long n_units = share.n;
  if (n_units <= 0) return;
  DecCursor& cur = share.cur;
  if (threadIdx.x < 2 * W) s_piece[threadIdx.x].state = 0;
  if (threadIdx.x == 0)
    s_out = {a.out, a.lse, a.o_ts, a.o_hs, a.heads, a.f16, (unsigned)a.group};
  __syncthreads();

  // this warp's run: strips [first, first + n_warp) of the CTA's
  const long long first = n_units * warp / W;
  const int n_warp = (int)(n_units * (warp + 1) / W - first);
  if (n_warp > 0) {
    DecLoader ld;
    ld.r = cur.r;
    ld.x = cur.x;
    ld.idx = ((long long)cur.h * cur.x.M + cur.m) * cur.x.S + cur.s;
    ld.left = n_units;
    dec_lane_advance<ROWS>(a, ld, first);
    cur.r = ld.r;
    cur.x = ld.x;
    cur.s = (int)(ld.idx % cur.x.S);
    cur.h = (int)(ld.idx / cur.x.S) / cur.x.M;
    cur.m = (int)(ld.idx / cur.x.S) % cur.x.M;
    ld.left = n_warp;
    ld.k = 0;
    ld.slot = 0;
    ld.sc_before = 0;
    dec_lane_advance<ROWS>(a, ld, lane >> 1);
    dec_lane_lookup(a, ld, lane);
    dec_lane_scales(a, ld);
    dec_lane_take(a, ld);
    const bool exists = ld.id >= 0;
    const uint32_t sk0 = ld.sk, sv0 = ld.sv;
    const DecOffsets off = {g * a.c.tstride + t * 16, (g + 8) * a.c.tstride + t * 16,
                            2 * t * a.c.tstride + g * CH, (2 * t + 8) * a.c.tstride + g * CH,
                            policy_evict_first()};
#pragma unroll 1
    for (int i = 0; i < Sh::STAGES - 1; ++i) dec_fetch<D, NT>(a, ld, off, n_warp, ring, lane);
    ld.sc_now = dec_pack_scales(exists, sk0, sv0);
    dec_lane_advance<ROWS>(a, ld, 16);
    dec_lane_lookup(a, ld, lane);
    int done = 0;      // strips consumed
    int slot_in = 0;   // ring slot of the next one

#pragma unroll 1
    while (done < n_warp) {
      const int nseg = min(cur.x.S - cur.s, n_warp - done);
      // ---- queries: lane (g, t) takes 16 dims of row 8 q + g (from 16 t, and
      // from 64 + 16 t), as f16 times 2^-shift; the scale's sign goes with
      // them, so that the factors are positive ----
      uint2 qf[NT][KS];
      // the lane's rows of the scores, 8 q + 2t + r: score factor, what they see
      float fac[NT][2], m[NT][2], l[NT][2];
      int lo[NT][2], hi[NT][2], lo_all, hi_all, lo_any, hi_any, i0, i1, hd;
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        uint4 w[D / 64][2];
        float mx = 0.f;
        const bool real = dec_tile_row<ROWS>(a, cur, 8 * q + g, i0, hd);
        const uint16_t* src = a.q + (long long)(cur.x.w.tok + i0) * a.q_ts + hd * a.q_hs + t * 16;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            w[c][i] = make_uint4(0, 0, 0, 0);
            if (real) w[c][i] = *reinterpret_cast<const uint4*>(src + c * 64 + i * 8);
            const float2 f0 = unpack16(w[c][i].x, a.f16), f1 = unpack16(w[c][i].y, a.f16),
                         f2 = unpack16(w[c][i].z, a.f16), f3 = unpack16(w[c][i].w, a.f16);
            mx = fmaxf(mx, fmaxf(fmaxf(fmaxf(fabsf(f0.x), fabsf(f0.y)), fmaxf(fabsf(f1.x), fabsf(f1.y))),
                                 fmaxf(fmaxf(fabsf(f2.x), fabsf(f2.y)), fmaxf(fabsf(f3.x), fabsf(f3.y)))));
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the row's largest value in [2^13, 2^14): f16's exponents reach 2^-38 of it
        const int be = (int)(__float_as_uint(mx) >> 23);
        const int sh = be == 0 || be == 255 ? 0 : min(max(be - 140, -120), 120);
        const float down =
            a.scale_log2 == 0.f ? 0.f : (a.scale_log2 < 0.f ? -pow2f(-sh) : pow2f(-sh));
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f0 = unpack16(w[c][i].x, a.f16), f1 = unpack16(w[c][i].y, a.f16),
                         f2 = unpack16(w[c][i].z, a.f16), f3 = unpack16(w[c][i].w, a.f16);
            qf[q][4 * c + 2 * i] = make_uint2(pack_f16x2(f0.x * down, f0.y * down),
                                              pack_f16x2(f1.x * down, f1.y * down));
            qf[q][4 * c + 2 * i + 1] = make_uint2(pack_f16x2(f2.x * down, f2.y * down),
                                                  pack_f16x2(f3.x * down, f3.y * down));
          }
        const float mine = fabsf(a.scale_log2) * pow2f(sh);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          fac[q][r] = __shfl_sync(0xffffffffu, mine, 4 * (2 * t + r));
          if (!dec_tile_row<ROWS>(a, cur, 8 * q + 2 * t + r, i0, hd)) i0 = cur.x.w.n - 1;
          attn_seen(a, cur.x.w, i0, lo[q][r], hi[q][r]);
          m[q][r] = -INFINITY;
          l[q][r] = 0.f;
        }
      }
      // what any and every row of the tile sees
      dec_tile_row<ROWS>(a, cur, 0, i0, hd);
      if (!dec_tile_row<ROWS>(a, cur, ROWS - 1, i1, hd)) i1 = cur.x.w.n - 1;
      attn_seen(a, cur.x.w, i0, lo_any, hi_all);
      attn_seen(a, cur.x.w, i1, lo_all, hi_any);

      bool large = false;       // some row's reference is past kAttnLarge

      float o[NT][CH / 2][4];   // value tile j: dims CH g + 2j (0, 1), CH g + 2j + 1 (2, 3)
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int j = 0; j < CH / 2; ++j) o[q][j][0] = o[q][j][1] = o[q][j][2] = o[q][j][3] = 0.f;

#pragma unroll 1
      for (int st = 0; st < nseg; ++st) {
        dec_fetch<D, NT>(a, ld, off, n_warp, ring, lane);
        cp_async_wait<Sh::STAGES - 1>();
        const uint32_t meta[2] = {dec_scales(ld, done, 0), dec_scales(ld, done, 1)};
        ++done;
        __syncwarp();
        const uint8_t* base = ringp + slot_in * (2 * Sh::HALF);
        const uint8_t* sp = base + lane * 16;
        const int p0 = (cur.x.s0 + cur.s + st) << 5;
        slot_in = slot_in + 1 == Sh::STAGES ? 0 : slot_in + 1;
        if (!((meta[0] | meta[1]) >> 16) || p0 >= hi_any || p0 + 32 <= lo_any) continue;
        // ---- scores: (tokens g, g + 8 of a half) x (rows 2t, 2t + 1) ----
        float s[NT][2][4];
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) s[q][h][0] = s[q][h][1] = s[q][h][2] = s[q][h][3] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 w[2][2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              w[h][i] = *reinterpret_cast<const uint4*>(sp + h * Sh::HALF + (i * (D / 64) + c) * 512);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x2(k == 0 ? w[h][0].x : k == 1 ? w[h][0].y : k == 2 ? w[h][0].z : w[h][0].w,
                              a0, a2);
              e4m3x4_to_f16x2(k == 0 ? w[h][1].x : k == 1 ? w[h][1].y : k == 2 ? w[h][1].z : w[h][1].w,
                              a1, a3);
#pragma unroll
              for (int q = 0; q < NT; ++q)
                mma_f16_16816(s[q][h], a0, a1, a2, a3, qf[q][4 * c + k].x, qf[q][4 * c + k].y);
            }
          }
        }
        // ---- weights ----
        float ke[2], ev[2], un[2];   // ev: down to kKvExpLow
        int more[2];                 // what is left of it below that
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = (int)((meta[h] >> 8) & 0xFFu) - 128;
          ke[h] = pow2f((int)(meta[h] & 0xFFu) - 128);
          more[h] = max(kKvExpLow - e, 0);
          ev[h] = (float)(e + more[h]);
          un[h] = pow2f(-e - more[h]);
        }
        const bool low = (more[0] | more[1]) != 0;
        const float evt[2] = {ev[0] - (float)more[0], ev[1] - (float)more[1]};
        const bool masked = p0 + 32 > hi_all || p0 < lo_all || !((meta[0] & meta[1]) >> 16);
        if (masked) {
#pragma unroll
          for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) {   // half i / 4, token g + 8 (i / 2 % 2), row i % 2
              const int j = p0 + 16 * (i >> 2) + 8 * ((i >> 1) & 1) + g;
              if (!(meta[i >> 2] >> 16) || j < lo[q][i & 1] || j >= hi[q][i & 1])
                s[q][i >> 2][i & 3] = -INFINITY;
            }
        }
        float x[NT][2];
        bool up = false;
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            // (a factor that underflowed to 0 makes NaN of -infinity, which fmaxf drops)
            float v = fmaxf(fmaf(fmaxf(s[q][0][r], s[q][0][2 + r]), fac[q][r] * ke[0], evt[0]),
                            fmaf(fmaxf(s[q][1][r], s[q][1][2 + r]), fac[q][r] * ke[1], evt[1]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            x[q][r] = v - kDecLead;
            up |= x[q][r] > m[q][r];
          }
        if (__any_sync(0xffffffffu, up)) {
          bool past = false;
#pragma unroll
          for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float n = fmaxf(m[q][r], x[q][r]);
              past |= n > -INFINITY && fabsf(n) >= kAttnLarge;
              const float half = attn_half_factor(m[q][r], n), d = half * half;
              m[q][r] = n;
              l[q][r] = l[q][r] * half * half;
#pragma unroll
              for (int j = 0; j < CH / 2; ++j) {
                o[q][j][r] *= d;
                o[q][j][2 + r] *= d;
              }
            }
          large |= __any_sync(0xffffffffu, past);
        }
        uint32_t pb[NT][2][2];
#pragma unroll
        for (int q = 0; q < NT; ++q) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float ref = m[q][r] == -INFINITY ? 0.f : m[q][r];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float f = fac[q][r] * ke[h], c = ev[h] - ref;
              float t0 = fmaf(s[q][h][r], f, c), t1 = fmaf(s[q][h][2 + r], f, c);
              if (large) {
                const float b = (float)more[h];
                t0 = fmaf(s[q][h][r], f, evt[h]) - ref;
                t1 = fmaf(s[q][h][2 + r], f, evt[h]) - ref;
                // (the lead rounded up to a step of t; a NaN stays)
                t0 = (t0 > 15.f ? 15.f : t0) + b;
                t1 = (t1 > 15.f ? 15.f : t1) + b;
              }

              s[q][h][r] = exp2_approx(t0);
              s[q][h][2 + r] = exp2_approx(t1);
            }
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int j = p0 + 16 * (i >> 2) + 8 * ((i >> 1) & 1) + g;
              if (!(meta[i >> 2] >> 16) || j < lo[q][i & 1] || j >= hi[q][i & 1])
                s[q][i >> 2][i & 3] = 0.f;
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              l[q][r] = fmaf(un[h], s[q][h][r] + s[q][h][2 + r], l[q][r]);
          if (low) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[q][h][i] *= pow2f(-more[h]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            pb[q][h][0] = movmatrix(pack_f16x2(s[q][h][0], s[q][h][1]));
            pb[q][h][1] = movmatrix(pack_f16x2(s[q][h][2], s[q][h][3]));
          }
        }
        // ---- values ----
        uint32_t nan = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* hp = sp + h * Sh::HALF;
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
            e4m3x4_to_f16x2(__byte_perm(vw[2][c], vw[3][c], 0x5140), a2, a3);
            e4m3x4_to_f16x2(__byte_perm(vw[0][c], vw[1][c], 0x7362), b0, b1);
            e4m3x4_to_f16x2(__byte_perm(vw[2][c], vw[3][c], 0x7362), b2, b3);
#pragma unroll
            for (int q = 0; q < NT; ++q) {
              mma_f16_16816(o[q][2 * c], a0, a1, a2, a3, pb[q][h][0], pb[q][h][1]);
              mma_f16_16816(o[q][2 * c + 1], b0, b1, b2, b3, pb[q][h][0], pb[q][h][1]);
            }
          }
        }
        if (masked && __any_sync(0xffffffffu, nan != 0)) {
          // lanes 4g + tt hold dims CH g .. of tokens 2tt, 2tt + 1, 2tt + 8, 2tt + 9
          const float qnan = __int_as_float(0x7FFFFFFF);
#pragma unroll 1
          for (int tok = 0; tok < 32; ++tok) {
            const int i = (tok & 1) + 2 * ((tok >> 3) & 1), j = p0 + tok;
            const bool there = ((tok < 16 ? meta[0] : meta[1]) >> 16) != 0;
            const int src = 4 * g + ((tok & 7) >> 1);
            const uint8_t* hp = base + (tok >> 4) * Sh::HALF + src * 16;
            const uint8_t* p =
                D == 128 ? hp + (Sh::KP + i) * 512 : hp + (Sh::KP + (i >> 1)) * 512 + (i & 1) * 8;
#pragma unroll
            for (int jj = 0; jj < CH; ++jj) {
              if ((p[jj] & 0x7F) != 0x7F) continue;
#pragma unroll
              for (int q = 0; q < NT; ++q)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                  if (there && j >= lo[q][r] && j < hi[q][r]) o[q][jj >> 1][2 * (jj & 1) + r] = qnan;
            }
          }
          __syncwarp();
        }
      }

      // ---- the tile's end, or the run's: then the ring is free ----
      const bool begins = cur.s == 0, ends = cur.s + nseg == cur.x.S, last = done == n_warp;
      if (last) {
        cp_async_wait<0>();
        __syncwarp();
      }
      float* slot = last ? reinterpret_cast<float*>(ringp) : slots + warp * Sh::SLOT;
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float v = l[q][r];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          const int row = 8 * q + 2 * t + r;
          if (!dec_tile_row<ROWS>(a, cur, row, i0, hd)) continue;
          if (begins && ends) {
            const float inv = attn_inverse(v);
            const long long tok = cur.x.w.tok + i0;
            uint16_t* dst = a.out + tok * a.o_ts + hd * a.o_hs + g * CH;
#pragma unroll
            for (int j = 0; j < CH / 2; j += 4)
              *reinterpret_cast<uint4*>(dst + 2 * j) =
                  make_uint4(pack16(o[q][j][r] * inv, o[q][j][2 + r] * inv, a.f16),
                             pack16(o[q][j + 1][r] * inv, o[q][j + 1][2 + r] * inv, a.f16),
                             pack16(o[q][j + 2][r] * inv, o[q][j + 2][2 + r] * inv, a.f16),
                             pack16(o[q][j + 3][r] * inv, o[q][j + 3][2 + r] * inv, a.f16));
            if (g == 0 && a.lse) a.lse[tok * a.heads + hd] = attn_lse(m[q][r], v);
          } else {
#pragma unroll
            for (int j = 0; j < CH / 2; ++j)
              *reinterpret_cast<float2*>(slot + row * D + j * 16 + 2 * g) =
                  make_float2(o[q][j][r], o[q][j][2 + r]);
            if (g == 0) {
              slot[ROWS * D + row] = m[q][r];
              slot[ROWS * D + ROWS + row] = v;
            }
          }
        }
      if (!(begins && ends) && lane == 0)
        s_piece[2 * warp + last] = {1 | (begins ? 2 : 0) | (ends ? 4 : 0), cur.h, cur.m,
                                    cur.x.w.tok, cur.x.w.n, cur.x.S,
                                    first + done - nseg - cur.s};
      if (!last) dec_next_tile<ROWS>(a, cur);
    }
  }
  __syncthreads();

  // ---- join the warps' pieces: consecutive pieces up to the next that begins
  // a tile are one tile; an item (tile, row) a warp ----
  const int state = lane < 2 * W ? s_piece[lane].state : 0;
  const unsigned valid = __ballot_sync(0xffffffffu, state & 1);
  const unsigned begin = __ballot_sync(0xffffffffu, (state & 3) == 3) & valid;
  const unsigned end = __ballot_sync(0xffffffffu, (state & 5) == 5) & valid;
  if (valid == 0) return;
  const unsigned heads = begin | (valid & -valid);   // first piece of each tile
  __shared__ DecJob s_job[2 * W];
  __shared__ int s_open[2];   // pieces of the tiles that the CTA's own ends cut
  const int jobs = __popc(heads);
  if (threadIdx.x < 2) s_open[threadIdx.x] = -1;
  __syncthreads();
  if (warp == 0 && ((heads >> lane) & 1u)) {
    const unsigned later = heads & ~((2u << lane) - 1);
    const unsigned span =
        valid & ~((1u << lane) - 1) & (later ? (later & -later) - 1 : ~0u);
    const bool b = (begin >> lane) & 1u, e = (end >> (31 - __clz(span))) & 1u;
    const DecPiece& p = s_piece[lane];
    s_job[__popc(heads & ((1u << lane) - 1))] = {
        slots, b && e ? nullptr : slots + (W + (b ? 1 : 0)) * Sh::SLOT,
        reinterpret_cast<const float*>(dec_smem), Sh::SLOT, 0, Sh::RING / 4, span, p.h,
        p.m, p.tok, p.n};
    if (!(b && e)) s_open[b ? 1 : 0] = lane;
  }
  __syncthreads();
  dec_join<D, ROWS>(&s_out, s_job, jobs, warp, W);

  dec_join_ctas<D, ROWS, W, Sh::SLOTS * Sh::SLOT, Sh::SLOT, false>(
      a, a.partial + W * Sh::SLOT, share, s_open[0] < 0 ? nullptr : s_piece + s_open[0],
      s_open[1] < 0 ? nullptr : s_piece + s_open[1], &s_out, s_job);
}

}  // namespace moe
