// Attention over the 8-bit cache for many query rows per KV head (verify
// steps, prompts): tcgen05 tensor cores.
//
// An item is TILE rows (query i, head of the group: row i * group + head) of
// one KV head of one batch row: 256 as two streams of 128 rows that share
// every tile of 128 keys (PAIR), or 128 rows whose two streams take the even
// and the odd tiles of keys (the launch says when).  The streams
// alternate on the tensor cores: while one's scores (S = Q K^T, M = 128 rows,
// N = 128 keys) go through the softmax, the other's products run.
//
// Roles (12 warps, 168 registers a thread): warps 0..3 and 4..7, one stream
// each, a thread a row: scores from tensor memory, running maximum and sum,
// weights back into tensor memory (in the columns of their scores) as the A
// operand of O += P V; the stream's first warp then issues its products, the
// values' and the next scores', which the stream waits for anyway.  Warps 8..11
// fetch codes, convert them to f16 and lay them out in shared memory as K-major
// core matrices (K rows = keys, V^T rows = dims, transposed in registers).
// Accumulators and S live in tensor memory (2 x 128 columns of S, 2 x D of O).
//
// Bounds: 4 * 128 * 128 * D operations of a pair of products take 0.67 us of
// an SM's tensor cores at D = 128; beside them 128 x 128 exponentials and
// their arithmetic per stream and tile, and 32 KB of codes to convert per tile
// of keys, which two streams share.
//
// Scales and weights as in kv_attention.cuh: t = score * log2(e) + ev per 16
// keys, weights 2^(t - M).  M is set 7 below the maximum, and again only when
// a weight passes 2^15, so that O in tensor memory is rarely rescaled and the
// largest weight stays between 2^7 and 2^15: f16 keeps all bits of keys up to
// 2^21 behind a leading one.  (Prompts 937 us; set 8 below 948, 10 below 993.)
//
// Work split and joins as there, in tiles of 128 keys in the order (batch row,
// row tile, KV head, keys).
//
// Measured at D = 128: prompts of 2,049 to 4,096 tokens behind 4,097 to 8,191,
// 32 heads over 8: 939 us, 915 TFLOP/s, 48% of the dense rate: 4,900 cycles a
// tile of 256 x 128, of which the products take 2,100; no unit is busy more
// than 40% of the time, the chain scores, softmax, values of two streams is
// (a softmax 2,400 cycles beside the other stream and the converters).  8 rows
// of 8 queries, 64 heads over 8, 4,090 to 8,185 tokens: 78 us, of which 11 before
// the first scores, 1.6 a tile of 128 x 128 (the converters'), 15 for the joins.
#pragma once

#include "kv_attention.cuh"
#include "tcgen05.cuh"

namespace moe {

constexpr int kPrWarps = 12;
constexpr int kPrThreads = 32 * kPrWarps;
constexpr int kPrKeys = 128;
// Tiles of keys a CTA takes at least (64 queries of 300 tokens: 40 us, with 2
// tiles 55), and may take over an equal share to keep to one item (few items
// are then split each on its own, as in kv_attention.cuh: 4 rows of 64 queries
// and 64 to 500 tokens 38 us against 76, 4 of 16 and 4,090 to 8,185 tokens 78
// against 97, 8 queries of 40,000 tokens 91 against 108, 8 rows of 8 and 4,090 to
// 8,185 77 against 82; with up to 16 tiles more 86).
constexpr int kPrLeast = 4;
constexpr int kPrSlack = 8;
constexpr float kPrFar = 0x1p100f;               // an exponent that no score comes near
constexpr float kPrLead = 7.f, kPrGrow = 15.f;   // the largest weight: set to, at most (log2)

template <int D, bool PAIR>
struct PrShape {
  static constexpr int TILE = PAIR ? 256 : 128;
  // All operands lie as 8 x 16 byte core matrices (8 rows or keys, 8 dims),
  // 128 bytes each, the 16 of 8 dims one after the other: element (row, dim) at
  // GROUP (dim / 8) + 16 row + 2 (dim % 8).  Q and K are K-major operands of
  // the scores in this order, V an MN-major one of the values (N = dims).  The
  // 16 bytes that pad a group of K and V spread the converters' stores over the
  // banks.
  static constexpr int QGROUP = 2048, GROUP = 2064;
  static constexpr int QBYTES = D / 8 * QGROUP, KBYTES = D / 8 * GROUP, VBYTES = KBYTES;
  // queries, one tile of keys, two of values, and three half tiles of codes
  // (keys or values) on their way: a tile and a half ahead of the converters
  static constexpr int KOFF = (PAIR ? 2 : 1) * QBYTES, VOFF = KOFF + KBYTES;
  static constexpr int ROFF = VOFF + 2 * VBYTES, RAW = kPrKeys * D, RAWS = 3;
  static constexpr int SMEM = ROFF + RAWS * RAW;
  // a slot of partial sums: O [TILE][D], m [TILE], l [TILE]; two a CTA
  static constexpr int SLOT = TILE * D + 2 * TILE;
  static constexpr int OCOL = 256;   // tensor memory: S at 0 and 128, O at OCOL + D t
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ void fma_f32x2(float& a, float& b, float g, float off) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\t"
      "mov.b64 z, {%3, %3};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(g), "f"(off));
}
__device__ __forceinline__ void add_f32x2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
// D += A B with A (f16, two of K a column) in tensor memory.
__device__ __forceinline__ void umma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f16: f16 x f16 -> fp32, both K-major, M = 128.
__device__ __forceinline__ constexpr uint32_t umma_idesc_f16(uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}
constexpr uint32_t kUmmaTransposeB = 1u << 16;   // B is MN-major

// ---------------------------------------------------------------------------
// Items and schedule
// ---------------------------------------------------------------------------
// Tiles of keys of the item of row tile m: [s0, s0 + S).
template <int TILE>
__device__ __forceinline__ void pr_span(const AttnArgs& a, const AttnRow& w, int m, int& s0,
                                        int& S) {
  const unsigned g = (unsigned)a.group;
  const int i0 = (int)((unsigned)TILE * m / g);
  const int i1 = min(w.n - 1, (int)(((unsigned)TILE * m + TILE - 1) / g));
  int lo, hi, unused;
  attn_seen(a, w, i0, lo, unused);
  attn_seen(a, w, i1, unused, hi);
  s0 = lo >> 7;
  S = max(1, (int)(((unsigned)hi + 127) >> 7) - s0);   // nothing seen: one tile, for the zeros
}

template <int TILE>
__device__ __forceinline__ int pr_tiles(const AttnArgs& a, const AttnRow& w) {
  return (int)(((unsigned)w.n * (unsigned)a.group + TILE - 1) / TILE);
}

struct PrCursor {
  int r, m, h, s;   // batch row, row tile, KV head, next tile of keys (from s0)
  AttnRow w;
  int M, s0, S;
};

template <int TILE>
__device__ __forceinline__ void pr_next_item(const AttnArgs& a, PrCursor& c) {
  c.s = 0;
  if (++c.h < a.c.heads) return;
  c.h = 0;
  if (++c.m >= c.M) {
    c.m = 0;
    do {
      if (++c.r >= a.rows) return;
      c.w = attn_row(a, c.r);
      c.M = pr_tiles<TILE>(a, c.w);
    } while (c.M == 0);
  }
  pr_span<TILE>(a, c.w, c.m, c.s0, c.S);
}

// Parts of at most `most` tiles of keys that an item of S is cut into.
__device__ __forceinline__ int pr_parts(int S, int most) { return (S - 1) / most + 1; }

// Sum of the parts over a batch row's row tiles: by the lane alone, or with
// the warp's lanes taking m = lane, lane + 32, ...
template <int TILE>
__device__ __forceinline__ long long pr_row_tiles(const AttnArgs& a, const AttnRow& w, int most,
                                                  int first, int step) {
  const int M = pr_tiles<TILE>(a, w);
  long long sum = 0;
  for (int m = first; m < M; m += step) {
    int s0, S;
    pr_span<TILE>(a, w, m, s0, S);
    sum += pr_parts(S, most);
  }
  return sum;
}

// The same of batch row r, every lane of a warp with its own r (r < 0:
// none); rows of many row tiles are summed by the whole warp.
template <int TILE>
__device__ __forceinline__ long long pr_warp_tiles(const AttnArgs& a, int most, int r) {
  constexpr int kAlone = 8;
  AttnRow w{0, 0, 0};
  if (r >= 0) w = attn_row(a, r);
  const bool big = pr_tiles<TILE>(a, w) > kAlone;
  long long sum = big ? 0 : pr_row_tiles<TILE>(a, w, most, 0, 1);
  for (unsigned rest = __ballot_sync(0xffffffffu, big); rest; rest &= rest - 1) {
    const int src = __ffs(rest) - 1;
    const AttnRow o{0, __shfl_sync(0xffffffffu, w.n, src), __shfl_sync(0xffffffffu, w.seq, src)};
    long long v = pr_row_tiles<TILE>(a, o, most, threadIdx.x & 31, 32);
#pragma unroll
    for (int k = 16; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
    if ((threadIdx.x & 31) == src) sum = v;
  }
  return sum * a.c.heads;
}

// This CTA's share of the tiles of keys and its cursor there; every thread calls.
template <int TILE>
__device__ __forceinline__ void pr_schedule(const AttnArgs& a, DecShare& sh, PrCursor& cur) {
  __shared__ long long s_sum[2][kPrWarps];
  __shared__ long long s_left;
  __shared__ int s_row, s_m;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = (a.rows + kPrWarps - 1) / kPrWarps;
  const int r0 = min(a.rows, warp * chunk), r1 = min(a.rows, r0 + chunk);
  auto sums = [&](int most, int set) {
    long long v = 0;
    for (int r = r0; r < r1; r += 32)
      v += pr_warp_tiles<TILE>(a, most, r + lane < r1 ? r + lane : -1);
#pragma unroll
    for (int k = 16; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
    if (lane == 0) s_sum[set][warp] = v;
    return v;
  };
  long long sum = sums(1, 0), total = 0, items = 0, before = 0;
  sums(INT32_MAX, 1);
  __syncthreads();
  for (int w = 0; w < kPrWarps; ++w) {
    if (w == warp) before = total;
    total += s_sum[0][w];
    items += s_sum[1][w];
  }
  // few items: each split on its own (as in dec_schedule) into parts of at most
  // `most` tiles, if there are no more parts than CTAs; with most = total / spare
  // there never are
  const long long even = max((total + gridDim.x - 1) / gridDim.x, (long long)kPrLeast);
  const long long spare = (long long)gridDim.x - items;
  int most = 1;
  bool apart = false;
  if (spare >= 0 && total > 0) {
    most = (int)(even + kPrSlack);
    if (spare > 0)
      most = (int)min((long long)most, max((total + spare - 1) / spare, (long long)kPrLeast));
    __syncthreads();
    const long long parts = sums(most, 0);
    __syncthreads();
    long long all = 0, first = 0;
    for (int w = 0; w < kPrWarps; ++w) {
      if (w == warp) first = all;
      all += s_sum[0][w];
    }
    apart = all <= gridDim.x;
    if (apart) {
      sum = parts;
      total = all;
      before = first;
    } else {
      most = 1;
    }
  }
  const long long u0 = apart ? blockIdx.x : even * blockIdx.x;
  sh.per = apart ? 0 : even;
  sh.u0 = apart ? 0 : u0;
  sh.n = apart ? (u0 < total ? 1 : 0) : min(even, total - u0);
  if (sh.n > 0 && u0 >= before && u0 < before + sum) {
    for (int r = r0;; r += 32) {
      const long long v = pr_warp_tiles<TILE>(a, most, r + lane < r1 ? r + lane : -1);
      long long inc = v;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, k);
        if (lane >= k) inc += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + inc > u0);
      if (!past) {
        before += __shfl_sync(0xffffffffu, inc, 31);
        continue;
      }
      const int src = __ffs(past) - 1;
      before += __shfl_sync(0xffffffffu, inc - v, src);
      // the row tile: lanes take 32 of them at a time
      const AttnRow w = attn_row(a, r + src);
      for (int m = 0;; m += 32) {
        int s0, S = 0;
        if (m + lane < pr_tiles<TILE>(a, w)) pr_span<TILE>(a, w, m + lane, s0, S);
        const long long x = S ? (long long)pr_parts(S, most) * a.c.heads : 0;
        long long y = x;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const long long o = __shfl_up_sync(0xffffffffu, y, k);
          if (lane >= k) y += o;
        }
        const unsigned in = __ballot_sync(0xffffffffu, before + y > u0);
        if (!in) {
          before += __shfl_sync(0xffffffffu, y, 31);
          continue;
        }
        const int mm = __ffs(in) - 1;
        before += __shfl_sync(0xffffffffu, y - x, mm);
        if (lane == 0) {
          s_row = r + src;
          s_m = m + mm;
          s_left = u0 - before;
        }
        break;
      }
      break;
    }
  }
  __syncthreads();
  if (sh.n <= 0) return;
  cur.r = s_row;
  cur.m = s_m;
  cur.w = attn_row(a, cur.r);
  cur.M = pr_tiles<TILE>(a, cur.w);
  pr_span<TILE>(a, cur.w, cur.m, cur.s0, cur.S);
  const int parts = pr_parts(cur.S, most);
  cur.h = (int)(s_left / parts);
  const int part = (int)(s_left - (long long)cur.h * parts);
  cur.s = part;
  if (apart) {
    cur.s = (int)((long long)cur.S * part / parts);
    sh.n = (long long)cur.S * (part + 1) / parts - cur.s;
    sh.c0 = blockIdx.x - part;
    sh.ctas = parts;
  }
}

// What every and any row of the item sees.
template <int TILE>
__device__ __forceinline__ void pr_seen(const AttnArgs& a, const PrCursor& c, int& lo_all,
                                        int& hi_all) {
  const unsigned g = (unsigned)a.group;
  int unused;
  attn_seen(a, c.w, (int)((unsigned)TILE * c.m / g), unused, hi_all);
  attn_seen(a, c.w, min(c.w.n - 1, (int)(((unsigned)TILE * c.m + TILE - 1) / g)), lo_all, unused);
}

// Keys at p0 .. p0 + 127 that some row of the item does not see.
__device__ __forceinline__ bool pr_masked(int p0, int lo_all, int hi_all) {
  return p0 + kPrKeys > hi_all || p0 < lo_all;
}

// ---------------------------------------------------------------------------
// Shared state
// ---------------------------------------------------------------------------
struct PrShared {
  // operands: tile n of keys uses barriers n & 1 (the keys' one buffer too: the
  // second stream may wait for a tile while the one before is not there yet)
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t sfull[2], ofull[2];                   // products of each stream
  uint64_t drained[2];                           // all of them, where a wait ran out
  uint32_t tmem;
  int dead;                 // a wait ran out
  int nan[8];               // by segment: a NaN value in a masked tile
  int open[2];              // the CTA's tiles cut by its ends: set
  DecPiece piece[2];        // and which they are
  // by tile of keys, of 16 keys each: 2^ek, ev, 2^-ev, ev; where ev is below
  // kKvExpLow: 2^ek, kPrFar, 2^-kKvExpLow, ev
  float4 scale[4][8];
  float m1[128], l1[128];   // the second stream's, when the two are joined
  unsigned nan1[4][128];
  DecOut out;
  DecShare share;
  DecJob job[2];
};

// Waits for a phase, two seconds at most; then marks the CTA dead, whose waits
// all end at once and whose results become NaN.
__device__ __forceinline__ void pr_wait(uint64_t* bar, uint32_t parity, PrShared& sh) {
  if (mbar_try_wait_long(bar, parity)) return;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait_long(bar, parity)) {
    if (*(volatile int*)&sh.dead) return;
    if (global_ns() - t0 > kWaitLimitNs) {
      *(volatile int*)&sh.dead = 1;
      return;
    }
  }
}

// ---------------------------------------------------------------------------
// Converters (warps 8..11): a tile of keys from codes to f16 operands
// ---------------------------------------------------------------------------
struct PrTile {      // a tile of keys as one lane sees it
  int id;            // lanes 0..7: block of the lane's 16 keys, -1: none
  int p0, seq, h, seg;
  bool masked, there;   // there: the tile exists
};

template <int TILE>
struct PrFeed {      // walks the CTA's tiles of keys
  PrCursor c;
  long long left;
  int seg, lo_all, hi_all;

  __device__ __forceinline__ void take(const AttnArgs& a, PrTile& t, int lane) {
    t.there = left > 0;
    t.id = -1;
    if (!t.there) return;
    t.p0 = (c.s0 + c.s) << 7;
    t.seq = c.w.seq;
    t.h = c.h;
    t.seg = seg;
    t.masked = pr_masked(t.p0, lo_all, hi_all);
    const int p = t.p0 + 16 * lane;
    if (lane < 8 && p < t.seq) t.id = __ldg(a.table + c.r * a.table_stride + (p >> a.c.bs_log2));
    if (--left > 0 && ++c.s == c.S) {
      pr_next_item<TILE>(a, c);
      ++seg;
      pr_seen<TILE>(a, c, lo_all, hi_all);
    }
  }
};

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Each thread copies (cp.async) the pieces that it converts itself into a ring
// of its own, so the copies need no barrier.  (Fetched into registers half a
// tile ahead, a tile took 4,700 cycles, mostly waiting.)  A piece is 16 dims of
// a key; four neighbouring lanes take neighbouring pieces (with neighbouring
// keys a copy of 512 bytes took 37 cycles of the L1).
template <int D, bool PAIR>
__device__ __forceinline__ void pr_convert(const AttnArgs& a, PrShared& sh, uint8_t* smem,
                                           const PrCursor& start, long long n_units) {
  using S = PrShape<D, PAIR>;
  constexpr int C = D / 64;                // pieces of a key a thread, 4 keys
  const int ct = threadIdx.x - 256, lane = ct & 31, warp = ct >> 5;
  const int chunk = lane & 3, key = 32 * warp + (lane >> 2);   // keys key + 8 i, dims 16 (chunk + 4 c)
  PrFeed<S::TILE> feed;
  feed.c = start;
  feed.left = n_units;
  feed.seg = 0;
  pr_seen<S::TILE>(a, start, feed.lo_all, feed.hi_all);
  PrTile t0, t1, t2, t3;      // being converted, the two being fetched, being looked up
  // (a tile of keys begins with a block)
  const int bs1 = (1 << a.c.bs_log2) - 1;
  const long long in_block[2] = {(key & bs1) * a.c.tstride + chunk * 16,
                                 ((key + 16) & bs1) * a.c.tstride + chunk * 16};
  // codes that few row tiles read leave L2 first (8 row tiles: 441 us against 454
  // when they may stay); those of a prompt are read again
  const uint64_t policy = PAIR ? policy_evict_normal() : policy_evict_first();
  const uint32_t raw = smem_addr(smem) + S::ROFF + ct * 16;
  int in_slot = 0, out_slot = 0;

  // where a lane's keys of a tile lie, and how many of each group of 16, from
  // its first on, are cached: the same for keys and values
  struct Place {
    long long at[2];
    int left[2];
  };
  auto place = [&](const PrTile& t) {
    Place w;
    const long long block =
        t.id >= 0 && t.id < a.c.n_blocks
            ? (long long)t.id * a.c.bstride + (long long)t.h * a.c.hstride : -1;
    // the warp's 32 keys lie in two groups of 16, each in one block
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const long long at = __shfl_sync(0xffffffffu, block, 2 * warp + g);
      w.left[g] = t.there && at >= 0 ? t.seq - t.p0 - key - 16 * g : 0;
      w.at[g] = w.left[g] > 0 ? at + in_block[g] : 0;
    }
    return w;
  };
  const long long ts8 = 8 * a.c.tstride;
  auto fetch = [&](const Place& w, const uint8_t* codes) {
    const uint32_t dst = raw + in_slot * S::RAW;
    in_slot = in_slot + 1 == S::RAWS ? 0 : in_slot + 1;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint8_t* src = codes + w.at[g];
      const bool in = w.left[g] > 0, in1 = w.left[g] > 8;
      const uint8_t* src1 = in1 ? src + ts8 : codes;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        cp_async<16>(dst + (2 * g * C + c) * 2048, src + (in ? 64 * c : 0), in, policy);
        cp_async<16>(dst + ((2 * g + 1) * C + c) * 2048, src1 + (in1 ? 64 * c : 0), in1, policy);
      }
    }
    cp_async_commit();
  };
  auto convert = [&](uint8_t* to, bool drop) {
    const uint8_t* from = smem + S::ROFF + out_slot * S::RAW + ct * 16;
    out_slot = out_slot + 1 == S::RAWS ? 0 : out_slot + 1;
    uint32_t any = 0;
    uint4 w[4 * C];   // all loads first: the stores could be to what they read
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) w[i] = *reinterpret_cast<const uint4*>(from + i * 2048);
    if (drop) {
#pragma unroll
      for (int i = 0; i < 4 * C; ++i) {
        w[i].x = drop_nan4(w[i].x, any);
        w[i].y = drop_nan4(w[i].y, any);
        w[i].z = drop_nan4(w[i].z, any);
        w[i].w = drop_nan4(w[i].w, any);
      }
    }
    uint8_t* d0 = to + 2 * chunk * S::GROUP + key * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint4& v = w[i * C + c];
        uint8_t* d = d0 + 8 * c * S::GROUP + 8 * i * 16;
        uint4 x, y;
        e4m3x4_to_f16x2(v.x, x.x, x.y);
        e4m3x4_to_f16x2(v.y, x.z, x.w);
        e4m3x4_to_f16x2(v.z, y.x, y.y);
        e4m3x4_to_f16x2(v.w, y.z, y.w);
        *reinterpret_cast<uint4*>(d) = x;
        *reinterpret_cast<uint4*>(d + S::GROUP) = y;
      }
    fence_async_shared();
    return any;
  };
  // scale bytes of a tile, lanes 0..7 of the first converter warp
  uint32_t ek = 0, ev = 0;
  auto fetch_scales = [&](const PrTile& t) {
    if (warp == 0 && t.id >= 0 && t.id < a.c.n_blocks) {
      const long long at = (long long)t.id * a.c.sstride + t.h;
      ek = __ldg(a.c.ks + at);
      ev = __ldg(a.c.vs + at);
    }
  };

  feed.take(a, t0, lane);
  feed.take(a, t1, lane);
  feed.take(a, t2, lane);
  Place p1 = place(t0), p2;   // of the two tiles being fetched
  fetch(p1, a.c.k);
  fetch(p1, a.c.v);
  p1 = place(t1);
  fetch(p1, a.c.k);
  fetch_scales(t0);
#pragma unroll 1
  for (int n = 0; t0.there; ++n) {
    feed.take(a, t3, lane);
    const bool block = t0.id >= 0 && t0.id < a.c.n_blocks;
    // ---- keys ----
    if (n > 0) pr_wait(&sh.kempty[(n - 1) & 1], ((n - 1) >> 1) & 1, sh);
    cp_async_wait<2>();
    if (warp == 0 && lane < 8) {
      const int e = kv_exp(ev);
      // a block outside the cache: weights 0
      sh.scale[n & 3][lane] =
          block ? make_float4(pow2f(kv_exp(ek)), e < kKvExpLow ? kPrFar : (float)e,
                              pow2f(-max(e, kKvExpLow)), (float)e)
                : make_float4(0.f, -INFINITY, 0.f, -INFINITY);
    }
    convert(smem + S::KOFF, false);
    mbar_arrive(&sh.kfull[n & 1]);
    fetch_scales(t1);
    fetch(p1, a.c.v);
    p2 = place(t2);
    // ---- values ----
    const int stage = n & 1;
    if (n > 1) pr_wait(&sh.vempty[stage], ((n >> 1) - 1) & 1, sh);
    cp_async_wait<2>();
    // a weight of 0 does not keep a NaN out of the sums: in masked tiles NaN
    // codes leave here and are given back to the rows that see them at the end
    if (convert(smem + S::VOFF + stage * S::VBYTES, t0.masked)) atomicOr(&sh.nan[t0.seg & 7], 1);
    mbar_arrive(&sh.vfull[stage]);
    fetch(p2, a.c.k);
    p1 = p2;
    t0 = t1;
    t1 = t2;
    t2 = t3;
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------
// Products of a stream, issued by its first warp; n: the tile of keys
// ---------------------------------------------------------------------------
// All lanes of the warp run this code and one issues: stream and stage are
// template arguments and tensor memory is allocated whole (address 0), so that
// every operand of an MMA is a constant of the code.  (Built in one thread's
// registers, the operands of an MMA cost 145 cycles to issue, more than twice
// its time on the tensor cores.)
__device__ __forceinline__ void pr_wait_keys(PrShared& sh, int n) {
  pr_wait(&sh.kfull[n & 1], (n >> 1) & 1, sh);
}
__device__ __forceinline__ void pr_wait_values(PrShared& sh, int n) {
  pr_wait(&sh.vfull[n & 1], (n >> 1) & 1, sh);
}
// The streams that share tiles of keys issue in turns (their first warps meet
// at a barrier of their own, where nobody polls): the queue of the tensor cores
// is short, so two streams that issue together both wait for both, compute
// their softmax together, and the tensor cores idle meanwhile.
__device__ __forceinline__ void pr_take_turn(int t) {
  asm volatile("bar.sync %0, 64;" ::"r"(8 + t) : "memory");
}
__device__ __forceinline__ void pr_pass_turn(int t) {
  asm volatile("bar.arrive %0, 64;" ::"r"(8 + (t ^ 1)) : "memory");
}

template <int D, bool PAIR, int T>
__device__ __forceinline__ void pr_scores_of(PrShared& sh, uint32_t base, int n) {
  using S = PrShape<D, PAIR>;
  if (elect_one()) {
    const uint64_t dq = umma_desc(base + (PAIR ? T * S::QBYTES : 0), S::QGROUP, 128);
    const uint64_t dk = umma_desc(base + S::KOFF, S::GROUP, 128);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      umma_f16(128 * T, dq + (2 * S::QGROUP / 16) * k, dk + (2 * S::GROUP / 16) * k,
               umma_idesc_f16(kPrKeys), k > 0);
    umma_commit(&sh.sfull[T]);
    umma_commit(&sh.kempty[n & 1]);
  }
  __syncwarp();
}
template <int D, bool PAIR>
__device__ __forceinline__ void pr_scores(PrShared& sh, uint32_t base, int t, int n) {
  if (t == 0) pr_scores_of<D, PAIR, 0>(sh, base, n);
  else pr_scores_of<D, PAIR, 1>(sh, base, n);
}
template <int D, bool PAIR, int T, int STAGE>
__device__ __forceinline__ void pr_values_of(PrShared& sh, uint32_t base, uint32_t add) {
  using S = PrShape<D, PAIR>;
  if (elect_one()) {
    // MN-major: 128 bytes between groups of 8 keys, GROUP between groups of 8 dims
    const uint64_t dv = umma_desc(base + S::VOFF + STAGE * S::VBYTES, 128, S::GROUP);
    constexpr uint32_t idesc = umma_idesc_f16(D) | kUmmaTransposeB;
    umma_f16_ta(S::OCOL + D * T, 128 * T, dv, idesc, add);
#pragma unroll
    for (int k = 1; k < kPrKeys / 16; ++k)
      umma_f16_ta(S::OCOL + D * T, 128 * T + 8 * k, dv + (256 / 16) * k, idesc, 1);
    umma_commit(&sh.ofull[T]);
    umma_commit(&sh.vempty[STAGE]);
  }
  __syncwarp();
}
template <int D, bool PAIR>
__device__ __forceinline__ void pr_values(PrShared& sh, uint32_t base, int t, int n, bool add) {
  if (t == 0) {
    if (n & 1) pr_values_of<D, PAIR, 0, 1>(sh, base, add);
    else pr_values_of<D, PAIR, 0, 0>(sh, base, add);
  } else {
    if (n & 1) pr_values_of<D, PAIR, 1, 1>(sh, base, add);
    else pr_values_of<D, PAIR, 1, 0>(sh, base, add);
  }
}

// A dead CTA's products in flight, before their memory is given back (a stream's
// first warp; a tenth of a second at most).
__device__ __noinline__ void pr_drain(PrShared& sh, int t) {
  __syncwarp();
  if (elect_one()) umma_commit(&sh.drained[t]);
  for (int i = 0; i < 100 && !mbar_try_wait_long(&sh.drained[t], 0); ++i) {
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// Softmax (warps 0..7): a thread a row of its stream
// ---------------------------------------------------------------------------
// Barriers of one stream's threads and of both streams'.
__device__ __forceinline__ void pr_stream_sync(int t) {
  __syncwarp();
  asm volatile("bar.sync %0, 128;" ::"r"(5 + t) : "memory");
}
__device__ __forceinline__ void pr_streams_sync() {
  __syncwarp();
  asm volatile("bar.sync 3, 256;" ::: "memory");
}

// Dims (bits) in which the row sees a NaN value among the masked tiles of
// keys [first, end) (step `step`) of the item: the rare path.
template <int D>
__device__ __noinline__ void pr_nan_dims(const AttnArgs& a, const PrCursor& c, int first, int end,
                                         int step, int lo, int hi, int lo_all, int hi_all,
                                         unsigned* bits) {
  for (int s = first; s < end; s += step) {
    const int p0 = (c.s0 + s) << 7;
    if (!pr_masked(p0, lo_all, hi_all)) continue;
    for (int j = max(p0, lo); j < min(p0 + kPrKeys, hi); ++j) {
      const int id = a.table[c.r * a.table_stride + (j >> a.c.bs_log2)];
      if (id < 0 || id >= a.c.n_blocks) continue;
      const uint8_t* v = a.c.v + (long long)id * a.c.bstride + (long long)c.h * a.c.hstride +
                         (long long)(j & ((1 << a.c.bs_log2) - 1)) * a.c.tstride;
      for (int d = 0; d < D; ++d)
        if ((v[d] & 0x7F) == 0x7F) bits[d >> 5] |= 1u << (d & 31);
    }
  }
}

// The row's sums in tensor memory times `by`.
template <int D>
__device__ __forceinline__ void pr_scale_sums(uint32_t to, float by) {
#pragma unroll 1
  for (int k = 0; k < D / 16; ++k) {
    float o[16];
    tmem_ld16(to + 16 * k, o);
    tmem_wait_ld();
    uint32_t r[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(o[e] * by);
    tmem_st16(to + 16 * k, r);
  }
}

// A tile's weights where a row of the warp has scores past kAttnLarge, or sees
// keys whose ev is below kKvExpLow (an exponent of kPrFar stands for it, so
// that the pass over the scores ends up here): two passes, the maximum of t,
// then t - M, which is exact near M.  (M alone, its rounding as large as the
// growth that a pass allows, need not settle.)  The
// weights go into the columns of scores that are read already.  ofull: the
// sums' barrier, null where the segment has none yet; returns M and the sum.
template <int D>
__device__ __noinline__ float2 pr_weights_apart(PrShared& sh, const float4* sc, uint32_t ts,
                                                uint32_t to, int from, unsigned len, float fac,
                                                float m, float l, uint64_t* ofull,
                                                uint32_t parity) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < kPrKeys; c += 16) {
    float s[16];
    tmem_ld16(ts + c, s);
    tmem_wait_ld();
    const float4 f = sc[c / 16];
    const float g = fmaxf(fac * f.x, 1e-38f);
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if ((unsigned)(c + k - from) < len) top = fmaxf(top, fmaf(s[k], g, f.w));
  }
  const bool grow = top - m > kPrGrow;   // (no: nothing seen, or both infinite)
  if (__any_sync(0xffffffffu, grow)) {
    float next = top - kPrLead;
    if (top - next > kPrGrow) next = top;   // a step of t is as wide
    const float half = grow ? attn_half_factor(m, next) : 1.f, down = half * half;
    if (grow) m = next;
    l = l * half * half;
    if (ofull) {
      pr_wait(ofull, parity, sh);
      __syncwarp();
      tc_fence_after();
      pr_scale_sums<D>(to, down);
    }
  }
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 1
  for (int c = 0; c < kPrKeys; c += 16) {
    float s[16];
    uint32_t p[8];
    __syncwarp();
    tmem_ld16(ts + c, s);
    tmem_wait_ld();
    const float4 f = sc[c / 16];
    const float g = fmaxf(fac * f.x, 1e-38f);
    const int more = max(kKvExpLow - max((int)f.w, kKvExpMin), 0);
    const float by = pow2f(-more);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
#pragma unroll
      for (int e = k; e < k + 2; ++e) {
        s[e] = (unsigned)(c + e - from) < len ? exp2_approx(fmaf(s[e], g, f.w) - ref + more) : 0.f;
        sum += s[e];
      }
      p[k / 2] = pack_f16x2(s[k] * by, s[k + 1] * by);
    }
    l = fmaf(f.z, sum, l);
    tmem_st8(ts + c / 2, p);
  }
  return make_float2(m, l);
}

template <int D, bool PAIR>
__device__ __forceinline__ void pr_softmax(const AttnArgs& a, PrShared& sh, uint8_t* smem,
                                           PrCursor c, long long n_units) {
  using S = PrShape<D, PAIR>;
  const int t = threadIdx.x >> 7, row = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const uint32_t base = smem_addr(smem);
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;   // (tensor memory begins at 0)
  const uint32_t ts = lanes + 128 * t, to = lanes + S::OCOL + D * t;
  float* slots = a.partial + 2ll * blockIdx.x * S::SLOT;
  uint32_t cnt = 0;     // tiles of this stream so far
  int n0 = 0, seg = 0;
  long long done = 0;
  if (PAIR && t == 1 && warp == 0) pr_pass_turn(1);   // the first turn is stream 0's
#pragma unroll 1
  while (done < n_units) {
    const int nseg = (int)min((long long)(c.S - c.s), n_units - done);
    int lo_all, hi_all, lo, hi;
    pr_seen<S::TILE>(a, c, lo_all, hi_all);
    // ---- this row's query as f16 times 2^-shift (the stream's own half, or
    // the first stream's threads for both) ----
    const unsigned rho = (unsigned)c.m * S::TILE + (PAIR ? 128 * t : 0) + row;
    const int i = (int)(rho / (unsigned)a.group);
    const int head = c.h * a.group + (int)(rho - (unsigned)i * (unsigned)a.group);
    const bool real = i < c.w.n;
    attn_seen(a, c.w, min(i, c.w.n - 1), lo, hi);
    if (!PAIR) pr_streams_sync();   // both streams are through with the last item's queries
    // A query of infinities or NaN is NaN where it sees a key, and 0 where it sees
    // only blocks outside the cache, whose scores it would make NaN too: it goes
    // in as zeros, and the sum of what it saw becomes NaN at the end.
    bool poison;
    float fac = 0.f;
    {
      const uint16_t* q = a.q + (long long)(c.w.tok + (real ? i : 0)) * a.q_ts + head * a.q_hs;
      uint8_t* dst = smem + (PAIR ? t * S::QBYTES : 0) + row * 16;
      float mx = 0.f;
      bool finite = true;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (real) w = *reinterpret_cast<const uint4*>(q + 8 * k);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack16(u[e], a.f16);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
          finite = finite && fabsf(f.x) < INFINITY && fabsf(f.y) < INFINITY;
        }
      }
      const int be = (int)(__float_as_uint(mx) >> 23);
      const int shift = be == 0 || be == 255 ? 0 : min(max(be - 140, -120), 120);
      const float down =
          a.scale_log2 == 0.f ? 0.f : (a.scale_log2 < 0.f ? -pow2f(-shift) : pow2f(-shift));
      fac = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2) * pow2f(shift);
      poison = !finite;
      if (PAIR || t == 0) {
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (real && finite) w = *reinterpret_cast<const uint4*>(q + 8 * k);
          const float2 f0 = unpack16(w.x, a.f16), f1 = unpack16(w.y, a.f16),
                       f2 = unpack16(w.z, a.f16), f3 = unpack16(w.w, a.f16);
          *reinterpret_cast<uint4*>(dst + k * S::QGROUP) = make_uint4(
              pack_f16x2(f0.x * down, f0.y * down), pack_f16x2(f1.x * down, f1.y * down),
              pack_f16x2(f2.x * down, f2.y * down), pack_f16x2(f3.x * down, f3.y * down));
        }
        fence_async_shared();
      }
    }
    // the queries are in place (and O of the last item read): the first scores
    tc_fence_before();
    if (PAIR) pr_stream_sync(t);
    else pr_streams_sync();
    if (warp == 0 && (PAIR || t < nseg)) {
      pr_wait_keys(sh, n0 + (PAIR ? 0 : t));
      __syncwarp();
      tc_fence_after();
      pr_scores<D, PAIR>(sh, base, t, n0 + (PAIR ? 0 : t));
    }

    float m = -INFINITY, l = 0.f;
    int mine = 0;       // tiles of this stream in the segment
#pragma unroll 1
    for (int j = PAIR ? 0 : t; j < nseg; j += PAIR ? 1 : 2, ++mine, ++cnt) {
      const int p0 = (c.s0 + c.s + j) << 7;
      const float4* sc = sh.scale[(n0 + j) & 3];
      const bool masked = pr_masked(p0, lo_all, hi_all);
      pr_wait(&sh.sfull[t], cnt & 1, sh);
      __syncwarp();
      tc_fence_after();
      // Weights against the running reference in one pass over the scores, in
      // registers until the tile's maximum is known; where a row of the warp
      // outgrows its reference (its first tile, then rarely) O and the sums
      // follow, and the pass is made again: once, as the new reference is within
      // 1 of its place below kAttnLarge.
      uint32_t p[kPrKeys / 2];
#pragma unroll 1
      for (;;) {
        const float ref = m == -INFINITY ? 0.f : m;
        float x = -INFINITY, lt = 0.f;
        __syncwarp();
        float sb[2][32];   // scores, the next 32 on their way
        tmem_ld32(ts, sb[0]);
#pragma unroll
        for (int c32 = 0; c32 < kPrKeys; c32 += 32) {
          float* s = sb[(c32 / 32) & 1];
          tmem_wait_ld();
          if (c32 + 32 < kPrKeys) tmem_ld32(ts + c32 + 32, sb[(c32 / 32 + 1) & 1]);
          if (masked) {
            const int from = lo - p0 - c32;
            const unsigned len = (unsigned)max(hi - lo, 0);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if ((unsigned)(k - from) >= len) s[k] = -INFINITY;
          }
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float4 f = sc[c32 / 16 + b];
            // (a factor of 0 would make NaN of a masked score)
            const float g = fmaxf(fac * f.x, 1e-38f), off = f.y - ref;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int k = 16 * b; k < 16 * b + 16; k += 2) {
              fma_f32x2(s[k], s[k + 1], g, off);
              x = fmaxf(fmaxf(x, s[k]), s[k + 1]);
              s[k] = exp2_approx(s[k]);
              s[k + 1] = exp2_approx(s[k + 1]);
              add_f32x2(s0, s1, s[k], s[k + 1]);
              p[(c32 + k) / 2] = pack_f16x2(s[k], s[k + 1]);
            }
            lt = fmaf(f.z, s0 + s1, lt);
          }
        }
        // (nothing seen yet, or a reference that t - M is not to be rounded against)
        const bool any = !(fabsf(m) < kAttnLarge);
        const bool grow = x > (any ? -INFINITY : kPrGrow);
        if (!__any_sync(0xffffffffu, grow)) {
          // into the columns of the scores
          l += lt;
          __syncwarp();
          tmem_st32(ts, p);
          tmem_st32(ts + 32, p + 32);
          break;
        }
        const float next = ref + x - kPrLead;
        if (__any_sync(0xffffffffu, grow && (!(fabsf(next) < kAttnLarge) || (any && m != -INFINITY)))) {
          const float2 r = pr_weights_apart<D>(
              sh, sc, ts, to, masked ? lo - p0 : 0, masked ? (unsigned)max(hi - lo, 0) : kPrKeys,
              fac, m, l, mine > 0 ? &sh.ofull[t] : nullptr, (cnt - 1) & 1);
          m = r.x;
          l = r.y;
          break;
        }
        const float half = grow ? attn_half_factor(m, next) : 1.f, down = half * half;
        if (grow) m = next;
        l = l * half * half;
        if (mine > 0) {
          pr_wait(&sh.ofull[t], (cnt - 1) & 1, sh);
          __syncwarp();
          tc_fence_after();
          pr_scale_sums<D>(to, down);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      pr_stream_sync(t);
      if (warp == 0) {
        constexpr int step = PAIR ? 1 : 2;
        const bool more = j + step < nseg;
        pr_wait_values(sh, n0 + j);
        if (more) pr_wait_keys(sh, n0 + j + step);
        __syncwarp();
        if (PAIR) pr_take_turn(t);
        tc_fence_after();
        pr_values<D, PAIR>(sh, base, t, n0 + j, mine > 0);
        if (more) pr_scores<D, PAIR>(sh, base, t, n0 + j + step);
        if (PAIR) pr_pass_turn(t);
      }
    }

    // ---- the item's end, or the CTA's ----
    if (mine > 0) pr_wait(&sh.ofull[t], (cnt - 1) & 1, sh);
    unsigned bits[4] = {0, 0, 0, 0};
    if (*(volatile int*)&sh.nan[seg & 7])
      pr_nan_dims<D>(a, c, c.s + (PAIR ? 0 : t), c.s + nseg, PAIR ? 1 : 2, lo, hi, lo_all, hi_all,
                     bits);
    const bool begins = c.s == 0, ends = c.s + nseg == c.S;
    float f0 = 1.f, f1 = 0.f;   // factors of this stream's sums and of the other's
    if (!PAIR) {
      // the first stream's threads join both: the second's O lies in the same
      // lanes of tensor memory
      tc_fence_before();
      if (t == 1) {
        sh.m1[row] = m;
        sh.l1[row] = l;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) sh.nan1[k][row] = bits[k];
      }
      pr_streams_sync();
      if (t == 0) {
        const float m1 = sh.m1[row], mx = fmaxf(m, m1);
        const float h0 = attn_half_factor(m, mx), h1 = nseg > 1 ? attn_half_factor(m1, mx) : 0.f;
        f0 = h0 * h0;
        f1 = h1 * h1;
        l = l * h0 * h0 + (nseg > 1 ? sh.l1[row] * h1 * h1 : 0.f);
        m = mx;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) bits[k] |= sh.nan1[k][row];
      }
    }
    __syncwarp();
    tc_fence_after();
    if (*(volatile int*)&sh.dead || (poison && l > 0.f)) l = __int_as_float(0x7FFFFFFF);
    if (PAIR || t == 0) {
      const float inv = attn_inverse(l);
      const long long tok = c.w.tok + i;
      float* slot = slots + (begins ? S::SLOT : 0);
      const int srow = (PAIR ? 128 * t : 0) + row;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        float o[16];
        __syncwarp();
        tmem_ld16(to + 16 * k, o);
        if (!PAIR && nseg > 1) {
          float o1[16];
          tmem_ld16(to + D + 16 * k, o1);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = fmaf(o1[e], f1, o[e] * f0);
        } else {
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if ((bits[k >> 1] >> (16 * (k & 1) + e)) & 1u) o[e] = __int_as_float(0x7FFFFFFF);
        if (real && begins && ends) {
          uint16_t* dst = a.out + tok * a.o_ts + head * a.o_hs + 16 * k;
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            *reinterpret_cast<uint4*>(dst + e) =
                make_uint4(pack16(o[e] * inv, o[e + 1] * inv, a.f16),
                           pack16(o[e + 2] * inv, o[e + 3] * inv, a.f16),
                           pack16(o[e + 4] * inv, o[e + 5] * inv, a.f16),
                           pack16(o[e + 6] * inv, o[e + 7] * inv, a.f16));
        } else if (real) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(slot + (long long)srow * D + 16 * k + e) =
                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      if (real) {
        if (begins && ends) {
          if (a.lse) a.lse[tok * a.heads + head] = attn_lse(m, l);
        } else {
          slot[S::TILE * D + srow] = m;
          slot[S::TILE * D + S::TILE + srow] = l;
        }
      }
    if (!(begins && ends) && threadIdx.x == 0) {
        sh.open[begins] = 1;
        sh.piece[begins] = {1 | (begins ? 2 : 0) | (ends ? 4 : 0), c.h, c.m, c.w.tok, c.w.n, c.S,
                            done - c.s};
      }
    }
    if (threadIdx.x == 0) sh.nan[(seg + 4) & 7] = 0;
    tc_fence_before();
    done += nseg;
    n0 += nseg;
    ++seg;
    if (done < n_units) pr_next_item<S::TILE>(a, c);
  }
}

template <int D, bool PAIR>
static __global__ void __launch_bounds__(kPrThreads, 1) kv_attention_tc(const AttnArgs a) {
  using S = PrShape<D, PAIR>;
  extern __shared__ __align__(128) uint8_t pr_smem[];
  __shared__ PrShared sh;
  const int warp = threadIdx.x >> 5;
  DecShare share;
  PrCursor cur;
  pr_schedule<S::TILE>(a, share, cur);
  const long long n_units = share.n;
  if (n_units <= 0) return;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.kfull[s], 128);
      mbar_init(&sh.kempty[s], PAIR ? 2 : 1);   // streams that read it
      mbar_init(&sh.vfull[s], 128);
      mbar_init(&sh.vempty[s], PAIR ? 2 : 1);
      mbar_init(&sh.sfull[s], 1);
      mbar_init(&sh.ofull[s], 1);
      mbar_init(&sh.drained[s], 1);
      sh.open[s] = 0;
    }
    for (int s = 0; s < 8; ++s) sh.nan[s] = 0;
    sh.dead = 0;
    sh.share = share;
    sh.out = {a.out, a.lse, a.o_ts, a.o_hs, a.heads, a.f16, (unsigned)a.group};
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(&sh.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (threadIdx.x == 0 && sh.tmem != 0) sh.dead = 1;   // never: all of it was allocated
  if (warp < 8) {
    pr_softmax<D, PAIR>(a, sh, pr_smem, cur, n_units);
    if (*(volatile int*)&sh.dead && (warp & 3) == 0) pr_drain(sh, warp >> 2);
  } else {
    pr_convert<D, PAIR>(a, sh, pr_smem, cur, n_units);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(sh.tmem);
  }

  // ---- items that the CTA's ends cut ----
  dec_join_ctas<D, S::TILE, kPrWarps, 2 * S::SLOT, S::SLOT, true>(
      a, a.partial, sh.share, sh.open[0] ? &sh.piece[0] : nullptr,
      sh.open[1] ? &sh.piece[1] : nullptr, &sh.out, sh.job);
}

}  // namespace moe
