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
// Work: strips of 16 tokens of (row of the batch, KV head, tile), ordered in
// that order; CTA i takes strips [i * per, (i + 1) * per), so that ragged
// lengths leave every SM the same bytes.  Inside a CTA the strips go round
// the warps, each with its own running maximum and sums, joined in shared
// memory at the end of a tile; a tile cut by a CTA boundary leaves partial
// sums in the workspace, which the second kernel joins in CTA order (results
// do not depend on timing).
//
// Loads: each thread copies (cp.async) exactly the 16-byte pieces that it
// feeds to its own MMAs, into a ring of its own in shared memory, so a strip
// needs no barrier at all; the ring only deepens the loads in flight (8 warps
// x 3 strips x 4 KB = 96 KB an SM; 1 us of latency at 6.7 TB/s needs 44 KB).
// The contraction order of either product is free, so the pieces need no
// shuffling: lane (g, t) = (lane / 4, lane % 4) holds, for the scores, 16
// consecutive dims (from 16 t, and from 64 + 16 t) of keys g and g + 8, and
// for the values CH = D / 8 consecutive dims (from CH g) of tokens 2t, 2t + 1,
// 2t + 8, 2t + 9, byte-transposed in registers.  Codes become f16 exactly
// (cvt.rn.f16x2.e4m3x2); queries enter as f16 scaled per row by a power of
// two, which keeps all of bf16's 8 bits.
//
// Scales: a strip lies in one block, so one exponent ek scales its scores and
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
  static constexpr int KP = D / 32;                // 16-byte key pieces a lane (2 keys)
  static constexpr int VP = 4 * CH / 16;           // the same for values (4 tokens)
  static constexpr int STAGES = D == 64 ? 8 : 4;
  static constexpr int STAGE = 32 * 16 * (KP + VP);   // bytes of one warp's strip
  static constexpr int RS = D + 8;                 // row stride of the join buffer (floats)
  static constexpr int SMEM = kDecWarps * (STAGES * STAGE + 16 * RS * 4 + STAGES * 4 + 16 * 8) +
                              16 * D * 2 + 16 * 4;
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
  x.s0 = lo >> 4;
  x.S = max(1, ((hi + 15) >> 4) - x.s0);   // a tile that sees nothing still writes its zeros
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

__device__ __forceinline__ void dec_advance(const AttnArgs& a, DecCursor& c, int n) {
  c.s += n;
  while (c.s >= c.x.S && c.r < a.rows) {
    c.s -= c.x.S;
    if (++c.m < c.x.M) continue;
    c.m = 0;
    if (++c.h < a.c.heads) continue;
    c.h = 0;
    do {
      if (++c.r >= a.rows) return;
      c.x = dec_row(a, c.r);
    } while (c.x.M == 0);
  }
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

// What one warp loads ahead: its next strip, with the block id already asked for.
struct DecLoader {
  DecCursor c;
  long long left;    // strips of the CTA from this one on
  int id;            // its block, -1: none
  int p0;            // its first token
  uint32_t sk, sv;   // scale bytes of the strip loaded before, on their way
  bool there;        // its block exists
  int stage, prev;   // ring slot of the next strip; of the one before (-1: none)
};

__device__ __forceinline__ void dec_lookup(const AttnArgs& a, DecLoader& l) {
  if (l.left <= 0) return;
  l.p0 = (l.c.x.s0 + l.c.s) << 4;
  l.id = l.p0 < l.c.x.w.seq
             ? __ldg(a.table + l.c.r * a.table_stride + (l.p0 >> a.c.bs_log2))
             : -1;
}

// Bytes of s_meta: the scale exponents of a stage's strip (+128 each), bit 16: its block exists.
template <int D>
__device__ __forceinline__ void dec_fetch(const AttnArgs& a, DecLoader& l, uint32_t ring,
                                          uint32_t* s_meta, int lane) {
  using Sh = DecShape<D>;
  if (l.prev >= 0) {   // the scales asked for one strip ago
    if (lane == 0)
      s_meta[l.prev] = (uint32_t)(kv_exp(l.sk) + 128) | (uint32_t)(kv_exp(l.sv) + 128) << 8 |
                       (l.there ? 1u << 16 : 0u);
    l.prev = -1;
  }
  if (l.left > 0) {
    const int g = lane >> 2, t = lane & 3;
    const bool there = l.id >= 0 && l.id < a.c.n_blocks;
    const long long id = there ? l.id : 0;
    const int off = l.p0 & ((1 << a.c.bs_log2) - 1), seq = l.c.x.w.seq;
    const long long at = id * a.c.bstride + l.c.h * a.c.hstride + off * a.c.tstride;
    const uint32_t dst = ring + l.stage * Sh::STAGE + lane * 16;
    const uint8_t* kp = a.c.k + at;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const int tok = g + 8 * i;
        const bool in = there && l.p0 + tok < seq;
        cp_async<16>(dst + (i * (D / 64) + c) * 512,
                     in ? kp + tok * a.c.tstride + c * 64 + t * 16 : kp, in);
      }
    const uint8_t* vp = a.c.v + at;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = 2 * t + (i & 1) + 8 * (i >> 1);
      const bool in = there && l.p0 + tok < seq;
      const uint8_t* src = in ? vp + tok * a.c.tstride + g * Sh::CH : vp;
      if constexpr (D == 128) cp_async<16>(dst + (Sh::KP + i) * 512, src, in);
      else cp_async<8>(dst + (Sh::KP + (i >> 1)) * 512 + (i & 1) * 8, src, in);
    }
    l.sk = __ldg(a.c.ks + id * a.c.sstride + l.c.h);
    l.sv = __ldg(a.c.vs + id * a.c.sstride + l.c.h);
    l.there = there;
    l.prev = l.stage;
    l.stage = l.stage + 1 == Sh::STAGES ? 0 : l.stage + 1;
    l.left -= kDecWarps;
    if (l.left > 0) dec_advance(a, l.c, kDecWarps);
    dec_lookup(a, l);
  }
  cp_async_commit();
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

template <int D>
static __global__ void __launch_bounds__(kDecThreads, 1) kv_attention_decode(const AttnArgs a) {
  using Sh = DecShape<D>;
  constexpr int CH = Sh::CH, KS = D / 16;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  float* s_join = reinterpret_cast<float*>(dec_smem + kDecWarps * Sh::STAGES * Sh::STAGE);
  float* s_ml = s_join + kDecWarps * 16 * Sh::RS;                       // [warp][2][16]
  uint32_t* s_metas = reinterpret_cast<uint32_t*>(s_ml + kDecWarps * 32);
  float* s_fac = reinterpret_cast<float*>(s_metas + kDecWarps * Sh::STAGES);   // [16]
  uint16_t* s_q = reinterpret_cast<uint16_t*>(s_fac + 16);              // [16][D]; the output too
  const uint32_t ring = smem_addr(dec_smem) + warp * Sh::STAGES * Sh::STAGE;
  const uint8_t* ringp = dec_smem + warp * Sh::STAGES * Sh::STAGE;
  uint32_t* s_meta = s_metas + warp * Sh::STAGES;

  pdl_launch_dependents();
  long long u0, n_units, per;
  DecCursor cur;
  dec_schedule(a, u0, n_units, per, cur);
  if (threadIdx.x == 0) a.desc[4 * blockIdx.x] = 0;
  if (n_units <= 0) return;

  DecLoader ld;
  ld.c = cur;
  ld.left = n_units - warp;
  ld.stage = 0;
  ld.prev = -1;
  ld.sk = ld.sv = 0;
  ld.there = false;
  if (ld.left > 0) dec_advance(a, ld.c, warp);
  dec_lookup(a, ld);
#pragma unroll 1
  for (int i = 0; i < Sh::STAGES - 1; ++i) dec_fetch<D>(a, ld, ring, s_meta, lane);

  int stage = 0;
  long long u = 0;              // strips done by the CTA, in its own order
  int next = warp;              // this warp's next strip, relative to the tile's first
  int part = 0;                 // tiles begun
  while (u < n_units) {
    const int nseg = (int)min((long long)(cur.x.S - cur.s), n_units - u);
    // ---- queries of the tile: f16 times 2^-shift, in shared memory ----
    for (int j = warp; j < 16; j += kDecWarps) {
      int i, head;
      const bool real = dec_tile_row(a, cur, j, i, head);
      float v[D / 32];
      float mx = 0.f;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) v[k] = 0.f;
      if (real) {
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
      const float down = pow2f(-sh);
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
        *reinterpret_cast<uint32_t*>(s_q + j * D + 2 * lane + 64 * k) =
            pack_f16x2(v[2 * k] * down, v[2 * k + 1] * down);
      if (lane == 0) s_fac[j] = real ? a.scale_log2 * pow2f(sh) : 0.f;
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
    // what the lane's two rows see, and what every row of the tile sees
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

    for (; next < nseg; next += kDecWarps) {
      dec_fetch<D>(a, ld, ring, s_meta, lane);
      cp_async_wait<Sh::STAGES - 1>();
      __syncwarp();
      const uint32_t meta = s_meta[stage];
      const uint8_t* sp = ringp + stage * Sh::STAGE + lane * 16;
      const int p0 = (cur.x.s0 + cur.s + next) << 4;
      stage = stage + 1 == Sh::STAGES ? 0 : stage + 1;
      if (!(meta >> 16) || p0 >= hi_any || p0 + 16 <= lo_any) continue;   // nothing to see
      const int ev = (int)((meta >> 8) & 0xFFu) - 128;
      const float ke = pow2f((int)(meta & 0xFFu) - 128);
      // ---- scores ----
      float s[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(sp + (i * (D / 64) + c) * 512);
          const uint32_t u4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t* q = qf[4 * c + k];
            mma_f16_16816(s[i], q[0], q[1], q[2], q[3], e4m3x2_to_f16x2(u4[k] & 0xFFFFu),
                          e4m3x2_to_f16x2(u4[k] >> 16));
          }
        }
      }
      // ---- weights ----
      const float f0 = fac0 * ke, f1 = fac1 * ke, evf = (float)ev;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[i][0] = fmaf(s[i][0], f0, evf);
        s[i][1] = fmaf(s[i][1], f0, evf);
        s[i][2] = fmaf(s[i][2], f1, evf);
        s[i][3] = fmaf(s[i][3], f1, evf);
      }
      const bool masked = p0 + 16 > hi_all || p0 < lo_all;
      if (masked) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int j = p0 + 8 * i + 2 * t + c;
            if (j < lo0 || j >= hi0) s[i][c] = -INFINITY;
            if (j < lo1 || j >= hi1) s[i][2 + c] = -INFINITY;
          }
      }
      float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
      if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float d0 = n0 == -INFINITY ? 1.f : exp2_approx(m0 - n0);
        const float d1 = n1 == -INFINITY ? 1.f : exp2_approx(m1 - n1);
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
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[i][0] = exp2_approx(s[i][0] - r0);
        s[i][1] = exp2_approx(s[i][1] - r0);
        s[i][2] = exp2_approx(s[i][2] - r1);
        s[i][3] = exp2_approx(s[i][3] - r1);
      }
      const float un = pow2f(-ev);
      l0 = fmaf(un, (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]), l0);
      l1 = fmaf(un, (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]), l1);
      const uint32_t pa0 = pack_f16x2(s[0][0], s[0][1]), pa1 = pack_f16x2(s[0][2], s[0][3]);
      const uint32_t pa2 = pack_f16x2(s[1][0], s[1][1]), pa3 = pack_f16x2(s[1][2], s[1][3]);
      // ---- values ----
      uint32_t vw[4][CH / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(sp + (Sh::KP + i) * 512);
          vw[i][0] = w.x;
          vw[i][1] = w.y;
          vw[i][2] = w.z;
          vw[i][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(sp + (Sh::KP + (i >> 1)) * 512 + (i & 1) * 8);
          vw[i][0] = w.x;
          vw[i][1] = w.y;
        }
      }
      uint32_t nan = 0;
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
        const uint32_t a0 = __byte_perm(vw[0][c], vw[1][c], 0x5140);
        const uint32_t a1 = __byte_perm(vw[0][c], vw[1][c], 0x7362);
        const uint32_t b0 = __byte_perm(vw[2][c], vw[3][c], 0x5140);
        const uint32_t b1 = __byte_perm(vw[2][c], vw[3][c], 0x7362);
        mma_f16_16816(o[4 * c], pa0, pa1, pa2, pa3, e4m3x2_to_f16x2(a0 & 0xFFFFu),
                      e4m3x2_to_f16x2(b0 & 0xFFFFu));
        mma_f16_16816(o[4 * c + 1], pa0, pa1, pa2, pa3, e4m3x2_to_f16x2(a0 >> 16),
                      e4m3x2_to_f16x2(b0 >> 16));
        mma_f16_16816(o[4 * c + 2], pa0, pa1, pa2, pa3, e4m3x2_to_f16x2(a1 & 0xFFFFu),
                      e4m3x2_to_f16x2(b1 & 0xFFFFu));
        mma_f16_16816(o[4 * c + 3], pa0, pa1, pa2, pa3, e4m3x2_to_f16x2(a1 >> 16),
                      e4m3x2_to_f16x2(b1 >> 16));
      }
      if (masked && __any_sync(0xffffffffu, nan != 0)) {
        // columns 2t, 2t + 1 of value tile j are dims CH (2t) + j, CH (2t + 1) + j:
        // lanes 8t + tt and 8t + 4 + tt hold them for token pair tt
        const float qnan = __int_as_float(0x7FFFFFFF);
        const uint8_t* base = ringp + (stage == 0 ? Sh::STAGES - 1 : stage - 1) * Sh::STAGE;
#pragma unroll 1
        for (int tok = 0; tok < 16; ++tok) {
          const int tt = (tok & 7) >> 1, i = (tok & 1) + 2 * (tok >> 3), j = p0 + tok;
          const bool see0 = j >= lo0 && j < hi0, see1 = j >= lo1 && j < hi1;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int src = 8 * t + 4 * c + tt;
            const uint8_t* p = D == 128 ? base + (Sh::KP + i) * 512 + src * 16
                                        : base + (Sh::KP + (i >> 1)) * 512 + src * 16 + (i & 1) * 8;
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

    // ---- join the warps' sums ----
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (t == 0) {
      s_ml[warp * 32 + g] = m0;
      s_ml[warp * 32 + g + 8] = m1;
      s_ml[warp * 32 + 16 + g] = l0;
      s_ml[warp * 32 + 24 + g] = l1;
    }
    __syncthreads();
    float n0 = -INFINITY, n1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      n0 = fmaxf(n0, s_ml[w * 32 + g]);
      n1 = fmaxf(n1, s_ml[w * 32 + g + 8]);
    }
    {
      const float d0 = m0 == -INFINITY ? (n0 == -INFINITY ? 1.f : 0.f) : exp2_approx(m0 - n0);
      const float d1 = m1 == -INFINITY ? (n1 == -INFINITY ? 1.f : 0.f) : exp2_approx(m1 - n1);
      float* dst = s_join + warp * 16 * Sh::RS;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        *reinterpret_cast<float2*>(dst + g * Sh::RS + j * 8 + 2 * t) =
            make_float2(o[j][0] * d0, o[j][1] * d0);
        *reinterpret_cast<float2*>(dst + (g + 8) * Sh::RS + j * 8 + 2 * t) =
            make_float2(o[j][2] * d1, o[j][3] * d1);
      }
    }
    __syncthreads();
    const bool whole = cur.s == 0 && nseg == cur.x.S;
    float* slot = a.partial + (2ll * blockIdx.x + (part > 0)) * kDecSlot<D>;
    for (int e = threadIdx.x; e < 16 * D / 4; e += kDecThreads) {
      const int row = e / (D / 4), col = (e % (D / 4)) * 4;   // join order: j * 8 + n
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, s_ml[w * 32 + row]);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float4 v =
            *reinterpret_cast<const float4*>(s_join + (w * 16 + row) * Sh::RS + col);
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
        const float mw = s_ml[w * 32 + row];
        l = fmaf(s_ml[w * 32 + 16 + row],
                 mw == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : exp2_approx(mw - m), l);
      }
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : l;   // nothing seen: 0; NaN stays NaN
        const int j = col >> 3, n = col & 7;
        uint16_t* so = s_q + row * D + j;
        so[n * CH] = (uint16_t)pack16(sum.x * inv, 0.f, a.f16);
        so[(n + 1) * CH] = (uint16_t)pack16(sum.y * inv, 0.f, a.f16);
        so[(n + 2) * CH] = (uint16_t)pack16(sum.z * inv, 0.f, a.f16);
        so[(n + 3) * CH] = (uint16_t)pack16(sum.w * inv, 0.f, a.f16);
        if (col == 0) s_fac[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      } else {
        *reinterpret_cast<float4*>(slot + row * D + col) = sum;
        if (col == 0) {
          slot[16 * D + row] = m;
          slot[16 * D + 16 + row] = l;
        }
      }
    }
    __syncthreads();
    if (whole) {
      for (int e = threadIdx.x; e < 16 * D / 8; e += kDecThreads) {
        const int row = e / (D / 8), d = (e % (D / 8)) * 8;
        int i, head;
        if (!dec_tile_row(a, cur, row, i, head)) continue;
        const long long tok = cur.x.w.tok + i;
        *reinterpret_cast<uint4*>(a.out + tok * a.o_ts + head * a.o_hs + d) =
            *reinterpret_cast<const uint4*>(s_q + row * D + d);
        if (d == 0 && a.lse) a.lse[tok * a.heads + head] = s_fac[row];
      }
      __syncthreads();   // the queries of the next tile go into s_q
    } else if (u + nseg == n_units && cur.s + nseg < cur.x.S &&
               threadIdx.x == 0 && (cur.s == 0)) {
      // this CTA begins a tile that later CTAs go on with
      const long long end = u0 + u + cur.x.S;   // the tile's end in strips of the call
      int* d = a.desc + 4 * blockIdx.x;
      d[1] = part > 0;
      d[2] = cur.r;
      d[3] = cur.h * cur.x.M + cur.m;
      d[0] = (int)((end - 1) / per) - (int)blockIdx.x + 1;
    }
    u += nseg;
    ++part;
    if (u < n_units) dec_advance(a, cur, nseg);
  }
  cp_async_wait<0>();
}

// Join of the tiles cut by CTA boundaries: block (i, j) takes rows 4j .. 4j+3
// of the tile that CTA i began, if any, and adds the partial sums of CTAs i,
// i + 1, ... in that order.
template <int D>
static __global__ void __launch_bounds__(D) kv_attention_join(const AttnArgs a) {
  pdl_wait_prerequisites();
  const int* d = a.desc + 4 * blockIdx.x;
  const int n = d[0];
  if (n == 0) return;
  DecCursor c;
  c.r = d[2];
  c.x = dec_row(a, c.r);
  c.h = d[3] / c.x.M;
  c.m = d[3] - c.h * c.x.M;
  const float* first = a.partial + (2ll * blockIdx.x + d[1]) * kDecSlot<D>;
  const float* rest = a.partial + 2ll * (blockIdx.x + 1) * kDecSlot<D>;
  constexpr int CH = D / 8;
  const int col = threadIdx.x, dim = (col & 7) * CH + (col >> 3);
  for (int row = 4 * blockIdx.y; row < 4 * blockIdx.y + 4; ++row) {
    int i, head;
    if (!dec_tile_row(a, c, row, i, head)) break;
    float m = first[16 * D + row];
    for (int k = 0; k < n - 1; ++k) m = fmaxf(m, rest[2ll * k * kDecSlot<D> + 16 * D + row]);
    float sum = 0.f, l = 0.f;
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float* p = k == 0 ? first : rest + 2ll * (k - 1) * kDecSlot<D>;
      const float mk = p[16 * D + row];
      const float f = mk == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : exp2_approx(mk - m);
      sum = fmaf(p[row * D + col], f, sum);
      l = fmaf(p[16 * D + 16 + row], f, l);
    }
    const long long tok = c.x.w.tok + i;
    a.out[tok * a.o_ts + head * a.o_hs + dim] =
        (uint16_t)pack16(sum * (l > 0.f ? 1.f / l : l), 0.f, a.f16);
    if (a.lse && threadIdx.x == 0)
      a.lse[tok * a.heads + head] =
          l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  }
}

}  // namespace moe
