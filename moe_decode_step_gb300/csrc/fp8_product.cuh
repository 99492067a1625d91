// Products of 8-bit activations with 8-bit or MXFP4 weights, dense or by expert.
//
// tcgen05 block-scaled MMAs (kind::mxf8f6f4): both operands enter as stored,
// E4M3 rows of 128 columns brought by TMA into 128-byte-swizzled tiles, E2M1
// weights unpacked on the way in (8 bytes of nibbles in every 16), and their
// E8M0 scales in tensor memory, so no product is scaled or converted by a
// thread.
//
// The weights are the M side and the rows of x ("tokens") the N side: a tile is
// 256 weight rows of a pair of CTAs (cta_group::2, 128 rows each) times up to 240
// tokens, so that an expert's tokens cost what they are, in steps of 16, and a
// pair's stage of K = 128 takes 64 KB of shared-memory writes for 2 x 256 x 240 x
// 128 operations, half of what a CTA alone would need.  240 tokens: two
// accumulators (480 columns) and the scales of two steps fit tensor memory, and
// one accumulator is stored while the next one is summed.
//
// Roles (8 warps a CTA): 0 copies tiles (rows of x by index through gather4, four
// a copy), 1 issues the MMAs (of the pair's first CTA), 2 and 3 lay the scales of
// the weights and the tokens out, 4..7 the results, a thread a weight row.  Pairs
// take tiles in the order (expert, 16 token tiles, weight rows, token tile): pairs
// next to one another read the same weights.  Calls with fewer tiles than pairs
// split K over `splits` pairs of a cluster, which add up through distributed
// shared memory, always in the same order.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "cluster.cuh"
#include "common.cuh"
#include "fp8_rows.cuh"
#include "tcgen05.cuh"

namespace moe {

constexpr int kGemmThreads = 256;
constexpr int kGemmK = 128;
constexpr int kGemmRows = 128;      // weight rows of a CTA's part of a tile
constexpr int kGemmTokens = 240;    // tokens of a tile at most
constexpr int kGemmMaxExperts = 1024;
constexpr int kGemmGroup = 16;      // token tiles that share a pass over the weights
constexpr int kGemmMaxStages = 12;
constexpr int kGemmMaxSplits = 4;   // pairs of a cluster (8 CTAs)

struct GemmShape {
  static constexpr int ABYTES = kGemmRows * kGemmK;
  static constexpr int SFA = 512, SFB = 1024;   // scales of a stage
  static constexpr int SFCOL = 480;             // tensor memory: accumulators at 0 and 240, scales
  // the ring of a call whose tiles have at most `tokens`: tiles, then scales
  __host__ __device__ static constexpr int stage(int tokens) {
    return ABYTES + tokens / 2 * kGemmK;   // multiples of 1,024, the swizzle's pattern
  }
  static constexpr int LIMIT = 227 * 1024 - 12 * 1024;   // beside the static part
  static constexpr int stages(int tokens) {
    const int n = (LIMIT - 1024) / (stage(tokens) + SFA + SFB);
    return n < kGemmMaxStages ? n : kGemmMaxStages;
  }
  static constexpr int smem(int tokens) {
    return stages(tokens) * (stage(tokens) + SFA + SFB) + 1024;   // (1,024: alignment)
  }
};

struct GemmArgs {
  int kb;                    // blocks of 128 columns
  int n, wide;               // output columns; weight rows (n, or 2 n)
  int rows, x_rows, experts;
  int tokens;                // of a tile at most, a multiple of 16
  int stages, splits;
  const int* offsets;        // or null
  const int* src;            // or null
  const uint8_t* xs;
  long long xs_stride;
  const uint8_t* ws;
  long long ws_stride, ws_expert;
  char* out;
  long long out_stride;      // bytes
  uint8_t* os;
  long long os_stride;
  int out_dtype, vec;        // vec: rows of out are 4-byte aligned
};

struct GemmShared {
  uint64_t full[kGemmMaxStages], empty[kGemmMaxStages];
  uint64_t acc_full[2], acc_empty[2], amax_full, drained;
  uint32_t tmem;
  int dead;                           // a wait ran out
  int tiles[kGemmMaxExperts + 1];     // token tiles before each expert
  int warp_sum[kGemmThreads / 32];
  unsigned amax[3][256];              // of a token's 128 results, by tile
};

// ---- barriers between the CTAs of a pair ----
__device__ __forceinline__ bool gemm_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, "
      "%3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
// Waits for a phase, two seconds at most; then the CTA is dead: its waits all
// end at once and its results become NaN.
__device__ __forceinline__ bool gemm_dead(GemmShared& sh) { return *(volatile int*)&sh.dead != 0; }
__device__ __forceinline__ void gemm_wait(uint64_t* bar, uint32_t parity, GemmShared& sh) {
  if (gemm_try_wait(bar, parity)) return;
  const unsigned long long t0 = global_ns();
  while (!gemm_try_wait(bar, parity)) {
    if (gemm_dead(sh)) return;
    if (global_ns() - t0 > kWaitLimitNs) {
      *(volatile int*)&sh.dead = 1;
      return;
    }
  }
}
// `addr`: from cluster_map.
__device__ __forceinline__ void gemm_arrive(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}

// ---- TMA; `bar` may be the other CTA's of the pair ----
__device__ __forceinline__ void tma_tile_2d(uint32_t dst, const CUtensorMap* map, int c, int r,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_tile_3d(uint32_t dst, const CUtensorMap* map, int c, int r,
                                            int e, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r), "r"(e), "r"(bar)
      : "memory");
}
// Four rows of a map whose box is one row.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int c,
                                            const int (&r)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
      : "memory");
}

// ---- MMAs of a pair: both CTAs' shared and tensor memory, at the same places ----
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst)),
               "n"(kTcCols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(kTcCols)
               : "memory");
}
// K-major operand with the 128-byte swizzle: rows of 128 bytes, groups of 8 rows.
__device__ __forceinline__ uint64_t umma_desc_sw128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor, kind::mxf8f6f4: A E4M3 (0) or E2M1 (5), B E4M3, E8M0
// scales, both K-major, M = 256; a_sf, b_sf: the scales' byte of the step.
__device__ __forceinline__ uint32_t umma_idesc_mxf8(uint32_t a_format, uint32_t a_sf,
                                                    uint32_t b_sf, uint32_t N) {
  return (b_sf << 4) | (a_format << 7) | ((N >> 3) << 17) | (1u << 23) | (16u << 24) |
         (a_sf << 29);
}
__device__ __forceinline__ void umma_mxf8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_sf_copy_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
// Arrive on `bar` of the CTAs in `mask` when all this thread issued has completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"(mask)
      : "memory");
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
struct GemmTile {
  int expert, row0, rows;   // first output row, rows of the tile
  int N;                    // rows, rounded up to 16
  int n0;                   // first output column
};

__device__ __forceinline__ int gemm_start(const GemmArgs& a, int e) {
  if (!a.offsets) return e ? a.rows : 0;
  return min(max(__ldg(a.offsets + e), 0), a.rows);
}

// Token tiles before each expert; every thread calls.
__device__ __forceinline__ void gemm_prefix(const GemmArgs& a, GemmShared& sh) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  constexpr int PER = kGemmMaxExperts / kGemmThreads;
  int v[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * PER + i;
    v[i] = 0;
    if (e < a.experts) {
      const int s = gemm_start(a, e);
      v[i] = (max(gemm_start(a, e + 1) - s, 0) + a.tokens - 1) / a.tokens;
    }
    sum += v[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) sh.warp_sum[warp] = inc;
  __syncthreads();
  int before = inc - sum;
  for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * PER + i;
    if (e < a.experts) sh.tiles[e] = before;
    before += v[i];
    if (e == a.experts - 1) sh.tiles[a.experts] = before;
  }
  __syncthreads();
}

template <bool SWIGLU>
__device__ __forceinline__ GemmTile gemm_tile(const GemmArgs& a, const GemmShared& sh, int nt,
                                              long long t) {
  int lo = 0, hi = a.experts;   // tiles[lo] * nt <= t < tiles[hi] * nt
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((long long)sh.tiles[mid] * nt <= t) lo = mid;
    else hi = mid;
  }
  // (experts without rows: lo is the last with this many tiles before it)
  const int mt = sh.tiles[lo + 1] - sh.tiles[lo];
  const long long l = t - (long long)sh.tiles[lo] * nt;
  const int g = (int)(l / ((long long)kGemmGroup * nt));
  const int gm = min(kGemmGroup, mt - g * kGemmGroup);
  const int in = (int)(l - (long long)g * kGemmGroup * nt);
  const int m = g * kGemmGroup + in % gm;
  const int s = gemm_start(a, lo), end = max(gemm_start(a, lo + 1), s);
  // an expert's tokens in equal parts, none of them empty: (mt - 1) * size <=
  // (mt - 1) * a.tokens < end - s
  const int size = ((end - s + mt - 1) / mt + 15) & ~15;
  GemmTile r;
  r.expert = lo;
  r.row0 = s + m * size;
  r.rows = min(size, end - r.row0);
  r.N = (r.rows + 15) & ~15;
  r.n0 = in / gm * (SWIGLU ? kGemmRows : 2 * kGemmRows);
  return r;
}

// The row of x behind token r of the tile (tokens past the tile: its last).
__device__ __forceinline__ int gemm_source(const GemmArgs& a, const GemmTile& w, int r) {
  const int i = w.row0 + min(r, w.rows - 1);
  const int s = a.src ? __ldg(a.src + i) : i;
  return min(max(s, 0), a.x_rows - 1);
}

// Walks a pair's tiles and each one's blocks of K: all of them, or (splits) this
// pair's part, whole groups of four.
template <bool SWIGLU>
struct GemmWalk {
  long long t, tiles, step;
  int nt, k0, k1;

  __device__ __forceinline__ GemmWalk(const GemmArgs& a, const GemmShared& sh) {
    constexpr int COLS = SWIGLU ? kGemmRows : 2 * kGemmRows;
    nt = (a.n + COLS - 1) / COLS;
    tiles = (long long)sh.tiles[a.experts] * nt;
    const int pair = blockIdx.x / 2, split = pair % a.splits;
    t = pair / a.splits;
    step = gridDim.x / 2 / a.splits;
    const int groups = (a.kb + 3) / 4;
    k0 = 4 * (int)((long long)groups * split / a.splits);
    k1 = min(a.kb, 4 * (int)((long long)groups * (split + 1) / a.splits));
  }
};

struct GemmRing {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next(const GemmArgs& a) {
    if (++stage == (uint32_t)a.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// ---------------------------------------------------------------------------
// Copies (warp 0)
// ---------------------------------------------------------------------------
template <bool W4, bool SWIGLU>
__device__ __forceinline__ void gemm_copy(const GemmArgs& a, GemmShared& sh, uint32_t base,
                                          const CUtensorMap* xt, const CUtensorMap* xg,
                                          const CUtensorMap* wm, uint32_t rank) {
  using S = GemmShape;
  const int lane = threadIdx.x & 31, half = rank & 1;
  const uint32_t stage_bytes = S::stage(a.tokens);
  GemmRing ring;
  uint32_t issued = 0;
  for (GemmWalk<SWIGLU> k(a, sh); k.t < k.tiles; k.t += k.step) {
    const GemmTile w = gemm_tile<SWIGLU>(a, sh, k.nt, k.t);
    // whole tiles of consecutive rows in one copy, others four rows a copy
    const bool gather = a.src || w.N != a.tokens;
    const bool mine = gather && 4 * lane < w.N / 2;
    int r[4];
    if (mine) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = gemm_source(a, w, half * (w.N / 2) + 4 * lane + i);
    }
    // the pair's bytes (nibbles count as the bytes they are read as)
    const uint32_t bytes = (W4 ? S::ABYTES : 2 * S::ABYTES) + w.N * kGemmK;
    for (int kb = k.k0; kb < k.k1; ++kb, ring.next(a), ++issued) {
      gemm_wait(&sh.empty[ring.stage], ring.phase ^ 1, sh);
      if (gemm_dead(sh)) return;
      const uint32_t bar = cluster_map(smem_addr(&sh.full[ring.stage]), rank & ~1u);
      const uint32_t at = base + ring.stage * stage_bytes;
      if (half == 0 && lane == 0) mbar_arrive_expect_tx(&sh.full[ring.stage], bytes);
      __syncwarp();
      if (SWIGLU) {
        // 16 gate rows and 16 up rows in turn: a warp's lanes
        if (lane < 8)
          tma_tile_3d(at + lane * 16 * kGemmK, wm, kb * kGemmK,
                      (lane & 1 ? a.n : 0) + w.n0 + half * 64 + (lane >> 1) * 16, w.expert, bar);
      } else if (lane == 0) {
        tma_tile_3d(at, wm, kb * kGemmK, w.n0 + half * kGemmRows, w.expert, bar);
      }
      if (!gather) {
        if (lane == 8)
          tma_tile_2d(at + S::ABYTES, xt, kb * kGemmK, w.row0 + half * (w.N / 2), bar);
      } else if (mine) {
        tma_gather4(at + S::ABYTES + lane * 4 * kGemmK, xg, kb * kGemmK, r, bar);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Scales (warps 2, 3): for 128 rows at a time, 16 bytes a lane: one word for each
// of the rows lane, lane + 32, lane + 64, lane + 96.  A word holds four bytes:
// of MXFP4 weights those of a stage's four steps, of others those of four stages,
// laid out with the first.  Read four stages at a time, one such group ahead.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t scale_word(const uint8_t* p, int k, int kb) {
  if (k + 4 <= kb && ((uintptr_t)(p + k) & 3) == 0)
    return __ldg(reinterpret_cast<const uint32_t*>(p + k));
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (k + i < kb) v |= (uint32_t)__ldg(p + k + i) << (8 * i);
  return v;
}

// R rows a lane (4: weights, 8: tokens).  PERK: a word of its own for each block.
template <int R, bool PERK>
__device__ __forceinline__ void scales_load(const uint8_t* const (&p)[R], int k, int kb,
                                            uint32_t (&v)[R * (PERK ? 4 : 1)]) {
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (!p[i]) continue;
    if (!PERK) {
      v[i] = scale_word(p[i], k, kb);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k + j < kb) v[4 * i + j] = scale_word(p[i], 4 * (k + j), 4 * kb);
    }
  }
}

template <int R, bool PERK, bool SWIGLU, class Rows>
__device__ __forceinline__ void gemm_scales(const GemmArgs& a, GemmShared& sh, uint8_t* dst,
                                            uint32_t rank, Rows rows_of) {
  constexpr int W = R * (PERK ? 4 : 1);
  const int lane = threadIdx.x & 31;
  GemmRing ring;
  for (GemmWalk<SWIGLU> k(a, sh); k.t < k.tiles; k.t += k.step) {
    const uint8_t* p[R];
    rows_of(k, p);
    uint32_t cur[W] = {}, next[W] = {};
    scales_load<R, PERK>(p, k.k0, a.kb, next);
    for (int k0 = k.k0; k0 < k.k1; k0 += 4) {
#pragma unroll
      for (int i = 0; i < W; ++i) cur[i] = next[i];
      if (k0 + 4 < k.k1) scales_load<R, PERK>(p, k0 + 4, a.kb, next);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (k0 + j >= k.k1) break;
        gemm_wait(&sh.empty[ring.stage], ring.phase ^ 1, sh);
        if (gemm_dead(sh)) return;
        if (PERK || j == 0) {
          uint4* to = reinterpret_cast<uint4*>(
              dst + ring.stage * (GemmShape::SFA + GemmShape::SFB));
#pragma unroll
          for (int g = 0; g < R / 4; ++g) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = cur[(4 * g + i) * (PERK ? 4 : 1) + (PERK ? j : 0)];
            to[32 * g + lane] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          fence_async_shared();
        }
        __syncwarp();
        if (lane == 0) gemm_arrive(cluster_map(smem_addr(&sh.full[ring.stage]), rank & ~1u));
        ring.next(a);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// MMAs (warp 1 of the pair's first CTA, one lane)
// ---------------------------------------------------------------------------
template <bool W4, bool SWIGLU>
__device__ __forceinline__ void gemm_mma(const GemmArgs& a, GemmShared& sh, uint32_t base,
                                         uint32_t rank) {
  using S = GemmShape;
  const uint32_t stage_bytes = S::stage(a.tokens), sf = base + a.stages * stage_bytes;
  const uint16_t both = (uint16_t)(3u << (rank & ~1u));
  GemmRing ring;
  const uint32_t tm = sh.tmem;
  uint32_t n = 0;
  for (GemmWalk<SWIGLU> k(a, sh); k.t < k.tiles; k.t += k.step, ++n) {
    const GemmTile w = gemm_tile<SWIGLU>(a, sh, k.nt, k.t);
    const uint32_t acc = tm + (n & 1) * kGemmTokens;
    gemm_wait(&sh.acc_empty[n & 1], (n >> 1 & 1) ^ 1, sh);
    tc_fence_after();
    for (int kb = k.k0; kb < k.k1; ++kb, ring.next(a)) {
      gemm_wait(&sh.full[ring.stage], ring.phase, sh);
      if (gemm_dead(sh)) return;
      tc_fence_after();
      const uint32_t at = base + ring.stage * stage_bytes;
      const uint32_t sc = sf + ring.stage * (S::SFA + S::SFB);
      const uint32_t kq = kb & 3, j4 = kb >> 2 & 1;
      // scales of this step (MXFP4 weights) or these four in turn in two places
      const uint32_t sfa = tm + S::SFCOL + 4 * (W4 ? kb & 1 : j4), sfb = tm + S::SFCOL + 8 + 8 * j4;
      if (W4 || kq == 0) umma_sf_copy_pair(sfa, umma_desc(sc, 0, 128));
      if (kq == 0) {
        umma_sf_copy_pair(sfb, umma_desc(sc + S::SFA, 0, 128));
        if (w.N > 128) umma_sf_copy_pair(sfb + 4, umma_desc(sc + S::SFA + 512, 0, 128));
      }
      const uint64_t da = umma_desc_sw128(at), db = umma_desc_sw128(at + S::ABYTES);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        umma_mxf8_pair(acc, da + 2 * j, db + 2 * j,
                       umma_idesc_mxf8(W4 ? 5 : 0, W4 ? j : kq, kq, w.N), sfa, sfb,
                       (kb > k.k0) || j > 0);
      umma_commit_pair(&sh.empty[ring.stage], both);
    }
    umma_commit_pair(&sh.acc_full[n & 1], both);
  }
}

// ---------------------------------------------------------------------------
// Results (warps 4..7): a thread a weight row (an output column), tokens in turn
// ---------------------------------------------------------------------------
// 32 columns of tokens from c on: this CTA's sums, or those of all splits.
__device__ __forceinline__ void gemm_sums(const GemmArgs& a, uint32_t taddr, uint32_t part,
                                          uint32_t rank, int c, float (&v)[32]) {
  if (a.splits == 1) {
    tmem_ld32(taddr + c, v);
    tmem_wait_ld();
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const uint32_t p = cluster_map(part, 2 * s + (rank & 1)) + c * 512;
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = ld_cluster_f32(p + i * 512);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += x[i];
  }
}

// 32 tokens of this thread's output column to out.
__device__ __forceinline__ void gemm_store(const GemmArgs& a, const GemmTile& w, int c, int col,
                                           const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  if (a.out_dtype == MOE_DTYPE_F32) {
    if (col >= a.n) return;
    char* p = a.out + (long long)(w.row0 + c) * a.out_stride + (long long)col * 4;
#pragma unroll
    for (int i = 0; i < 32; ++i, p += a.out_stride)
      if (c + i < w.rows) *reinterpret_cast<float*>(p) = v[i];
    return;
  }
  const int f16 = a.out_dtype == MOE_DTYPE_F16;
  // two tokens at a time: even lanes take the first one's pair of columns, odd
  // lanes the second's
  const int odd = lane & 1, col2 = col - odd;
  char* p = a.out + (long long)(w.row0 + c + odd) * a.out_stride + (long long)col2 * 2;
#pragma unroll
  for (int i = 0; i < 32; i += 2, p += 2 * a.out_stride) {
    const float x = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
    const uint32_t u = odd ? pack16(x, v[i + 1], f16) : pack16(v[i], x, f16);
    if (c + i + odd >= w.rows) continue;
    if (a.vec && col2 + 1 < a.n) {
      *reinterpret_cast<uint32_t*>(p) = u;
    } else {
      if (col2 < a.n) *reinterpret_cast<uint16_t*>(p) = (uint16_t)u;
      if (col2 + 1 < a.n) *reinterpret_cast<uint16_t*>(p + 2) = (uint16_t)(u >> 16);
    }
  }
}

// silu(gate) * up of 32 tokens: lanes below 16 hold gates, the others the ups of
// the same columns; lane l gets the results of column l & 15, of the tokens 2 i (below
// 16) or 2 i + 1.
__device__ __forceinline__ void gemm_swiglu(const float (&v)[32], float* h) {
  const bool up = (threadIdx.x & 16) != 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float x = __shfl_xor_sync(0xffffffffu, up ? v[2 * i] : v[2 * i + 1], 16);
    const float g = up ? x : v[2 * i], u = up ? v[2 * i + 1] : x;
    h[i] = __fdividef(g, 1.f + __expf(-g)) * u;
  }
}

// Maxima of 16 values each over 16 lanes: lane l gets value l & 15's.
__device__ __forceinline__ float gemm_max16(float (&m)[16]) {
  const int lane = threadIdx.x;
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1) {
    const bool upper = (lane & w) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= w) continue;
      const float x = __shfl_xor_sync(0xffffffffu, upper ? m[i] : m[i + w], w);
      m[i] = fmaxf(upper ? m[i + w] : m[i], x);
    }
  }
  return m[0];
}

template <bool SWIGLU>
__device__ __forceinline__ void gemm_results(const GemmArgs& a, GemmShared& sh, uint8_t* smem,
                                             uint32_t rank) {
  const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3, half = rank & 1;
  const uint32_t tm = sh.tmem + ((uint32_t)(q * 32) << 16);
  const uint32_t part = smem_addr(smem) + (threadIdx.x & 127) * 4;
  const int split = (blockIdx.x / 2) % a.splits;
  const float nan = __int_as_float(0x7FFFFFFF);
  uint32_t n = 0;
  for (GemmWalk<SWIGLU> k(a, sh); k.t < k.tiles; k.t += k.step, ++n) {
    const GemmTile w = gemm_tile<SWIGLU>(a, sh, k.nt, k.t);
    if (!gemm_dead(sh)) gemm_wait(&sh.acc_full[n & 1], n >> 1 & 1, sh);
    tc_fence_after();
    const uint32_t acc = tm + (n & 1) * kGemmTokens;
    if (a.splits > 1) {
      // this pair's part of K to shared memory (the ring is idle: every copy was
      // waited for and every product is done), then the tokens are shared out
      for (int c = 0; c < w.N; c += 32) {
        float v[32];
        tmem_ld32(acc + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i < w.N)
            *reinterpret_cast<float*>(smem + (c + i) * 512 + (threadIdx.x & 127) * 4) = v[i];
      }
      cluster_sync();
    }
    const bool dead = gemm_dead(sh);
    auto mine = [&](int c) { return c < w.N && (a.splits == 1 || (c >> 5) % a.splits == split); };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) gemm_arrive(cluster_map(smem_addr(&sh.acc_empty[n & 1]), rank & ~1u));
    };
    if (!SWIGLU) {
      const int col = w.n0 + half * kGemmRows + q * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < w.N; c += 32) {
        if (!mine(c)) continue;
        float v[32];
        gemm_sums(a, acc, part, rank, c, v);
        if (dead) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = nan;
        }
        if (c + 32 >= w.N) release();
        gemm_store(a, w, c, col, v);
      }
    } else {
      const int col = w.n0 + half * 64 + q * 16 + (lane & 15), late = lane >> 4;
      if (a.out_dtype != MOE_DTYPE_E4M3) {
#pragma unroll 1
        for (int c = 0; c < w.N; c += 32) {
          if (!mine(c)) continue;
          float v[32], h[16];
          gemm_sums(a, acc, part, rank, c, v);
          if (c + 32 >= w.N) release();
          gemm_swiglu(v, h);
          const int f16 = a.out_dtype == MOE_DTYPE_F16;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = c + 2 * i + late;
            if (t >= w.rows || col >= a.n) continue;
            const float x = dead ? nan : h[i];
            char* p = a.out + (long long)(w.row0 + t) * a.out_stride;
            if (a.out_dtype == MOE_DTYPE_F32) reinterpret_cast<float*>(p)[col] = x;
            else reinterpret_cast<uint16_t*>(p)[col] = (uint16_t)pack16(x, 0.f, f16);
          }
        }
      } else {
        // a token's 128 results lie in both CTAs: each warp's maxima go to both.
        // A tile's buffer is cleared two tiles after its last reader.
        unsigned* clear = sh.amax[(n + 1) % 3] + q * 64;
        clear[lane] = clear[lane + 32] = 0;
        const uint32_t am = smem_addr(sh.amax[n % 3]);
        const uint32_t here = cluster_map(am, rank), there = cluster_map(am, rank ^ 1);
        float h[kGemmTokens / 2 + 8];
#pragma unroll
        for (int c = 0; c < kGemmTokens; c += 32) {
          if (!mine(c)) continue;
          float v[32], m[16];
          gemm_sums(a, acc, part, rank, c, v);
          gemm_swiglu(v, h + c / 2);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            m[i] = col < a.n ? fp8_finite_max(0.f, h[c / 2 + i]) : 0.f;
          const unsigned top = __float_as_uint(gemm_max16(m));
          const int t = c + 2 * (lane & 15) + late;
          max_cluster_u32(here + t * 4, top);
          max_cluster_u32(there + t * 4, top);
        }
        release();
        if (lane == 0) {
          const uint32_t bar = smem_addr(&sh.amax_full);
          gemm_arrive(cluster_map(bar, rank));
          gemm_arrive(cluster_map(bar, rank ^ 1));
        }
        if (!gemm_dead(sh)) gemm_wait(&sh.amax_full, n & 1, sh);
        const unsigned* amax = sh.amax[n % 3];
        const bool lost = gemm_dead(sh);
#pragma unroll
        for (int c = 0; c < kGemmTokens; c += 32) {
          if (!mine(c)) continue;
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            // four tokens' codes of this column, turned among four lanes into four
            // columns' codes of one token
            uint32_t u = 0;
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const int t = c + 2 * (i + j) + late;
              const float e0 = pow2f(-fp8_block_exp(__uint_as_float(amax[t])));
              const float e1 = pow2f(-fp8_block_exp(__uint_as_float(amax[t + 2])));
              u |= f32x2_to_e4m3x2(h[c / 2 + i + j] * e0, h[c / 2 + i + j + 1] * e1) << (8 * j);
            }
            if (lost) u = 0x7F7F7F7Fu;
            const uint32_t x = __shfl_xor_sync(0xffffffffu, u, 1);
            u = lane & 1 ? __byte_perm(u, x, 0x3715) : __byte_perm(u, x, 0x6240);
            const uint32_t y = __shfl_xor_sync(0xffffffffu, u, 2);
            u = lane & 2 ? __byte_perm(u, y, 0x3276) : __byte_perm(u, y, 0x5410);
            const int t = c + 2 * (i + (lane & 3)) + late, at = col & ~3;
            if (t >= w.rows) continue;
            char* p = a.out + (long long)(w.row0 + t) * a.out_stride + at;
            if (a.vec && at + 3 < a.n) {
              *reinterpret_cast<uint32_t*>(p) = u;
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (at + j < a.n) p[j] = (char)(u >> (8 * j));
            }
          }
        }
        if (half == 0) {
          for (int t = threadIdx.x & 127; t < w.rows; t += 128)
            if (mine(t & ~31))
              a.os[(long long)(w.row0 + t) * a.os_stride + (w.n0 >> 7)] =
                  (uint8_t)(fp8_block_exp(__uint_as_float(amax[t])) + 127);
        }
      }
    }
  }
}

template <bool W4, bool SWIGLU>
static __global__ void __launch_bounds__(kGemmThreads, 1)
    fp8_product_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap xt,
                       const __grid_constant__ CUtensorMap xg,
                       const __grid_constant__ CUtensorMap wm) {
  using S = GemmShape;
  extern __shared__ uint8_t gemm_raw[];
  __shared__ GemmShared sh;
  uint8_t* smem = gemm_raw + ((1024 - (smem_addr(gemm_raw) & 1023)) & 1023);
  const uint32_t base = smem_addr(smem), rank = cluster_rank();
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sh.full[s], 5);    // the copies' bytes, two warps' scales of both CTAs
      mbar_init(&sh.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.acc_full[s], 1);
      mbar_init(&sh.acc_empty[s], 8);   // four warps of both CTAs
    }
    mbar_init(&sh.amax_full, 8);
    mbar_init(&sh.drained, 1);
    sh.dead = 0;
    fence_barrier_init();
  }
  sh.amax[0][threadIdx.x] = 0;
  if (warp == 1) tmem_alloc_pair(&sh.tmem);
  gemm_prefix(a, sh);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();

  if (warp == 0) {
    gemm_copy<W4, SWIGLU>(a, sh, base, &xt, &xg, &wm, rank);
  } else if (warp == 1) {
    if ((rank & 1) == 0 && (threadIdx.x & 31) == 0) gemm_mma<W4, SWIGLU>(a, sh, base, rank);
  } else if (warp == 2) {
    gemm_scales<4, W4, SWIGLU>(
        a, sh, smem + a.stages * S::stage(a.tokens), rank,
        [&](const GemmWalk<SWIGLU>& k, const uint8_t* (&p)[4]) {
          const GemmTile w = gemm_tile<SWIGLU>(a, sh, k.nt, k.t);
          const int lane = threadIdx.x & 31, half = rank & 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            int r = w.n0 + half * kGemmRows + 32 * i + lane;
            if (SWIGLU) r = (lane & 16 ? a.n : 0) + w.n0 + half * 64 + 16 * i + (lane & 15);
            r = min(r, a.wide - 1);
            p[i] = a.ws + w.expert * a.ws_expert + (W4 ? r : r >> 7) * a.ws_stride;
          }
        });
  } else if (warp == 3) {
    gemm_scales<8, false, SWIGLU>(
        a, sh, smem + a.stages * S::stage(a.tokens) + S::SFA, rank,
        [&](const GemmWalk<SWIGLU>& k, const uint8_t* (&p)[8]) {
          const GemmTile w = gemm_tile<SWIGLU>(a, sh, k.nt, k.t);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = (threadIdx.x & 31) + 32 * i;
            p[i] = 32 * i < w.N ? a.xs + gemm_source(a, w, r) * a.xs_stride : nullptr;
          }
        });
  } else {
    gemm_results<SWIGLU>(a, sh, smem, rank);
  }
  __syncwarp();
  if (a.splits > 1 && warp < 4) {   // the results' warps' one, where the cluster has a tile
    const GemmWalk<SWIGLU> k(a, sh);
    if (k.t < k.tiles) cluster_sync();
  }
  if (gemm_dead(sh) && warp == 1) {
    // products and copies in flight, before their memory is given back: bounded too
    if ((threadIdx.x & 31) == 0) {
      if ((rank & 1) == 0) {
        umma_commit_pair(&sh.drained, (uint16_t)(1u << rank));
        for (int i = 0; i < 100 && !gemm_try_wait(&sh.drained, 0); ++i) {
        }
      }
      const unsigned long long t0 = global_ns();
      while (global_ns() - t0 < 2000000) {
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // (nor does a CTA leave while another may read its sums)
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(sh.tmem);
  }
}

}  // namespace moe
