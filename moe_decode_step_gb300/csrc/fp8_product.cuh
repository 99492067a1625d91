// Products of 8-bit activations with 8-bit or MXFP4 weights, dense or by expert.
//
// tcgen05 block-scaled MMAs (kind::mxf8f6f4): both operands enter as stored,
// E4M3 rows of 128 columns brought by TMA into 128-byte-swizzled tiles, E2M1
// weights unpacked on the way in (8 bytes of nibbles in every 16), and their
// E8M0 scales in tensor memory, so no product is scaled or converted by a
// thread.  Products are exact and summed in fp32; the tensor cores' additions cut
// rather than round (3e-7 of the results' rms at K = 4,096, where fp32 products are
// 1e-7 off).
//
// The weights are the M side and the rows of x ("tokens") the N side: a tile is
// 256 weight rows of a pair of CTAs (cta_group::2, 128 rows each) times up to 240
// tokens, so that an expert's tokens cost what they are, in steps of 16, and a
// pair's stage of K = 128 takes 64 KB of shared-memory writes for 2 x 256 x 240 x
// 128 operations, half of what a CTA alone would need.  240 tokens: two
// accumulators (480 columns) and the scales of two steps fit tensor memory, and
// one accumulator is stored while the next one is summed.
//
// Roles (16 warps a CTA): 0 copies tiles, 1 issues the MMAs (of the pair's first
// CTA), 2 and 3 lay the scales of the weights and the tokens out, 4..11 the results,
// a thread a weight row, in two groups that take tokens in turn, 12..15 bring rows of
// x by index.  Pairs take tiles in the order (expert, 16 token tiles, weight rows,
// token tile): pairs next to one another read the same weights.  Calls with fewer
// tiles than pairs split K over `splits` pairs of a cluster, which add up through
// distributed shared memory, always in the same order.
//
// Measured on the device, calls in a graph (and one by one with the caches flushed
// between them, the host's time included): 8 tokens of 16 of 896 MXFP4 experts, gates
// and ups 4,096 x 7,168, 288 us (286), 97% of a copy's rate; one row times 7,168 x 8,192
// 15.6 (15.8), 28 tiles by two pairs each, of which 7 are the start, the end and the
// join, then 7.0 TB/s; 64 rows times 10,240 x 7,168 18.6 (18.9), 40 tiles on 80 SMs, 7 and
// 6.1 TB/s; 8,192 rows times 7,168 x 8,192 274 to 300 (320), 3.2 to 3.5 PFLOP/s (power,
// and shared memory's 128 bytes a cycle); 4,096 tokens of 8 of 128 experts, gates and ups
// 4,096 x 4,096, 485 to 525 (575), and 7,168 x 2,048 in MXFP4 380 to 400 (439), 2.1 to 2.3
// and 2.4 to 2.5 PFLOP/s (copies, shared memory and the exchange of results: the tensor
// cores are busy half of the time).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "cluster.cuh"
#include "common.cuh"
#include "fp8_rows.cuh"
#include "tcgen05.cuh"

namespace moe {

constexpr int kGemmThreads = 512;
constexpr int kGemmK = 128;
constexpr int kGemmRows = 128;      // weight rows of a CTA's part of a tile
constexpr int kGemmTokens = 240;    // tokens of a tile at most
constexpr int kGemmMaxExperts = 1024;
constexpr int kGemmGroup = 16;      // token tiles that share a pass over the weights
constexpr int kGemmMaxStages = 12;
constexpr int kGemmMaxSplits = 4;   // pairs of a cluster (8 CTAs)

struct GemmShape {
  static constexpr int ABYTES = kGemmRows * kGemmK;
  // scales of four blocks of K: 4 bytes a row, of MXFP4 weights 4 a row and block
  static constexpr int SFA = 512, SFB = 1024, SFSLOT = 4 * SFA + SFB, SFSLOTS = 3;
  static constexpr int SFCOL = 480;             // tensor memory: accumulators at 0 and 240, scales
  // the ring of a call whose tiles have at most `tokens`: stages of `per` blocks of K
  // (weights, then tokens; all in multiples of 1,024, the swizzle's pattern), then
  // the scales
  __host__ __device__ static constexpr int stage(int tokens, int per) {
    return per * (ABYTES + tokens / 2 * kGemmK);
  }
  static constexpr int STATIC = 22 * 1024;   // GemmShared at most
  static constexpr int LIMIT = 227 * 1024 - STATIC;
  static constexpr int stages(int tokens, int per) {
    const int n = (LIMIT - 1024 - SFSLOTS * SFSLOT) / stage(tokens, per);
    return n < kGemmMaxStages ? n : kGemmMaxStages;
  }
  static constexpr int smem(int tokens, int per) {
    // (1,024: alignment)
    return stages(tokens, per) * stage(tokens, per) + SFSLOTS * SFSLOT + 1024;
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
  const uint8_t* x;
  long long x_stride;
  int k;
  const uint8_t* xs;
  long long xs_stride;
  const uint8_t* ws;
  long long ws_stride, ws_expert;
  char* out;
  long long out_stride;      // bytes
  uint8_t* os;
  long long os_stride;
  int out_dtype, vec;        // vec: rows of out are aligned to 16 bytes, of codes to 4
  int xs_align, ws_align;    // of the scales' rows: 16, 8, 4 or 1
  int fault;                 // 0, or 1 + the pair whose copies are left out (a test's)
  unsigned long long wait_ns;   // of a wait at most
};

struct GemmMaps {
  CUtensorMap w;
  CUtensorMap x[kGemmTokens / 16];   // boxes of 8, 16, .. rows: a CTA's part of a tile's tokens
};

struct GemmShared {
  uint64_t full[kGemmMaxStages], empty[kGemmMaxStages], loaded[kGemmMaxStages];
  uint64_t sf_full[GemmShape::SFSLOTS], sf_empty[GemmShape::SFSLOTS];
  uint64_t acc_full[2], acc_empty[2], amax_full[2][2], drained;
  uint32_t tmem;
  int dead;                           // a wait ran out
  int first[kGemmMaxExperts + 1];     // output row of each expert
  int tiles[kGemmMaxExperts + 1];     // token tiles before each expert
  int warp_scan[kGemmThreads / 32];
  // SwiGLU, by group of warps: four tokens' gates or ups on their way from each warp
  // to the one that holds the others, in turn in two places;
  float4 swap[2][4][2][32];
  // 8 bits: of 64 tokens the largest result of each of the pair's warps that have
  // them, in turn in two places, and the scales' reciprocals
  float amax[2][2][4][64];
  alignas(16) float inv[2][64];
};
static_assert(sizeof(GemmShared) <= GemmShape::STATIC, "the ring's room is the block's less this");
static_assert(GemmShape::stages(kGemmTokens, 2) >= 3, "the rows' loaders count on three stages");

// ---- barriers between the CTAs of a pair ----
// Waits for a phase, two seconds at most; then the CTA is dead: its waits end with
// false and its results become NaN.  So do the whole cluster's (gemm_spread), since a
// CTA's sums are its peer's products, or the other pairs' parts of K too: every wait
// that sums depend on ends at the issuing thread, which passes it on ahead of the
// sums' barrier.  (Not from the waits: with that loop behind each of them a prompt's
// gates and ups took 608 us for 485; with the limit in shared memory 500.)
__device__ __forceinline__ bool gemm_dead(GemmShared& sh) { return *(volatile int*)&sh.dead != 0; }
__device__ __forceinline__ void gemm_spread(GemmShared& sh) {
  if (!gemm_dead(sh)) return;
  const uint32_t ctas = cluster_size();
  for (uint32_t c = 0; c < ctas; ++c)
    asm volatile("st.volatile.shared::cluster.u32 [%0], 1;" ::"r"(
                     cluster_map(smem_addr(&sh.dead), c))
                 : "memory");
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}
__device__ __forceinline__ bool gemm_wait(uint64_t* bar, uint32_t parity, GemmShared& sh,
                                          const GemmArgs& a) {
  if (mbar_try_wait_long(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait_long(bar, parity)) {
    if (gemm_dead(sh)) return false;
    if (global_ns() - t0 > a.wait_ns) {
      *(volatile int*)&sh.dead = 1;
      return false;
    }
  }
  return true;
}
// The same for a whole warp, whose lanes go on, or give up, together.
__device__ __forceinline__ bool gemm_wait_warp(uint64_t* bar, uint32_t parity, GemmShared& sh,
                                               const GemmArgs& a) {
  return __all_sync(0xffffffffu, gemm_wait(bar, parity, sh, a));
}
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// `addr`: from cluster_map.  (Without a release to the cluster, which waits for the
// thread's loads and stores too: what is handed over lies in this CTA, whose own
// tensor cores read it, or is no data at all.)
__device__ __forceinline__ void gemm_arrive(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// ---- TMA; `bar` may be the other CTA's of the pair ----
// A block of K at column c: dimensions (column, row[, gate or up], matrix), of x
// (column, row).  Two blocks from block b on: K is two dimensions, (column, row, gate
// or up, block, matrix) and (column, row, block).  (No more dimensions than needed: a
// block a copy with five took a prompt 322 us for 298.)
__device__ __forceinline__ void tma_weights(uint32_t dst, const CUtensorMap* map, int c, int r,
                                            int e, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r), "r"(e), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_gates_ups(uint32_t dst, const CUtensorMap* map, int c, int r,
                                              int e, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %6, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r), "r"(e), "r"(bar), "r"(0)
      : "memory");
}
__device__ __forceinline__ void tma_tokens(uint32_t dst, const CUtensorMap* map, int c, int r,
                                           uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_weights2(uint32_t dst, const CUtensorMap* map, int r, int b,
                                             int e, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%6, %2, %6, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(r), "r"(b), "r"(e), "r"(bar), "r"(0)
      : "memory");
}
__device__ __forceinline__ void tma_tokens2(uint32_t dst, const CUtensorMap* map, int r, int b,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%5, %2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(r), "r"(b), "r"(bar), "r"(0)
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
  return min(max(__ldg(a.offsets + e), 0), a.rows);
}

// Inclusive scan over the block's threads.
template <class Op>
__device__ __forceinline__ int gemm_scan(int v, GemmShared& sh, Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = op(v, x);
  }
  __syncthreads();
  if (lane == 31) sh.warp_scan[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v = op(v, sh.warp_scan[w]);
  return v;
}

// First rows of the experts (none below an earlier one's: so no two experts have a
// row in common, whatever the offsets hold) and token tiles before each; every
// thread calls.
__device__ __forceinline__ void gemm_prefix(const GemmArgs& a, GemmShared& sh) {
  if (!a.offsets) {   // one matrix: no scans (they take 1.4 us)
    if (threadIdx.x < 2) {
      sh.first[threadIdx.x] = threadIdx.x * a.rows;
      sh.tiles[threadIdx.x] = threadIdx.x * ((a.rows + a.tokens - 1) / a.tokens);
    }
    __syncthreads();
    return;
  }
  constexpr int PER = (kGemmMaxExperts + kGemmThreads) / kGemmThreads;
  const int e0 = threadIdx.x * PER;
  int first[PER], top = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (e0 + i <= a.experts) top = max(top, gemm_start(a, e0 + i));
    first[i] = top;
  }
  const int upto = gemm_scan(top, sh, [](int x, int y) { return max(x, y); });
  // (the maximum before this thread's: a scan of maxima one thread on)
  int* scan = reinterpret_cast<int*>(sh.amax);   // (not in use yet)
  if (threadIdx.x + 1 < kGemmThreads) scan[threadIdx.x + 1] = upto;
  if (threadIdx.x == 0) scan[0] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (e0 + i <= a.experts) sh.first[e0 + i] = max(first[i], scan[threadIdx.x]);
  __syncthreads();
  int v[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i;
    v[i] = e < a.experts ? (sh.first[e + 1] - sh.first[e] + a.tokens - 1) / a.tokens : 0;
    sum += v[i];
  }
  int before = gemm_scan(sum, sh, [](int x, int y) { return x + y; }) - sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (e0 + i <= a.experts) sh.tiles[e0 + i] = before;
    before += v[i];
  }
  __syncthreads();
}

// Walks a pair's tiles and each one's blocks of K: all of them, or (splits) this
// pair's part, whole groups of four.  Whole warps call.
template <bool SWIGLU>
struct GemmWalk {
  unsigned t, tiles, step;   // (the host has seen that they are fewer than 2^31)
  int nt, k0, k1, expert;

  __device__ __forceinline__ GemmWalk(const GemmArgs& a, const GemmShared& sh) {
    constexpr int COLS = SWIGLU ? kGemmRows : 2 * kGemmRows;
    nt = (a.n + COLS - 1) / COLS;
    tiles = (unsigned)sh.tiles[a.experts] * nt;
    const int pair = blockIdx.x / 2, split = pair % a.splits;
    t = pair / a.splits;
    step = gridDim.x / 2 / a.splits;
    const int groups = (a.kb + 3) / 4;
    k0 = 4 * (int)((long long)groups * split / a.splits);
    k1 = min(a.kb, 4 * (int)((long long)groups * (split + 1) / a.splits));
    expert = 0;
  }

  __device__ __forceinline__ GemmTile tile(const GemmArgs& a, const GemmShared& sh) {
    // the expert with tiles[expert] * nt <= t < tiles[expert + 1] * nt, from the last on
    const int lane = threadIdx.x & 31;
    for (;;) {
      const int e = expert + 1 + lane;
      const unsigned past =
          __ballot_sync(0xffffffffu, e >= a.experts || (unsigned)sh.tiles[e] * nt > t);
      if (past) {
        expert += __ffs(past) - 1;
        break;
      }
      expert += 32;
    }
    const int mt = sh.tiles[expert + 1] - sh.tiles[expert];
    const int s = sh.first[expert], rows = sh.first[expert + 1] - s;
    unsigned in = t - (unsigned)sh.tiles[expert] * nt, n = in;
    int m = 0, size = (rows + 15) & ~15;
    if (mt > 1) {
      int g = 0, gm = mt;
      if (mt > kGemmGroup) {
        const unsigned pass = kGemmGroup * nt;
        g = in / pass;
        in -= g * pass;
        gm = min(kGemmGroup, mt - g * kGemmGroup);
      }
      n = in / (unsigned)gm;
      m = g * kGemmGroup + (int)(in - n * gm);
      // an expert's tokens in equal parts, none of them empty: (mt - 1) * size <=
      // (mt - 1) * a.tokens < rows
      size = (int)((((unsigned)rows + mt - 1) / (unsigned)mt + 15) & ~15u);
    }
    GemmTile r;
    r.expert = expert;
    r.row0 = s + m * size;
    r.rows = min(size, rows - m * size);
    r.N = (r.rows + 15) & ~15;
    r.n0 = n * (SWIGLU ? kGemmRows : 2 * kGemmRows);
    return r;
  }
};

// The row of x behind token r of the tile (tokens past the tile: its last).
__device__ __forceinline__ int gemm_source(const GemmArgs& a, const GemmTile& w, int r) {
  const int i = w.row0 + min(r, w.rows - 1);
  const int s = a.src ? __ldg(a.src + i) : i;
  return min(max(s, 0), a.x_rows - 1);
}

struct GemmRing {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// ---------------------------------------------------------------------------
// Copies (warp 0)
// ---------------------------------------------------------------------------
template <bool W4, bool SWIGLU, int PER>
__device__ __forceinline__ void gemm_copy(const GemmArgs& a, GemmShared& sh, uint32_t base,
                                          const GemmMaps& maps, uint32_t rank) {
  using S = GemmShape;
  if (a.fault == (int)(blockIdx.x / 2) + 1) return;
  const int lane = threadIdx.x & 31, half = rank & 1;
  const uint32_t stage_bytes = S::stage(a.tokens, PER);
  const uint32_t full = cluster_map(smem_addr(sh.full), rank & ~1u);
  GemmRing ring;
  for (GemmWalk<SWIGLU> k(a, sh); k.t < k.tiles; k.t += k.step) {
    const GemmTile w = k.tile(a, sh);
    // the pair's bytes a block (nibbles count as the bytes they are read as; blocks
    // past the last are zeros)
    const uint32_t bytes =
        (W4 ? S::ABYTES : 2 * S::ABYTES) + (a.src ? 0u : (uint32_t)w.N * kGemmK);
    const CUtensorMap* xm = &maps.x[w.N / 16 - 1];
    for (int kb = k.k0; kb < k.k1; kb += PER, ring.next(a.stages)) {
      if (!gemm_wait_warp(&sh.empty[ring.stage], ring.phase ^ 1, sh, a)) return;
      const uint32_t bar = full + ring.stage * 8, at = base + ring.stage * stage_bytes;
      if (half == 0 && lane == 0) mbar_arrive_expect_tx(&sh.full[ring.stage], PER * bytes);
      __syncwarp();
      // as few copies as can be: each takes the copy engine some 30 ns beside its rows
      if constexpr (PER == 2) {
        if (lane == 0)
          tma_weights2(at, &maps.w, w.n0 + half * (SWIGLU ? 64 : kGemmRows), kb, w.expert, bar);
        if (lane == 8 && !a.src)
          tma_tokens2(at + PER * S::ABYTES, xm, w.row0 + half * (w.N / 2), kb, bar);
      } else {
        if (lane == 0) {
          if (SWIGLU) tma_gates_ups(at, &maps.w, kb * kGemmK, w.n0 + half * 64, w.expert, bar);
          else tma_weights(at, &maps.w, kb * kGemmK, w.n0 + half * kGemmRows, w.expert, bar);
        }
        if (!a.src && lane == 8)
          tma_tokens(at + S::ABYTES, xm, kb * kGemmK, w.row0 + half * (w.N / 2), bar);
      }
    }
  }
  // the last arrivals from the pair's first CTA are in before this one may leave
  for (int i = 0; i < a.stages; ++i, ring.next(a.stages))
    if (!gemm_wait_warp(&sh.empty[ring.stage], ring.phase ^ 1, sh, a)) return;
}

// ---------------------------------------------------------------------------
// Rows of x by index (warps 12..14, a stage each in turn): 4 rows of eight
// 16-byte pieces at a time, laid out as the swizzle has them (piece c of row r at c ^
// (r % 8)).  Columns past K become zeros.  (The copy engine's gather takes it some
// 50 ns for four rows of 128 bytes: with 130 tokens a tile a block took 0.9 us, and
// with 8 a CTA 0.3 instead of 0.2.)  Warp 15 hands the blocks over to the tensor
// cores: the fence that this takes waits for every copy that its thread has under
// way, so the threads that copy must not need it (a block then took 0.45 us, however
// few its rows).
// A warp may wait for a stage's barrier every third use of it only.  It cannot take a
// phase for the one two before: its last fill, three before this one, was let in
// after all fills up to the ring's length before that one were done with, and this
// stage's use two before is among them (rings have three stages at least).
// ---------------------------------------------------------------------------
constexpr int kGemmLoaders = 3;   // warps

template <bool SWIGLU, int PER>
__device__ __forceinline__ void gemm_load_rows(const GemmArgs& a, GemmShared& sh, uint32_t base,
                                               uint32_t rank) {
  using S = GemmShape;
  const int lane = threadIdx.x & 31, half = rank & 1, sub = lane >> 3, c = lane & 7;
  const uint32_t stage_bytes = S::stage(a.tokens, PER);
  // even passes' rows are 0..3 of 8, odd ones' 4..7
  const uint32_t to0 = base + PER * S::ABYTES + sub * kGemmK + ((c ^ sub) << 4);
  const uint32_t to1 = base + PER * S::ABYTES + (4 + sub) * kGemmK + ((c ^ (4 + sub)) << 4);
  // the next tile's rows are read ahead (behind the copies under way they took 3 us a
  // tile)
  int ahead[4] = {};
  auto read_rows = [&](const GemmTile& w) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (32 * i + lane < w.N / 2) ahead[i] = gemm_source(a, w, half * (w.N / 2) + 32 * i + lane);
  };
  GemmRing ring;
  int turn = (int)(threadIdx.x >> 5) - 12;   // fills until this warp's next one
  GemmWalk<SWIGLU> k(a, sh);
  GemmTile next{};
  if (k.t < k.tiles) {
    next = k.tile(a, sh);
    read_rows(next);
  }
  while (k.t < k.tiles) {
    const GemmTile w = next;
    const int rows = w.N / 2;   // a multiple of 8
    unsigned src[kGemmTokens / 8];
#pragma unroll
    for (int i = 0; i < kGemmTokens / 8; ++i)
      src[i] = __shfl_sync(0xffffffffu, ahead[i / 8], i % 8 * 4 + sub);
    k.t += k.step;
    if (k.t < k.tiles) {
      next = k.tile(a, sh);
      read_rows(next);
    }
    for (int kb = k.k0; kb < k.k1; kb += PER, ring.next(a.stages)) {
      if (turn-- > 0) continue;
      turn = kGemmLoaders - 1;
      if (!gemm_wait_warp(&sh.empty[ring.stage], ring.phase ^ 1, sh, a)) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
      }
#pragma unroll 1
      for (int b = 0; b < PER && kb + b < k.k1; ++b) {
        const uint32_t at = ring.stage * stage_bytes + b * (rows * kGemmK);
        const bool in = (kb + b) * kGemmK + c * 16 < a.k;   // (k is a multiple of 16)
        const uint8_t* x = a.x + (in ? (kb + b) * kGemmK + c * 16 : 0);
        const uint32_t size = in ? 16 : 0;
#pragma unroll
        for (int i = 0; i < kGemmTokens / 8; i += 2) {
          if (4 * i >= rows) break;
          const uint32_t to = at + i / 2 * 8 * kGemmK;
          asm volatile("" : "+r"(src[i]), "+r"(src[i + 1]));   // (offsets are not kept: registers)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to0 + to),
                       "l"(x + (uint64_t)src[i] * (uint32_t)a.x_stride), "r"(size)
                       : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to1 + to),
                       "l"(x + (uint64_t)src[i + 1] * (uint32_t)a.x_stride), "r"(size)
                       : "memory");
        }
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                       smem_addr(&sh.loaded[ring.stage]))
                   : "memory");
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// All stages that have arrived, up to four, behind one fence.
template <bool SWIGLU, int PER>
__device__ __forceinline__ void gemm_hand_over(const GemmArgs& a, GemmShared& sh, uint32_t rank) {
  const int lane = threadIdx.x & 31;
  const uint32_t full = cluster_map(smem_addr(sh.full), rank & ~1u);
  const GemmWalk<SWIGLU> k(a, sh);
  long long left = 0;
  if (k.t < k.tiles)
    left = (long long)((k.tiles - 1 - k.t) / k.step + 1) * ((k.k1 - k.k0 + PER - 1) / PER);
  GemmRing ring;
  while (left > 0) {
    if (!gemm_wait_warp(&sh.loaded[ring.stage], ring.phase, sh, a)) return;
    uint32_t mine = ring.stage;   // lane l's stage
    int n = 1;
    for (ring.next(a.stages); n < 4 && n < left; ++n, ring.next(a.stages)) {
      if (!__all_sync(0xffffffffu, mbar_test_wait(&sh.loaded[ring.stage], ring.phase))) break;
      if (lane == n) mine = ring.stage;
    }
    fence_async_shared();
    if (lane < n) gemm_arrive(full + mine * 8);
    left -= n;
  }
}

// ---------------------------------------------------------------------------
// Scales (warps 2, 3): four blocks of K at a time, for 128 rows at a time, 16 bytes
// a lane: one word for each of the rows lane, lane + 32, lane + 64, lane + 96.  A
// word holds the bytes of the four blocks, or (MXFP4 weights) of a block's four
// steps.  A ring of their own, read a batch of 8 blocks ahead.
// ---------------------------------------------------------------------------
// Words of R rows a lane (4: weights, 8: tokens) from byte `at` on, of rows of
// `end` bytes; `align`: what every row's start is a multiple of (16, 8, 4 or 1); `at` is a
// multiple of 4 (splits begin at groups of four blocks).
template <int R, int W>
__device__ __forceinline__ void scales_load(const uint8_t* const (&p)[R], int at, int end,
                                            int align, uint32_t (&v)[R][W]) {
  if (W == 2 && align >= 8 && (at & 7) == 0 && at + 8 <= end) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(p[i] + at));
      v[i][0] = u.x;
      v[i][1] = u.y;
    }
  } else if (W % 4 == 0 && align == 16 && (at & 15) == 0 && at + 4 * W <= end) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j + 3 < W; j += 4) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p[i] + at + 4 * j));
        v[i][j] = u.x;
        v[i][j + 1] = u.y;
        v[i][j + 2] = u.z;
        v[i][j + 3] = u.w;
      }
  } else if (align >= 4 && (at + 4 * W <= end || (end & 3) == 0)) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (at + 4 * j < end) v[i][j] = __ldg(reinterpret_cast<const uint32_t*>(p[i] + at) + j);
  } else {
#pragma unroll 1
    for (int j = 0; j < W; ++j)
      for (int b = 0; b < 4; ++b) {
        if (at + 4 * j + b >= end) break;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const uint32_t u = (uint32_t)__ldg(p[i] + at + 4 * j + b) << (8 * b);
#pragma unroll
          for (int k = 0; k < W; ++k)   // (no indexed registers)
            if (k == j) v[i][k] = b ? v[i][k] | u : u;
        }
      }
  }
}

template <int R, bool PERK, bool SWIGLU, class Rows>
__device__ __forceinline__ void gemm_scales(const GemmArgs& a, GemmShared& sh, uint8_t* dst,
                                            uint32_t rank, int align, Rows rows_of) {
  using S = GemmShape;
  constexpr int BATCH = 8, W = PERK ? 8 : 2, BYTES = PERK ? 4 : 1;   // a block
  const int lane = threadIdx.x & 31;
  const uint32_t full = cluster_map(smem_addr(sh.sf_full), rank & ~1u);
  GemmRing ring;
  for (GemmWalk<SWIGLU> k(a, sh); k.t < k.tiles; k.t += k.step) {
    const uint8_t* p[R];
    rows_of(k, p);
    uint32_t cur[R][W], next[R][W] = {};
    scales_load(p, BYTES * k.k0, BYTES * a.kb, align, next);
    for (int k0 = k.k0; k0 < k.k1; k0 += BATCH) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) cur[i][j] = next[i][j];
      if (k0 + BATCH < k.k1) scales_load(p, BYTES * (k0 + BATCH), BYTES * a.kb, align, next);
#pragma unroll
      for (int s = 0; s < BATCH / 4; ++s) {
        if (k0 + 4 * s >= k.k1) break;
        if (!gemm_wait_warp(&sh.sf_empty[ring.stage], ring.phase ^ 1, sh, a)) return;
        uint4* to = reinterpret_cast<uint4*>(dst + ring.stage * S::SFSLOT);
#pragma unroll
        for (int j = 0; j < (PERK ? 4 : 1); ++j)
#pragma unroll
          for (int g = 0; g < R / 4; ++g) {
            const int c = PERK ? 4 * s + j : s;
            to[32 * (j + g) + lane] = make_uint4(cur[4 * g][c], cur[4 * g + 1][c],
                                                 cur[4 * g + 2][c], cur[4 * g + 3][c]);
          }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) gemm_arrive(full + ring.stage * 8);
        ring.next(S::SFSLOTS);
      }
    }
  }
  for (int i = 0; i < S::SFSLOTS; ++i, ring.next(S::SFSLOTS))   // (as the copies' end)
    if (!gemm_wait_warp(&sh.sf_empty[ring.stage], ring.phase ^ 1, sh, a)) return;
}

// ---------------------------------------------------------------------------
// MMAs (warp 1 of the pair's first CTA)
// ---------------------------------------------------------------------------
// One thread, chosen once a tile: the loop's own latency counts.  A block's four MMAs
// take the tensor cores 480 cycles at most; with the whole warp in the loop (a
// choice of the lane, a vote on every wait, an early test of the next barrier a
// block) it took 640, without the last two 490, so 230.  Where a wait ran out, the
// others end at once and what is issued is garbage of no effect.
template <bool W4, bool SWIGLU, int PER>
__device__ __forceinline__ void gemm_mma(const GemmArgs& a, GemmShared& sh, uint32_t base,
                                         uint32_t rank) {
  using S = GemmShape;
  const uint32_t stage_bytes = S::stage(a.tokens, PER), sf = base + a.stages * stage_bytes;
  const uint16_t both = (uint16_t)(3u << (rank & ~1u));
  const uint64_t da0 = umma_desc_sw128(base), db0 = umma_desc_sw128(base + PER * S::ABYTES);
  const uint64_t ds0 = umma_desc(sf, 0, 128);
  GemmRing ring, sr;
  const uint32_t tm = sh.tmem;
  uint32_t n = 0;
  for (GemmWalk<SWIGLU> k(a, sh); k.t < k.tiles; k.t += k.step, ++n) {
    const GemmTile w = k.tile(a, sh);
    const uint32_t acc = tm + (n & 1) * kGemmTokens, id = umma_idesc_mxf8(W4 ? 5 : 0, 0, 0, w.N);
    gemm_wait(&sh.acc_empty[n & 1], (n >> 1 & 1) ^ 1, sh, a);
    if (elect_one()) {
      for (int kb = k.k0; kb < k.k1; kb += 4) {
        const uint32_t j4 = kb >> 2 & 1, sfb = tm + S::SFCOL + 8 + 8 * j4;
        const uint64_t ds = ds0 + sr.stage * (S::SFSLOT >> 4);
        gemm_wait(&sh.sf_full[sr.stage], sr.phase, sh, a);
        tc_fence_after();
        umma_sf_copy_pair(sfb, ds + (4 * S::SFA >> 4));
        if (w.N > 128) umma_sf_copy_pair(sfb + 4, ds + ((4 * S::SFA + 512) >> 4));
        if (!W4) umma_sf_copy_pair(tm + S::SFCOL + 4 * j4, ds);
#pragma unroll
        for (uint32_t b = 0; b < 4; ++b) {
          if (kb + (int)b >= k.k1) break;
          // scales of this block (MXFP4 weights) or these four, in turn in two places
          const uint32_t sfa = tm + S::SFCOL + 4 * (W4 ? b & 1 : j4);
          const uint64_t off = ring.stage * (stage_bytes >> 4);
          uint64_t da = da0 + off, db = db0 + off;
          if constexpr (PER == 2) {   // the second block of a stage
            da += (b & 1) * (S::ABYTES >> 4);
            db += (b & 1) * (w.N / 2 * kGemmK >> 4);
          }
          if (PER == 1 || (b & 1) == 0) {
            gemm_wait(&sh.full[ring.stage], ring.phase, sh, a);
            tc_fence_after();
          }
          if (W4) umma_sf_copy_pair(sfa, ds + b * (S::SFA >> 4));
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j)
            umma_mxf8_pair(acc, da + 2 * j, db + 2 * j, id | (W4 ? j : b) << 29 | b << 4, sfa, sfb,
                           (kb > k.k0) || b > 0 || j > 0);
          if (PER == 1 || (b & 1) || kb + (int)b + 1 >= k.k1) {
            umma_commit_pair(&sh.empty[ring.stage], both);
            ring.next(a.stages);
          }
        }
        umma_commit_pair(&sh.sf_empty[sr.stage], both);
        sr.next(S::SFSLOTS);
      }
      gemm_spread(sh);
      umma_commit_pair(&sh.acc_full[n & 1], both);
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// Results (warps 4..11): a thread a weight row (an output column), tokens in turn
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

// T tokens of this thread's output column to out.
template <int T>
__device__ __forceinline__ void gemm_store(const GemmArgs& a, const GemmTile& w, int c, int col,
                                           const float (&v)[T]) {
  const int lane = threadIdx.x & 31;
  if (a.out_dtype == MOE_DTYPE_F32) {
    if (col >= a.n) return;
    char* p = a.out + (long long)(w.row0 + c) * a.out_stride + (long long)col * 4;
#pragma unroll
    for (int i = 0; i < T; ++i, p += a.out_stride)
      if (c + i < w.rows) *reinterpret_cast<float*>(p) = v[i];
    return;
  }
  const int f16 = a.out_dtype == MOE_DTYPE_F16;
  if (!a.vec) {   // rows at odd places: a warp's columns of a token side by side
    char* p = a.out + (long long)(w.row0 + c) * a.out_stride + (long long)col * 2;
#pragma unroll
    for (int i = 0; i < T; ++i, p += a.out_stride)
      if (c + i < w.rows && col < a.n)
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack16(v[i], 0.f, f16);
    return;
  }
  // eight tokens of eight lanes' columns are turned among the lanes, so that each
  // stores eight columns of one token (16 bytes; by 4 bytes a lane the stores
  // took as long as a tile of K = 2,048: 692 us for 408 without them)
  const int b0 = lane & 1, b1 = lane >> 1 & 1, b2 = lane >> 2 & 1, col8 = col & ~7;
  char* p = a.out + (long long)(w.row0 + c + (lane & 7)) * a.out_stride + (long long)col8 * 2;
#pragma unroll
  for (int i = 0; i < T; i += 8, p += 8 * a.out_stride) {
    // columns (col & ~1, + 1) of token 2 j + b0
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = v[i + 2 * j], hi = v[i + 2 * j + 1];
      const float x = __shfl_xor_sync(0xffffffffu, b0 ? lo : hi, 1);
      u[j] = b0 ? pack16(x, hi, f16) : pack16(lo, x, f16);
    }
    // columns col & ~3 .. + 3 of token 4 j + 2 b1 + b0: words (2 j, 2 j + 1)
    uint32_t s[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t lo = u[2 * j], hi = u[2 * j + 1];
      const uint32_t x = __shfl_xor_sync(0xffffffffu, b1 ? lo : hi, 2);
      s[2 * j] = b1 ? x : lo;
      s[2 * j + 1] = b1 ? hi : x;
    }
    // all eight of token 4 b2 + 2 b1 + b0
    const uint32_t x0 = __shfl_xor_sync(0xffffffffu, b2 ? s[0] : s[2], 4);
    const uint32_t x1 = __shfl_xor_sync(0xffffffffu, b2 ? s[1] : s[3], 4);
    const uint4 o = b2 ? make_uint4(x0, x1, s[2], s[3]) : make_uint4(s[0], s[1], x0, x1);
    if (c + i + (lane & 7) >= w.rows) continue;
    if (col8 + 7 < a.n) {
      *reinterpret_cast<uint4*>(p) = o;
    } else {
      const uint32_t t[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col8 + j < a.n)
          reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(t[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// silu(gate) * up of 32 tokens: warps 0 and 1 of a group hold gates, 2 and 3 the ups of
// the same columns.  The first two get the results of the first 16 tokens, the others
// of the rest; what each needs of the other goes through shared memory, four tokens
// at a time, in turn in two places: a warp writes a place again only behind the
// barrier of the turn between, which the other passes when it has read it.  (Fast
// functions: their errors are below those of the sums, and no result differs more
// with exact ones, which took a prompt's gates and ups from 484 to 606 us.  The
// division gives 0 where the denominator passes 2^126, gates below -87.3, whose silu
// is less than 1.1e-36; another formula for them took 526 us.)
__device__ __forceinline__ void gemm_swiglu(GemmShared& sh, int group, int q, const float (&v)[32],
                                            float* h) {
  const int lane = threadIdx.x & 31;
  const bool up = q >= 2;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const int b = i >> 2 & 1;
    sh.swap[group][q][b][lane] = up ? make_float4(v[i], v[i + 1], v[i + 2], v[i + 3])
                                    : make_float4(v[i + 16], v[i + 17], v[i + 18], v[i + 19]);
    asm volatile("bar.sync %0, 64;" ::"r"(3 + 2 * group + (q & 1)) : "memory");
    const float4 o = sh.swap[group][q ^ 2][b][lane];
    const float x[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float g = up ? x[j] : v[i + j], u = up ? v[i + j + 16] : x[j];
      h[i + j] = __fdividef(g, 1.f + __expf(-g)) * u;
    }
  }
}

// Maxima of 16 values each over the warp: lane l gets value l & 15's.
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
  return fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], 16));
}

template <bool SWIGLU>
__device__ __forceinline__ void gemm_results(const GemmArgs& a, GemmShared& sh, uint8_t* smem,
                                             uint32_t rank) {
  const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3, half = rank & 1;
  const int group = (threadIdx.x >> 7) - 1, gt = threadIdx.x & 127;
  const uint32_t tm = sh.tmem + ((uint32_t)(q * 32) << 16);
  const uint32_t part = smem_addr(smem) + gt * 4;
  const int split = (blockIdx.x / 2) % a.splits;
  const float nan = __int_as_float(0x7FFFFFFF);
  const uint32_t acc_empty = cluster_map(smem_addr(sh.acc_empty), rank & ~1u);
  uint32_t n = 0, batch = 0;
  for (GemmWalk<SWIGLU> k(a, sh); k.t < k.tiles; k.t += k.step, ++n) {
    const GemmTile w = k.tile(a, sh);
    if (!gemm_dead(sh)) gemm_wait(&sh.acc_full[n & 1], n >> 1 & 1, sh, a);   // (dead: NaN)
    tc_fence_after();
    const uint32_t acc = tm + (n & 1) * kGemmTokens;
    // tokens go to splits and groups in turn, `unit` at a time; the groups begin in
    // turn too (a tile may have a unit only)
    int unit = 32, c0 = 32 * ((group ^ (n & 1)) * a.splits + split);
    if (SWIGLU && a.out_dtype == MOE_DTYPE_E4M3) unit = 64, c0 *= 2;
    const int step = 2 * unit * a.splits;
    if (a.splits > 1) {
      // this pair's part of K to shared memory (the ring is idle: every copy was
      // waited for and every product is done), then the tokens are shared out
      for (int c = 32 * group; c < w.N; c += 64) {
        float v[32];
        tmem_ld32(acc + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i < w.N) *reinterpret_cast<float*>(smem + (c + i) * 512 + gt * 4) = v[i];
      }
      cluster_sync();
    }
    const bool dead = gemm_dead(sh);
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) gemm_arrive(acc_empty + (n & 1) * 8);
    };
    if (c0 >= w.N) release();
    if (!SWIGLU) {
      const int col = w.n0 + half * kGemmRows + q * 32 + lane;
#pragma unroll 1
      for (int c = c0; c < w.N; c += step) {
        float v[32];
        gemm_sums(a, acc, part, rank, c, v);
        if (c + step >= w.N) release();
        if (dead) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = nan;
        }
        gemm_store(a, w, c, col, v);
      }
      continue;
    }
    // this warp's results: column col of the tokens from 16 on, or below (gemm_swiglu)
    const int col = w.n0 + half * 64 + (q & 1) * 32 + lane, late = q >= 2 ? 16 : 0;
    if (a.out_dtype != MOE_DTYPE_E4M3) {
#pragma unroll 1
      for (int c = c0; c < w.N; c += step) {
        float v[32], h[16];
        gemm_sums(a, acc, part, rank, c, v);
        if (c + step >= w.N) release();
        gemm_swiglu(sh, group, q, v, h);
        if (dead) {
#pragma unroll
          for (int i = 0; i < 16; ++i) h[i] = nan;
        }
        gemm_store(a, w, c + late, col, h);
      }
      continue;
    }
    // 8 bits.  A token's 128 results lie in both CTAs, in two warps each: each warp
    // sends its largest to both CTAs, 64 tokens at a time, whose results stay in
    // registers.  Places and barriers are taken in turn: a peer that has ended a batch
    // may send the next one's words before all of its own of this batch have landed
    // here, and they must not count for it; those after next it sends only when it has
    // this CTA's of the next batch, which follow the wait for this one, and its
    // reading (the barrier below).
#pragma unroll 1
    for (int c1 = c0; c1 < w.N; c1 += step, ++batch) {
      uint64_t* bar = &sh.amax_full[group][batch & 1];
      const uint32_t slot = smem_addr(sh.amax[group][batch & 1][half * 2 + (q & 1)]);
      const uint32_t here = cluster_map(slot, rank), there = cluster_map(slot, rank ^ 1);
      const uint32_t bar_here = cluster_map(smem_addr(bar), rank);
      const uint32_t bar_there = cluster_map(smem_addr(bar), rank ^ 1);
      const bool wide = c1 + 32 < w.N;   // more than 32 tokens left
      if (gt == 0) mbar_arrive_expect_tx(bar, wide ? 4 * 64 * 4 : 4 * 32 * 4);
      float h[32];
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        if (c && !wide) continue;
        float v[32], m[16];
        gemm_sums(a, acc, part, rank, c1 + c, v);   // (past N: nobody's)
        gemm_swiglu(sh, group, q, v, h + c / 2);
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i] = col < a.n ? fp8_finite_max(0.f, h[c / 2 + i]) : 0.f;
        const float top = gemm_max16(m);
        const int t = c + late + (lane & 15);
        // (the lower lanes to this CTA, the others to its peer)
        st_async_f32((lane < 16 ? here : there) + t * 4, top, lane < 16 ? bar_here : bar_there);
      }
      if (c1 + step >= w.N) release();
      const bool lost = !gemm_wait(bar, batch >> 1 & 1, sh, a) || dead;
      if (gt < 64) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = fmaxf(amax, sh.amax[group][batch & 1][i][gt]);
        const int e = fp8_block_exp(amax);
        sh.inv[group][gt] = pow2f(-e);
        if (half == 0 && c1 + gt < w.rows)
          a.os[(long long)(w.row0 + c1 + gt) * a.os_stride + (w.n0 >> 7)] =
              lost ? 255 : (uint8_t)(e + 127);
      }
      asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        if (i == 16 && !wide) break;
        // four tokens' codes of this column, turned among four lanes into four
        // columns' codes of one token
        const int t0 = (i & 16) * 2 + late + (i & 15);
        const float4 inv = *reinterpret_cast<const float4*>(&sh.inv[group][t0]);
        uint32_t u = f32x2_to_e4m3x2(h[i] * inv.x, h[i + 1] * inv.y) |
                     f32x2_to_e4m3x2(h[i + 2] * inv.z, h[i + 3] * inv.w) << 16;
        if (lost) u = 0x7F7F7F7Fu;
        if (!a.vec) {   // rows at odd places: a warp's columns of a token side by side
          char* p = a.out + (long long)(w.row0 + c1 + t0) * a.out_stride + col;
#pragma unroll
          for (int j = 0; j < 4; ++j, p += a.out_stride)
            if (c1 + t0 + j < w.rows && col < a.n) *p = (char)(u >> (8 * j));
          continue;
        }
        const uint32_t x = __shfl_xor_sync(0xffffffffu, u, 1);
        u = lane & 1 ? __byte_perm(u, x, 0x3715) : __byte_perm(u, x, 0x6240);
        const uint32_t y = __shfl_xor_sync(0xffffffffu, u, 2);
        u = lane & 2 ? __byte_perm(u, y, 0x3276) : __byte_perm(u, y, 0x5410);
        const int t = c1 + t0 + (lane & 3), at = col & ~3;
        if (t >= w.rows) continue;
        char* p = a.out + (long long)(w.row0 + t) * a.out_stride + at;
        if (at + 3 < a.n) {
          *reinterpret_cast<uint32_t*>(p) = u;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (at + j < a.n) p[j] = (char)(u >> (8 * j));
        }
      }
      asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");   // (inv is read)
    }
  }
}

// PER: blocks of K a stage.
template <bool W4, bool SWIGLU, int PER>
static __global__ void __launch_bounds__(kGemmThreads, 1)
    fp8_product_kernel(const __grid_constant__ GemmArgs a,
                       const __grid_constant__ GemmMaps maps) {
  using S = GemmShape;
  extern __shared__ uint8_t gemm_raw[];
  __shared__ GemmShared sh;
  uint8_t* smem = gemm_raw + ((1024 - (smem_addr(gemm_raw) & 1023)) & 1023);
  const uint32_t base = smem_addr(smem), rank = cluster_rank();
  const int warp = threadIdx.x >> 5;
  if (warp == 0) {
    const int s = threadIdx.x;
    if (s < a.stages) {
      mbar_init(&sh.full[s], a.src ? 3 : 1);   // the copies, what the pair's loaders brought
      mbar_init(&sh.loaded[s], 32);
      mbar_init(&sh.empty[s], 1);
    }
    if (s < S::SFSLOTS) {
      mbar_init(&sh.sf_full[s], 4);   // two warps of both CTAs
      mbar_init(&sh.sf_empty[s], 1);
    }
    if (s < 2) {
      mbar_init(&sh.acc_full[s], 1);
      mbar_init(&sh.acc_empty[s], 16);   // eight warps of both CTAs
      mbar_init(&sh.amax_full[s][0], 1);
      mbar_init(&sh.amax_full[s][1], 1);
    }
    if (s == 0) {
      mbar_init(&sh.drained, 1);
      sh.dead = 0;
      asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.w) : "memory");
    }
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(&sh.tmem);
  pdl_wait_prerequisites();   // (the launch before may still be running up to here)
  gemm_prefix(a, sh);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();

  if (warp == 0) {
    gemm_copy<W4, SWIGLU, PER>(a, sh, base, maps, rank);
  } else if (warp == 1) {
    if ((rank & 1) == 0) gemm_mma<W4, SWIGLU, PER>(a, sh, base, rank);
  } else if (warp == 2) {
    gemm_scales<4, W4, SWIGLU>(
        a, sh, smem + a.stages * S::stage(a.tokens, PER), rank, a.ws_align,
        [&](GemmWalk<SWIGLU>& k, const uint8_t* (&p)[4]) {
          const GemmTile w = k.tile(a, sh);
          const int lane = threadIdx.x & 31, half = rank & 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            int r = w.n0 + half * kGemmRows + 32 * i + lane;
            if (SWIGLU) r = (i < 2 ? 0 : a.n) + w.n0 + half * 64 + 32 * (i & 1) + lane;
            r = min(r, a.wide - 1);
            p[i] = a.ws + w.expert * a.ws_expert + (W4 ? r : r >> 7) * a.ws_stride;
          }
        });
  } else if (warp == 3) {
    gemm_scales<8, false, SWIGLU>(
        a, sh, smem + a.stages * S::stage(a.tokens, PER) + 4 * S::SFA, rank, a.xs_align,
        [&](GemmWalk<SWIGLU>& k, const uint8_t* (&p)[8]) {
          const GemmTile w = k.tile(a, sh);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = (threadIdx.x & 31) + 32 * i;
            p[i] = a.xs + gemm_source(a, w, r) * a.xs_stride;
          }
        });
  } else if (warp < 12) {
    gemm_results<SWIGLU>(a, sh, smem, rank);
  } else if (a.src) {
    if (warp < 15) gemm_load_rows<SWIGLU, PER>(a, sh, base, rank);
    else gemm_hand_over<SWIGLU, PER>(a, sh, rank);
  }
  pdl_launch_dependents();
  __syncwarp();
  // the results' warps' wait for the cluster, where it has a tile
  if (a.splits > 1 && (warp < 4 || warp >= 12)) {
    const GemmWalk<SWIGLU> k(a, sh);
    if (k.t < k.tiles) cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) gemm_spread(sh);
  __syncwarp();
  cluster_sync();   // (nor does a CTA leave while another may read its sums)
  if (gemm_dead(sh)) {
    // (no wait is left to run out, so all of the cluster are here or none)  Products,
    // copies and words in flight, before their memory is given back: bounded too
    if (warp == 1) {
      if (elect_one()) {
        if ((rank & 1) == 0) {
          umma_commit_pair(&sh.drained, (uint16_t)(1u << rank));
          for (int i = 0; i < 100 && !mbar_try_wait_long(&sh.drained, 0); ++i) {
          }
        }
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 2000000) {
        }
      }
      __syncwarp();
    }
    __syncthreads();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(sh.tmem);
  }
}

}  // namespace moe
