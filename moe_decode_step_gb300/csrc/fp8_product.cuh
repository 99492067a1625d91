// Products of 8-bit activations with 8-bit or MXFP4 weights, dense or by expert.
//
// tcgen05 block-scaled MMAs (kind::mxf8f6f4): both operands enter as stored,
// E4M3 rows of 128 columns brought by TMA into 128-byte-swizzled tiles, E2M1
// weights unpacked on the way in (8 bytes of nibbles in every 16), and their
// E8M0 scales in tensor memory, so no product is scaled or converted by a
// thread.  A tile is 128 output rows x 256 weight rows; K goes 128 columns at a
// time through a ring of stages.
//
// Roles (8 warps): 0 copies tiles (TMA; rows of x picked by index through
// gather4, four a copy), 1 issues the MMAs, 2 and 3 lay the scales of x and of
// the weights out, 4..7 the results, a thread a row.  The CTAs, one an SM, take
// tiles in the order (expert, 16 row tiles, weight rows, row tile): CTAs next to
// one another read the same weights.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "common.cuh"
#include "fp8_rows.cuh"
#include "tcgen05.cuh"

namespace moe {

constexpr int kGemmThreads = 256;
constexpr int kGemmM = 128, kGemmN = 256, kGemmK = 128;
constexpr int kGemmStages = 4;
constexpr int kGemmMaxExperts = 1024;
constexpr int kGemmGroup = 16;   // row tiles that share a pass over the weights

struct GemmShape {
  static constexpr int ABYTES = kGemmM * kGemmK, BBYTES = kGemmN * kGemmK;
  static constexpr int STAGE = ABYTES + BBYTES;
  static constexpr int SFA = 512, SFB = 1024;              // scales of a stage
  static constexpr int SFOFF = kGemmStages * STAGE;
  static constexpr int OUTROW = 144;                       // 128 bytes of a row, bank-shifted
  static constexpr int OUTOFF = SFOFF + kGemmStages * (SFA + SFB);
  static constexpr int SMEM = OUTOFF + 4 * 32 * OUTROW + 1024;   // (1,024: alignment)
  static constexpr int SFCOL = 488;                        // tensor memory: scales, 12 columns twice
};

struct GemmArgs {
  int K, kb;                 // columns, blocks of 128 of them
  int n, wide;               // output columns; weight rows (n, or 2 n)
  int rows, x_rows, experts;
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
  int out_dtype, vec;        // vec: rows of out are 16-byte aligned
};

struct GemmShared {
  uint64_t full[kGemmStages], empty[kGemmStages];
  uint64_t acc_full, acc_empty, drained;
  uint32_t tmem;
  int dead;                           // a wait ran out
  int tiles[kGemmMaxExperts + 1];     // row tiles before each expert
  int warp_sum[kGemmThreads / 32];
};

// Waits for a phase, two seconds at most; then the CTA is dead: its waits all
// end at once and its results become NaN.
__device__ __forceinline__ bool gemm_dead(GemmShared& sh) { return *(volatile int*)&sh.dead != 0; }
__device__ __forceinline__ void gemm_wait(uint64_t* bar, uint32_t parity, GemmShared& sh) {
  if (mbar_try_wait_long(bar, parity)) return;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait_long(bar, parity)) {
    if (gemm_dead(sh)) return;
    if (global_ns() - t0 > kWaitLimitNs) {
      *(volatile int*)&sh.dead = 1;
      return;
    }
  }
}

// ---- TMA ----
__device__ __forceinline__ void tma_tile_2d(uint32_t dst, const CUtensorMap* map, int c, int r,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_tile_3d(uint32_t dst, const CUtensorMap* map, int c, int r,
                                            int e, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r), "r"(e), "r"(smem_addr(bar))
      : "memory");
}
// Four rows of a map whose box is one row.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int c,
                                            const int (&r)[4], uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(smem_addr(bar))
      : "memory");
}

// ---- MMA ----
// K-major operand with the 128-byte swizzle: rows of 128 bytes, groups of 8 rows.
__device__ __forceinline__ uint64_t umma_desc_sw128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor, kind::mxf8f6f4: A E4M3, B E4M3 (0) or E2M1 (5), E8M0
// scales, both K-major, M = 128; b_sf: the scale byte of the step.
__device__ __forceinline__ constexpr uint32_t umma_idesc_mxf8(uint32_t b_format, uint32_t b_sf,
                                                              uint32_t N) {
  return (b_sf << 4) | (b_format << 10) | ((N >> 3) << 17) | (1u << 23) | (8u << 24);
}
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
struct GemmTile {
  int expert, row0, rows;   // first output row, rows of the tile
  int n0;                   // first output column
};

__device__ __forceinline__ int gemm_start(const GemmArgs& a, int e) {
  if (!a.offsets) return e ? a.rows : 0;
  return min(max(__ldg(a.offsets + e), 0), a.rows);
}

// Row tiles before each expert; every thread calls.
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
      v[i] = (max(gemm_start(a, e + 1) - s, 0) + kGemmM - 1) / kGemmM;
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
  GemmTile r;
  r.expert = lo;
  r.row0 = s + m * kGemmM;
  r.rows = min(kGemmM, end - r.row0);
  r.n0 = in / gm * (SWIGLU ? kGemmN / 2 : kGemmN);
  return r;
}

// The row of x behind row r of the tile (rows past the tile: its last).
__device__ __forceinline__ int gemm_source(const GemmArgs& a, const GemmTile& w, int r) {
  const int i = w.row0 + min(r, w.rows - 1);
  const int s = a.src ? __ldg(a.src + i) : i;
  return min(max(s, 0), a.x_rows - 1);
}

struct GemmRing {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kGemmStages) {
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
                                          const CUtensorMap* wm, long long tiles, int nt) {
  using S = GemmShape;
  const int lane = threadIdx.x & 31;
  GemmRing ring;
  uint32_t issued = 0;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const GemmTile w = gemm_tile<SWIGLU>(a, sh, nt, t);
    // whole tiles of consecutive rows in one copy (past an expert's end it reads
    // the next one's, whose results nobody takes), others four rows a copy
    const bool gather = a.src || (a.offsets && w.rows <= kGemmM / 2);
    const bool mine = gather && 4 * lane < w.rows;
    int r[4];
    if (mine) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = gemm_source(a, w, 4 * lane + i);
    }
    // (nibbles count as the bytes they are read as)
    const uint32_t bytes =
        (W4 ? S::BBYTES / 2 : S::BBYTES) + (gather ? (uint32_t)(w.rows + 3) / 4 * 4 * kGemmK : (uint32_t)S::ABYTES);
    for (int k = 0; k < a.kb; ++k, ring.next(), ++issued) {
      gemm_wait(&sh.empty[ring.stage], ring.phase ^ 1, sh);
      if (gemm_dead(sh)) {
        // the copies in flight, before their memory is given back: bounded too
        for (uint32_t i = 0; i < min(issued, (uint32_t)kGemmStages); ++i) {
          const uint32_t f = issued - 1 - i;
          for (int j = 0; j < 20 && !mbar_try_wait_long(&sh.full[f % kGemmStages],
                                                 f / kGemmStages & 1); ++j) {
          }
        }
        return;
      }
      uint64_t* bar = &sh.full[ring.stage];
      const uint32_t at = base + ring.stage * S::STAGE;
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (lane < 2)
        tma_tile_3d(at + S::ABYTES + lane * (S::BBYTES / 2), wm, k * kGemmK,
                    lane == 0 ? w.n0 : SWIGLU ? a.n + w.n0 : w.n0 + kGemmN / 2, w.expert, bar);
      if (!gather) {
        if (lane == 2) tma_tile_2d(at, xt, k * kGemmK, w.row0, bar);
      } else if (mine) {
        tma_gather4(at + lane * 4 * kGemmK, xg, k * kGemmK, r, bar);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Scales (warps 2, 3): per stage, for 128 rows at a time, 16 bytes a lane: one
// word for each of the rows lane, lane + 32, lane + 64, lane + 96.  They are
// read four stages at a time and one such group ahead.
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

// R rows a lane (4: x, 8: weights).  PERK: a word of its own for each K block
// (MXFP4), else a byte.
template <int R, bool PERK>
__device__ __forceinline__ void scales_load(const uint8_t* const (&p)[R], int k, int kb,
                                            uint32_t (&v)[R * (PERK ? 4 : 1)]) {
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (!PERK) {
      v[i] = scale_word(p[i], k, kb);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = k + j < kb ? scale_word(p[i], 4 * (k + j), 4 * kb) : 0;
    }
  }
}

template <int R, bool PERK, class Rows>
__device__ __forceinline__ void gemm_scales(const GemmArgs& a, GemmShared& sh, uint8_t* dst,
                                            long long tiles, int nt, bool swiglu, Rows rows_of) {
  const int lane = threadIdx.x & 31;
  GemmRing ring;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const uint8_t* p[R];
    rows_of(t, p);
    uint32_t cur[R * (PERK ? 4 : 1)], next[R * (PERK ? 4 : 1)];
    scales_load<R, PERK>(p, 0, a.kb, next);
    for (int k0 = 0; k0 < a.kb; k0 += 4) {
#pragma unroll
      for (int i = 0; i < R * (PERK ? 4 : 1); ++i) cur[i] = next[i];
      if (k0 + 4 < a.kb) scales_load<R, PERK>(p, k0 + 4, a.kb, next);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (k0 + j >= a.kb) break;
        gemm_wait(&sh.empty[ring.stage], ring.phase ^ 1, sh);
        if (gemm_dead(sh)) return;
        uint4* to = reinterpret_cast<uint4*>(dst + ring.stage * (GemmShape::SFA + GemmShape::SFB));
#pragma unroll
        for (int g = 0; g < R / 4; ++g) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = PERK ? cur[(4 * g + i) * (PERK ? 4 : 1) + (PERK ? j : 0)]
                        : cur[4 * g + i] >> (8 * j) & 0xFFu;
          to[32 * g + lane] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full[ring.stage]);
        ring.next();
      }
    }
  }
}

// ---------------------------------------------------------------------------
// MMAs (warp 1, one lane)
// ---------------------------------------------------------------------------
template <bool W4>
__device__ __forceinline__ void gemm_mma(const GemmArgs& a, GemmShared& sh, uint32_t base,
                                         long long tiles) {
  using S = GemmShape;
  GemmRing ring;
  const uint32_t tm = sh.tmem;
  uint32_t n = 0, sf = 0;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x, ++n) {
    gemm_wait(&sh.acc_empty, (n & 1) ^ 1, sh);
    tc_fence_after();
    for (int k = 0; k < a.kb; ++k, ring.next(), sf ^= 1) {
      gemm_wait(&sh.full[ring.stage], ring.phase, sh);
      if (gemm_dead(sh)) return;
      tc_fence_after();
      const uint32_t at = base + ring.stage * S::STAGE;
      const uint32_t sc = base + S::SFOFF + ring.stage * (S::SFA + S::SFB);
      const uint32_t sfa = tm + S::SFCOL + 12 * sf, sfb = sfa + 4;
      umma_sf_copy(sfa, umma_desc(sc, 0, 128));
      umma_sf_copy(sfb, umma_desc(sc + S::SFA, 0, 128));
      umma_sf_copy(sfb + 4, umma_desc(sc + S::SFA + 512, 0, 128));
      const uint64_t da = umma_desc_sw128(at), db = umma_desc_sw128(at + S::ABYTES);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        umma_mxf8(tm, da + 2 * j, db + 2 * j, umma_idesc_mxf8(W4 ? 5 : 0, W4 ? j : 0, kGemmN), sfa,
                  sfb, (k | j) != 0);
      umma_commit(&sh.empty[ring.stage]);
    }
    umma_commit(&sh.acc_full);
  }
}

// ---------------------------------------------------------------------------
// Results (warps 4..7): a thread a row; 128 bytes of every row at a time go
// through shared memory, so that eight lanes write a row's piece together.
// ---------------------------------------------------------------------------
template <int SIZE>   // of an element
__device__ __forceinline__ void gemm_flush(const GemmArgs& a, const GemmTile& w, const uint8_t* stage,
                                           int col, int left) {
  // left: bytes of the 128 inside the row
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
  const int seg = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3), row = quarter * 32 + r;
    if (row >= w.rows) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * GemmShape::OUTROW + seg * 16);
    char* p = a.out + (w.row0 + row) * a.out_stride + (long long)col * SIZE + seg * 16;
    if (a.vec && seg * 16 + 16 <= left) {
      *reinterpret_cast<uint4*>(p) = v;
    } else {
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int b = 0; b < 16; b += SIZE) {
        if (seg * 16 + b + SIZE > left) continue;
        const uint32_t x = u[b / 4] >> (8 * (b % 4));
        if (SIZE == 1) *reinterpret_cast<uint8_t*>(p + b) = (uint8_t)x;
        else if (SIZE == 2) *reinterpret_cast<uint16_t*>(p + b) = (uint16_t)x;
        else *reinterpret_cast<uint32_t*>(p + b) = x;
      }
    }
  }
}

// 32 results of this thread's row to out, from column col on.
__device__ __forceinline__ void gemm_put32(const GemmArgs& a, const GemmTile& w, uint8_t* stage,
                                           int col, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  uint4* to = reinterpret_cast<uint4*>(stage + lane * GemmShape::OUTROW);
  if (a.out_dtype == MOE_DTYPE_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      to[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                         __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
    __syncwarp();
    gemm_flush<4>(a, w, stage, col, min(32, a.n - col) * 4);
  } else {
    const int f16 = a.out_dtype == MOE_DTYPE_F16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      to[i] = make_uint4(pack16(v[8 * i], v[8 * i + 1], f16), pack16(v[8 * i + 2], v[8 * i + 3], f16),
                         pack16(v[8 * i + 4], v[8 * i + 5], f16),
                         pack16(v[8 * i + 6], v[8 * i + 7], f16));
    __syncwarp();
    gemm_flush<2>(a, w, stage, col, min(32, a.n - col) * 2);
  }
  __syncwarp();
}

template <bool SWIGLU>
__device__ __forceinline__ void gemm_results(const GemmArgs& a, GemmShared& sh, uint8_t* smem,
                                             long long tiles, int nt) {
  using S = GemmShape;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
  uint8_t* stage = smem + S::OUTOFF + quarter * 32 * S::OUTROW;
  const uint32_t tm = sh.tmem + ((uint32_t)(quarter * 32) << 16);
  uint32_t n = 0;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x, ++n) {
    const GemmTile w = gemm_tile<SWIGLU>(a, sh, nt, t);
    if (!gemm_dead(sh)) gemm_wait(&sh.acc_full, n & 1, sh);
    const bool dead = gemm_dead(sh);
    tc_fence_after();
    const float nan = __int_as_float(0x7FFFFFFF);
    if (!SWIGLU) {
#pragma unroll 1
      for (int c = 0; c < kGemmN; c += 32) {
        if (w.n0 + c >= a.n) break;
        float v[32];
        tmem_ld32(tm + c, v);
        tmem_wait_ld();
        if (dead) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = nan;
        }
        gemm_put32(a, w, stage, w.n0 + c, v);
      }
      tc_fence_before();
      mbar_arrive(&sh.acc_empty);
    } else {
      float h[128];
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        float g[32], u[32];
        tmem_ld32(tm + c, g);
        tmem_ld32(tm + 128 + c, u);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          h[c + i] = dead ? nan : __fdividef(g[i], 1.f + __expf(-g[i])) * u[i];
      }
      tc_fence_before();
      mbar_arrive(&sh.acc_empty);
      if (a.out_dtype == MOE_DTYPE_E4M3) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (w.n0 + i < a.n) amax = fp8_finite_max(amax, h[i]);
        const int e = fp8_block_exp(amax), row = quarter * 32 + lane;
        const float inv = pow2f(-e);
        uint2* to = reinterpret_cast<uint2*>(stage + lane * S::OUTROW);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float x[8] = {h[8 * i],     h[8 * i + 1], h[8 * i + 2], h[8 * i + 3],
                              h[8 * i + 4], h[8 * i + 5], h[8 * i + 6], h[8 * i + 7]};
          to[i] = fp8_codes8(x, inv);
        }
        __syncwarp();
        gemm_flush<1>(a, w, stage, w.n0, min(128, a.n - w.n0));
        __syncwarp();
        if (row < w.rows) a.os[(w.row0 + row) * a.os_stride + (w.n0 >> 7)] = (uint8_t)(e + 127);
      } else {
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          if (w.n0 + c >= a.n) break;
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = h[c + i];
          gemm_put32(a, w, stage, w.n0 + c, v);
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
  const uint32_t base = smem_addr(smem);
  const int warp = threadIdx.x >> 5;
  gemm_prefix(a, sh);
  const int nt = (a.n + (SWIGLU ? kGemmN / 2 : kGemmN) - 1) / (SWIGLU ? kGemmN / 2 : kGemmN);
  const long long tiles = (long long)sh.tiles[a.experts] * nt;
  if (blockIdx.x >= tiles) return;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kGemmStages; ++s) {
      mbar_init(&sh.full[s], 3);    // the copies' bytes, two warps' scales
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.acc_full, 1);
    mbar_init(&sh.acc_empty, 128);
    mbar_init(&sh.drained, 1);
    sh.dead = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&sh.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == 0) {
    gemm_copy<W4, SWIGLU>(a, sh, base, &xt, &xg, &wm, tiles, nt);
  } else if (warp == 1) {
    if ((threadIdx.x & 31) == 0) gemm_mma<W4>(a, sh, base, tiles);
  } else if (warp == 2) {
    gemm_scales<4, false>(a, sh, smem + S::SFOFF, tiles, nt, SWIGLU,
                          [&](long long t, const uint8_t* (&p)[4]) {
                            const GemmTile w = gemm_tile<SWIGLU>(a, sh, nt, t);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                              p[i] = a.xs + gemm_source(a, w, (threadIdx.x & 31) + 32 * i) *
                                                a.xs_stride;
                          });
  } else if (warp == 3) {
    gemm_scales<8, W4>(a, sh, smem + S::SFOFF + S::SFA, tiles, nt, SWIGLU,
                       [&](long long t, const uint8_t* (&p)[8]) {
                         const GemmTile w = gemm_tile<SWIGLU>(a, sh, nt, t);
#pragma unroll
                         for (int i = 0; i < 8; ++i) {
                           int r = w.n0 + (threadIdx.x & 31) + 32 * i;
                           if (SWIGLU && i >= 4) r += a.n - kGemmN / 2;
                           r = min(r, a.wide - 1);
                           p[i] = a.ws + w.expert * a.ws_expert + (W4 ? r : r >> 7) * a.ws_stride;
                         }
                       });
  } else {
    gemm_results<SWIGLU>(a, sh, smem, tiles, nt);
  }
  __syncwarp();
  if (gemm_dead(sh) && warp == 1) {   // products in flight likewise
    if ((threadIdx.x & 31) == 0) {
      umma_commit(&sh.drained);
      for (int i = 0; i < 100 && !mbar_try_wait_long(&sh.drained, 0); ++i) {
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(sh.tmem);
  }
}

}  // namespace moe
