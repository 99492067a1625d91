// New keys and values into the 8-bit cache.
//
// The tokens a step writes into one block share its scale, so the unit of
// work is a group: the consecutive tokens of one block, found at its first
// token (the leader: the slot before it lies in another block).  Tokens that
// are skipped may stand between those of a block: a path of its own.  Of a group of
// one head and one side: the largest magnitude, the exponent, then the codes;
// where the block held tokens and its exponent grows, their codes are rounded
// to the new scale first.
// HBM would bound long calls (2 bytes read, 1 written an element); issue slots do
// (73% busy).  Latency bounds short ones.  A CTA looks after the leaders among `chunk` slots: many (a decode
// batch, a token each) go a warp each; few (a prompt, whole blocks) one after
// the other to all eight warps, which hold a group's values in registers
// between the maximum and the codes, so that they are read once.  Measured: 16
// prompts of 517 to 1,531 tokens, 8 heads of 128, blocks of 64: 33.5 us, 3.0 TB/s
// (74 us with a warp a group; five CTAs an SM hide each other's chain of slot,
// values, maximum and codes, with two 55 us).  64 rows' one token each: 7.5 us,
// the host's time for the call.
#pragma once

#include "kv_cache.cuh"

namespace moe {

constexpr int kAppendWarps = 8;
constexpr int kAppendThreads = 32 * kAppendWarps;
constexpr int kAppendCtas = 5;  // an SM
constexpr int kAppendFew = 4;   // leaders of a CTA up to which all warps share each

struct AppendArgs {
  KvView c;
  const uint16_t* src[2];
  long long ts[2], hs[2];   // elements
  int f16;
  const int* slot;
  int n_tokens, chunk;      // chunk: 8 or 64 slots a CTA
};

__device__ __forceinline__ int append_block_of(const AppendArgs& a, int slot) {
  return slot >= 0 && (slot >> a.c.bs_log2) < a.c.n_blocks ? slot >> a.c.bs_log2 : -1;
}

// Largest finite magnitude of 8 elements and `amax`.
__device__ __forceinline__ float append_max(const uint4& w, int f16, float amax) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack16(u[j], f16);
    const float x = fabsf(f.x), y = fabsf(f.y);
    if (x <= 3.4028235e38f) amax = fmaxf(amax, x);
    if (y <= 3.4028235e38f) amax = fmaxf(amax, y);
  }
  return amax;
}
// Codes of 8 elements times inv.
__device__ __forceinline__ uint2 append_codes(const uint4& w, int f16, float inv) {
  const float2 f0 = unpack16(w.x, f16), f1 = unpack16(w.y, f16), f2 = unpack16(w.z, f16),
               f3 = unpack16(w.w, f16);
  return make_uint2(f32x2_to_e4m3x2(f0.x * inv, f0.y * inv) |
                        f32x2_to_e4m3x2(f1.x * inv, f1.y * inv) << 16,
                    f32x2_to_e4m3x2(f2.x * inv, f2.y * inv) |
                        f32x2_to_e4m3x2(f3.x * inv, f3.y * inv) << 16);
}

// The codes of tokens [sub, sub + step, ..) below off, LPT threads a token, to
// an exponent that is `down` higher.
__device__ __forceinline__ void append_round_again(uint8_t* dst, long long tstride, int sub,
                                                   int step, int off, float down) {
  for (int i = sub; i < off; i += step) {
    uint2* p = reinterpret_cast<uint2*>(dst + i * tstride);
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

// Tokens [t0, t0 + n) of head h, side s (0 K, 1 V) into block b from offset
// off, by one warp (THREADS 32) or the whole CTA.
template <int D, int THREADS>
__device__ __forceinline__ void append_group(const AppendArgs& a, int s, int h, int b, int off,
                                             int t0, int n) {
  constexpr int LPT = D / 8;             // threads a token (8 elements each)
  constexpr int TPP = THREADS / LPT;     // tokens a pass
  constexpr int HELD = THREADS == 32 ? 2 : 64 / TPP;   // passes kept in registers
  __shared__ float s_max[kAppendWarps];
  const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int sub = tid / LPT, part = tid % LPT;
  const uint16_t* src = a.src[s] + t0 * a.ts[s] + h * a.hs[s] + part * 8;
  uint8_t* dst = (s ? a.c.v : a.c.k) + b * a.c.bstride + h * a.c.hstride + part * 8;
  uint8_t* sp = (s ? a.c.vs : a.c.ks) + b * a.c.sstride + h;
  const int old = off > 0 ? kv_exp(*sp) : kKvExpMin;
  uint4 held[HELD];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const int i = sub + k * TPP;
    if (i < n) held[k] = __ldg(reinterpret_cast<const uint4*>(src + i * a.ts[s]));
  }
#pragma unroll
  for (int k = 0; k < HELD; ++k)
    if (sub + k * TPP < n) amax = append_max(held[k], a.f16, amax);
  for (int i = sub + HELD * TPP; i < n; i += TPP)
    amax = append_max(__ldg(reinterpret_cast<const uint4*>(src + i * a.ts[s])), a.f16, amax);
  amax = warp_max(amax);
  if (THREADS > 32) {
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendWarps; ++w) amax = fmaxf(amax, s_max[w]);
    __syncthreads();   // (and every thread has read the old scale)
  } else {
    __syncwarp();
  }
  const int e = max(kv_block_exp(amax), old);
  if (off > 0 && old < e) {
    const float down = pow2f(old - e);
    for (int i = sub; i < off; i += TPP) {
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
  if (tid == 0) *sp = (uint8_t)(e + 127);
  const float inv = pow2f(-e);
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const int i = sub + k * TPP;
    if (i < n)
      *reinterpret_cast<uint2*>(dst + (off + i) * a.c.tstride) =
          append_codes(held[k], a.f16, inv);
  }
  for (int i = sub + HELD * TPP; i < n; i += TPP)
    *reinterpret_cast<uint2*>(dst + (off + i) * a.c.tstride) = append_codes(
        __ldg(reinterpret_cast<const uint4*>(src + i * a.ts[s])), a.f16, inv);
}

// The block of the last token before t that is not skipped, less than a block's
// tokens away; -1: none.
__device__ __forceinline__ int append_block_before(const AppendArgs& a, int t) {
  const int far = min((1 << a.c.bs_log2) - 1, t);
  int b = -1;
  for (int j = 1; j <= far && b < 0; ++j) b = append_block_of(a, __ldg(a.slot + t - j));
  return b;
}

// Groups with skipped tokens among or beside them, a warp each, values read
// twice: rare, so its code and registers stay out of the others'.  Those of the
// chunk whose leaders are in `own`, or (own all ones) dealt round the warps.  A
// group's tokens lie in as many entries of the slot map as a block has tokens.
template <int D>
__device__ __noinline__ void append_sparse(const AppendArgs& a, unsigned long long own) {
  constexpr int LPT = D / 8, TPP = 32 / LPT;
  const int lane = threadIdx.x & 31, sub = lane / LPT, part = lane % LPT;
  const int h = blockIdx.y >> 1, s = blockIdx.y & 1, c0 = blockIdx.x * a.chunk;
  unsigned long long leaders = 0;
  for (int k = 0; k < a.chunk; k += 32) {
    int b = -1;
    if (k + lane < min(a.chunk, a.n_tokens - c0)) b = append_block_of(a, __ldg(a.slot + c0 + k + lane));
    const bool leads = b >= 0 && b != append_block_before(a, c0 + k + lane);
    leaders |= (unsigned long long)__ballot_sync(0xffffffffu, leads) << k;
  }
  for (int k = 0; leaders; ++k, leaders &= leaders - 1) {
    if (own == ~0ull ? k % kAppendWarps != (int)(threadIdx.x >> 5) : !(own & leaders & -leaders)) continue;
    const int t0 = c0 + __ffsll((long long)leaders) - 1, first = __ldg(a.slot + t0);
    const int b = first >> a.c.bs_log2, mask = (1 << a.c.bs_log2) - 1, off = first & mask;
    const int n = min(mask + 1, a.n_tokens - t0);
    const uint16_t* src = a.src[s] + t0 * a.ts[s] + h * a.hs[s] + part * 8;
    uint8_t* dst = (s ? a.c.v : a.c.k) + b * a.c.bstride + h * a.c.hstride + part * 8;
    uint8_t* sp = (s ? a.c.vs : a.c.ks) + b * a.c.sstride + h;
    const int old = off > 0 ? kv_exp(*sp) : kKvExpMin;
    float amax = 0.f;
    for (int i = sub; i < n; i += TPP)
      if (append_block_of(a, __ldg(a.slot + t0 + i)) == b)
        amax = append_max(__ldg(reinterpret_cast<const uint4*>(src + i * a.ts[s])), a.f16, amax);
    amax = warp_max(amax);
    __syncwarp();
    const int e = max(kv_block_exp(amax), old);
    if (off > 0 && old < e) append_round_again(dst, a.c.tstride, sub, TPP, off, pow2f(old - e));
    if (lane == 0) *sp = (uint8_t)(e + 127);
    const float inv = pow2f(-e);
    for (int i = sub; i < n; i += TPP) {
      const int slot = __ldg(a.slot + t0 + i);
      if (append_block_of(a, slot) == b)
        *reinterpret_cast<uint2*>(dst + (slot & mask) * a.c.tstride) = append_codes(
            __ldg(reinterpret_cast<const uint4*>(src + i * a.ts[s])), a.f16, inv);
    }
    __syncwarp();
  }
}

template <int D>
static __global__ void __launch_bounds__(kAppendThreads, kAppendCtas) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * a.chunk;
  const int h = blockIdx.y >> 1, s = blockIdx.y & 1;
  const int mask = (1 << a.c.bs_log2) - 1;
  // leaders among this chunk's slots (every warp finds them for itself), and
  // where the slot after each lane's begins another block
  unsigned long long leaders = 0, ends = 0;
  bool beside = false;   // a skipped token
  for (int k = 0; k < a.chunk; k += 32) {
    int b = -1, prev = -1, next = -1;
    if (k + lane < min(a.chunk, a.n_tokens - c0)) {
      const int t = c0 + k + lane;
      b = append_block_of(a, __ldg(a.slot + t));
      if (t > 0) prev = append_block_of(a, __ldg(a.slot + t - 1));
      if (t < a.n_tokens - 1) next = append_block_of(a, __ldg(a.slot + t + 1));
    }
    leaders |= (unsigned long long)__ballot_sync(0xffffffffu, b >= 0 && b != prev) << k;
    ends |= (unsigned long long)__ballot_sync(0xffffffffu, b != next) << k;
    beside |= b >= 0 && ((prev < 0 && c0 + k + lane > 0) || (next < 0 && c0 + k + lane < a.n_tokens - 1));
  }
  if (__any_sync(0xffffffffu, beside)) {
    append_sparse<D>(a, ~0ull);
    return;
  }
  unsigned long long sparse = 0;   // groups that meet one past the chunk, a warp each
  const bool few = __popcll(leaders) <= kAppendFew;
  for (int k = 0; leaders; ++k, leaders &= leaders - 1) {
    if (!few && k % kAppendWarps != warp) continue;
    const int l = __ffsll((long long)leaders) - 1;
    const int t0 = c0 + l, slot = __ldg(a.slot + t0);
    const int b = slot >> a.c.bs_log2, off = slot & mask;
    // the group's length: to the first end, past the chunk by looking on
    const int room = min(mask + 1 - off, a.n_tokens - t0);
    const unsigned long long e = ends >> l;
    int n = min(a.chunk - l, room);
    if (e) {
      n = min(__ffsll((long long)e), room);
    } else {
      for (unsigned m = ~0u; m == ~0u;) {
        const int i = n + lane;
        const int at = i <= room && i < a.n_tokens - t0 ? append_block_of(a, __ldg(a.slot + t0 + i)) : b;
        m = __ballot_sync(0xffffffffu, at == b && i < room);
        const unsigned skipped = __ballot_sync(0xffffffffu, at < 0);
        const int in = m == ~0u ? 32 : __ffs(~m) - 1;
        n += in;
        if (in < 32 && ((skipped >> in) & 1u)) n = 0;
      }
      if (n == 0) {
        if (k % kAppendWarps == warp) sparse |= leaders & -leaders;
        continue;
      }
    }
    if (few) append_group<D, kAppendThreads>(a, s, h, b, off, t0, n);
    else append_group<D, 32>(a, s, h, b, off, t0, n);
  }
  if (sparse) append_sparse<D>(a, sparse);
}

}  // namespace moe
