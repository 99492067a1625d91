// Rows to their 8-bit form, with or without the norm in front; weights to theirs.
//
// One pass: a row is held in registers between its sum of squares and its
// outputs, 8 elements (16 bytes of bf16) at a time, so that x and the residual
// are read once.  HBM bounds long calls, the launch short ones.  A scale's 128
// columns are 16 neighbouring lanes' elements: its maximum takes four shuffles.
// Measured on the device: 8,192 rows of 7,168 with a residual and both outputs 79 us,
// 6.7 TB/s; one row 3.5 us.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "kv_cache.cuh"
#include "moe_decode.h"

namespace moe {

// Scale exponents of 8-bit activations and weights: 2^-e and 2^e are normal
// fp32 numbers for all of them, and 448 * 2^120 is above every finite one.
constexpr int kFp8ExpMin = -126;

// Smallest e >= kFp8ExpMin with amax <= 448 * 2^e (448 = 1.75 * 2^8), for finite
// amax >= 0.
__device__ __forceinline__ int fp8_block_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, kFp8ExpMin);
}

__device__ __forceinline__ float fp8_finite_max(float amax, float v) {
  const float a = fabsf(v);
  return a <= 3.4028235e38f ? fmaxf(amax, a) : amax;
}

__device__ __forceinline__ uint2 fp8_codes8(const float (&v)[8], float inv) {
  return make_uint2(f32x2_to_e4m3x2(v[0] * inv, v[1] * inv) |
                        f32x2_to_e4m3x2(v[2] * inv, v[3] * inv) << 16,
                    f32x2_to_e4m3x2(v[4] * inv, v[5] * inv) |
                        f32x2_to_e4m3x2(v[6] * inv, v[7] * inv) << 16);
}

// Eight elements of a tensor of `dtype` (16-byte aligned), as they lie.
template <bool F32>
struct Raw8 {
  uint4 a[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw8(const void* p, int64_t at) {
  Raw8<F32> r;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (F32 ? 4 : 2));
  r.a[0] = q[0];
  if (F32) r.a[F32 ? 1 : 0] = q[1];
  return r;
}
template <bool F32>
__device__ __forceinline__ void raw8_to_float(const Raw8<F32>& r, int f16, float (&v)[8]) {
  if (F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = r.a[F32 ? i : 0];
      v[4 * i] = __uint_as_float(u.x);
      v[4 * i + 1] = __uint_as_float(u.y);
      v[4 * i + 2] = __uint_as_float(u.z);
      v[4 * i + 3] = __uint_as_float(u.w);
    }
  } else {
    const uint32_t u[4] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16(u[i], f16);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t at, int f16, const float (&v)[8]) {
  uint4* q = reinterpret_cast<uint4*>(static_cast<char*>(p) + at * (F32 ? 4 : 2));
  if (F32) {
    q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
    q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                      __float_as_uint(v[7]));
  } else {
    q[0] = make_uint4(pack16(v[0], v[1], f16), pack16(v[2], v[3], f16), pack16(v[4], v[5], f16),
                      pack16(v[6], v[7], f16));
  }
}

struct NormArgs {
  const void* x;
  long long xs;
  void* res;          // or null
  long long rs;
  const void* gamma;  // null: no norm
  void* out;          // or null
  long long os;
  uint8_t* codes;     // or null
  long long cs;
  uint8_t* scales;
  long long ss;
  long long rows;
  int d, f16, gamma_dtype;
  float eps;
};

__device__ __forceinline__ void load_gamma8(const void* g, int dtype, int at, float (&v)[8]) {
  if (dtype == MOE_DTYPE_F32) raw8_to_float<true>(load_raw8<true>(g, at), 0, v);
  else raw8_to_float<false>(load_raw8<false>(g, at), dtype == MOE_DTYPE_F16, v);
}

// T threads a row (a power of two, 32 at least), each with NV times 8 elements;
// blockDim.x / T rows a CTA.
template <int T, int NV, bool F32, bool NORM>
static __global__ void __launch_bounds__(T < 256 ? 256 : T)
    rms_norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int THREADS = T < 256 ? 256 : T, ROWS = THREADS / T, WARPS = T / 32;
  __shared__ float s_sum[THREADS / 32];
  pdl_wait_prerequisites();
  pdl_launch_dependents();
  const int t = threadIdx.x % T, sub = threadIdx.x / T;
  const long long row = (long long)blockIdx.x * ROWS + sub;
  const bool there = row < a.rows;
  Raw8<F32> rx[NV], rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (i * T + t);
    if (there && c < a.d) rx[i] = load_raw8<F32>(a.x, row * a.xs + c);
  }
  if (NORM && a.res) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * T + t);
      if (there && c < a.d) rr[i] = load_raw8<F32>(a.res, row * a.rs + c);
    }
  }
  float v[NV][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (i * T + t);
    if (there && c < a.d) {
      raw8_to_float<F32>(rx[i], a.f16, v[i]);
      if (NORM && a.res) {
        float r[8];
        raw8_to_float<F32>(rr[i], a.f16, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += r[j];
        store8<F32>(a.res, row * a.rs + c, a.f16, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
  if (NORM) {
    auto row_sum = [&](float s) {
      s = warp_sum(s);
      if (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = s;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "n"(T) : "memory");
        s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += s_sum[sub * WARPS + w];
      }
      return s;
    };
    sum = row_sum(sum);
    float eps = a.eps, last = 1.f;
    // squares past fp32's range, or (with little or no eps) so near its lower end that
    // they lose bits: once more from values times f, a power of two.  Then values enter
    // times f, large ones by its square root and their norm by the other one (neither
    // leaves the range)
    const float all = fmaf((float)a.d, eps, sum);
    if (__builtin_expect(!(all >= 0x1p-100f && sum <= 3.4028235e38f), 0)) {
      const bool high = !(sum <= 3.4028235e38f);
      const float f = high ? 0x1p-80f : 0x1p100f, first = high ? 0x1p-40f : f;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = v[i][j] * f;
          sum = fmaf(u, u, sum);
          v[i][j] *= first;
        }
      // (s_sum has been read)
      if (WARPS > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "n"(T) : "memory");
      sum = row_sum(sum);
      eps = eps * f * f;
      if (high) last = 0x1p-40f;
    }
    const float scale = last / sqrtf(sum / (float)a.d + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = 8 * (i * T + t);
      if (c >= a.d) continue;
      float g[8];
      load_gamma8(a.gamma, a.gamma_dtype, c, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * scale * g[j];
      if (there && a.out) store8<F32>(a.out, row * a.os + c, a.f16, v[i]);
    }
  }
  if (!a.codes) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = 8 * (i * T + t);
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fp8_finite_max(amax, v[i][j]);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (there && c < a.d) {
      const int e = fp8_block_exp(amax);
      *reinterpret_cast<uint2*>(a.codes + row * a.cs + c) = fp8_codes8(v[i], pow2f(-e));
      if ((t & 15) == 0) a.scales[row * a.ss + (c >> 7)] = (uint8_t)(e + 127);
    }
  }
}

// Weights: a CTA of 256 threads per 128 x 128, whose elements are read singly (k
// may be odd) and twice, the second time out of the caches.  A one-time layout: 16
// matrices of 4,096 x 7,168 bf16 1.74 ms, 0.81 TB/s.
template <int DTYPE>
__device__ __forceinline__ float pack_element(const void* w, long long at) {
  if (DTYPE == MOE_DTYPE_F32) return static_cast<const float*>(w)[at];
  const uint32_t u = static_cast<const uint16_t*>(w)[at];
  return unpack16(u, DTYPE == MOE_DTYPE_F16).x;
}

template <int DTYPE>
static __global__ void __launch_bounds__(256)
    fp8_pack_kernel(const void* w, long long n, long long k, uint8_t* codes, uint8_t* scales) {
  __shared__ float s_max[8];
  const long long nb = (n + 127) / 128, kb = (k + 127) / 128;
  const long long mat = blockIdx.x / (nb * kb), at = blockIdx.x % (nb * kb);
  const long long r0 = at / kb * 128, c0 = at % kb * 128, base = mat * n * k;
  const int col = threadIdx.x & 127, sub = threadIdx.x >> 7;
  const long long c = c0 + col;
  float amax = 0.f;
#pragma unroll 8
  for (int i = sub; i < 128; i += 2)
    if (r0 + i < n && c < k)
      amax = fp8_finite_max(amax, pack_element<DTYPE>(w, base + (r0 + i) * k + c));
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, s_max[i]);
  const int e = fp8_block_exp(amax);
  const float inv = pow2f(-e);
#pragma unroll 8
  for (int i = sub; i < 128; i += 2) {
    const long long at = base + (r0 + i) * k + c;
    if (r0 + i < n && c < k)
      codes[at] = (uint8_t)f32x2_to_e4m3x2(pack_element<DTYPE>(w, at) * inv, 0.f);
  }
  if (threadIdx.x == 0) scales[mat * nb * kb + at] = (uint8_t)(e + 127);
}

}  // namespace moe
