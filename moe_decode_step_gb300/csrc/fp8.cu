// C ABI of the 8-bit products, norms and the experts of any number of rows.
#include <cuda.h>

#include "fp8_product.cuh"
#include "fp8_rows.cuh"
#include "host.cuh"
#include "moe_decode.h"
#include "moe_rows.cuh"

using namespace moe;

namespace {

// A launch that may begin while the one before it in the stream ends: every kernel
// here waits for that before it touches memory (decode steps are chains of such
// calls, whose starts take as long as their work).  cluster: CTAs of one.
template <class... Args>
int launch(void (*kernel)(Args...), unsigned grid_x, unsigned grid_y, int threads, int smem,
           int cluster, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid_x, grid_y);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_fail(e);
  }
  return end();
}

// Rows that are written lie apart.
bool overlap(long long rows, int64_t stride, int64_t d) { return rows > 1 && stride < d; }

bool dtype16or32(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F16 || t == MOE_DTYPE_F32; }

template <int T, int NV>
int launch_norm(const NormArgs& a, bool f32, cudaStream_t st) {
  constexpr int THREADS = T < 256 ? 256 : T, ROWS = THREADS / T;
  const unsigned grid = (unsigned)((a.rows + ROWS - 1) / ROWS);
  void (*kernel)(NormArgs) =
      a.gamma ? (f32 ? rms_norm_kernel<T, NV, true, true> : rms_norm_kernel<T, NV, false, true>)
              : (f32 ? rms_norm_kernel<T, NV, true, false> : rms_norm_kernel<T, NV, false, false>);
  return launch(kernel, grid, 1, THREADS, 0, 1, st, a);
}

int run_norm(const NormArgs& a, int dtype, void* stream) {
  if (a.rows == 0) return MOE_OK;
  if (a.rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  const int rc = begin(&dev);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = dtype == MOE_DTYPE_F32;
  if (a.d <= 1024) return launch_norm<32, 4>(a, f32, st);
  if (a.d <= 4096) return launch_norm<128, 4>(a, f32, st);
  if (a.d <= 8192) return launch_norm<256, 4>(a, f32, st);
  return launch_norm<512, 4>(a, f32, st);
}

// Tensor map of bytes (or of E2M1 nibbles that become 16 bytes each 16) with
// 128-byte-swizzled boxes of 128 columns.
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

int encoder(Encode* out) {
  static std::atomic<void*> known{nullptr};   // a symbol of the driver: the same for every caller
  void* fn = known.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn) {
      cudaGetLastError();
      return MOE_ERR_UNSUPPORTED;
    }
    known.store(fn, std::memory_order_release);
  }
  *out = reinterpret_cast<Encode>(fn);
  return MOE_OK;
}

int encode_map(Encode fn, CUtensorMap* map, bool nibbles, const void* p, int rank,
               const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(map, nibbles ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B
                                     : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                        rank, const_cast<void*>(p), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_UNSUPPORTED;
}
// Boxes of one block of 128 columns (zeros past their end), or of two: of K in whole
// blocks, the block a dimension of its own.
int encode_rows(Encode fn, CUtensorMap* map, const moe_fp8_product_t& t, int per, int box_rows) {
  const cuuint64_t k = t.k, rows = t.x_rows, row = t.x_stride;
  if (per == 2) {
    const cuuint64_t dims[3] = {kGemmK, rows, k / kGemmK}, strides[2] = {row, kGemmK};
    const cuuint32_t box[3] = {kGemmK, (cuuint32_t)box_rows, 2};
    return encode_map(fn, map, false, t.x, 3, dims, strides, box);
  }
  const cuuint64_t dims[2] = {k, rows}, strides[1] = {row};
  const cuuint32_t box[2] = {kGemmK, (cuuint32_t)box_rows};
  return encode_map(fn, map, false, t.x, 2, dims, strides, box);
}
int encode_weights(Encode fn, CUtensorMap* map, const moe_fp8_product_t& t, int per, bool swiglu) {
  const bool w4 = t.w_format == MOE_WEIGHTS_MXFP4;
  const cuuint64_t k = t.k, n = swiglu ? t.n / 2 : t.n, e = t.n_experts, row = t.w_stride;
  const cuuint64_t mat = e > 1 ? (cuuint64_t)t.w_expert_stride : row * t.n;
  const cuuint32_t rows = swiglu ? kGemmRows / 2 : kGemmRows, sides = swiglu ? 2 : 1;
  if (per == 2) {
    const cuuint64_t dims[5] = {kGemmK, n, sides, k / kGemmK, e};
    const cuuint64_t strides[4] = {row, row * n, (cuuint64_t)(w4 ? kGemmK / 2 : kGemmK), mat};
    const cuuint32_t box[5] = {kGemmK, rows, sides, 2, 1};
    return encode_map(fn, map, w4, t.w, 5, dims, strides, box);
  }
  if (swiglu) {
    const cuuint64_t dims[4] = {k, n, sides, e}, strides[3] = {row, row * n, mat};
    const cuuint32_t box[4] = {kGemmK, rows, sides, 1};
    return encode_map(fn, map, w4, t.w, 4, dims, strides, box);
  }
  const cuuint64_t dims[3] = {k, n, e}, strides[2] = {row, mat};
  const cuuint32_t box[3] = {kGemmK, rows, 1};
  return encode_map(fn, map, w4, t.w, 3, dims, strides, box);
}

// Token tiles and weight tiles of a call at most, as far as the host knows.
long long tiles_at_most(const GemmArgs& a, bool swiglu) {
  const int cols = swiglu ? kGemmRows : 2 * kGemmRows;
  const long long m = a.offsets ? (long long)a.rows / a.tokens + std::min(a.experts, a.rows)
                                : ((long long)a.rows + a.tokens - 1) / a.tokens;
  return m * ((a.n + cols - 1) / cols);
}

// Clusters of `ctas` CTAs of the product kernel (each has an SM to itself) that the
// current device holds at once: fewer than its SMs would make, where a GPC's are no
// multiple of `ctas` (of 152, 36 of four and 15 of eight).  Asked for once per device.
int clusters_at_once(int ctas, int* out) {
  static std::atomic<int> known[kMaxDevices][4];   // by log2(ctas), one more than they are
  int dev = 0, at = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  while (2 << at <= ctas) ++at;
  int n = known[dev][at].load(std::memory_order_relaxed);
  if (!n) {
    void (*kernel)(GemmArgs, GemmMaps) = fp8_product_kernel<false, false, 1>;
    cudaLaunchAttribute of{};
    of.id = cudaLaunchAttributeClusterDimension;
    of.val.clusterDim.x = ctas;
    of.val.clusterDim.y = of.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = GemmShape::LIMIT;
    cfg.attrs = &of;
    cfg.numAttrs = 1;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  GemmShape::LIMIT)) ||
        (e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg))) {
      cudaGetLastError();
      return cuda_fail(e);
    }
    known[dev][at].store(++n, std::memory_order_relaxed);   // (alike in every thread)
  }
  *out = n - 1;
  return MOE_OK;
}

// moe_debug_set_product_fault's
std::atomic<int> product_fault{0};
std::atomic<unsigned long long> product_wait_ns{0};

template <bool W4, bool SWIGLU, int PER>
int launch_product(GemmArgs a, const GemmMaps& maps, int n_sm, cudaStream_t st) {
  a.stages = GemmShape::stages(a.tokens, PER);
  const int smem = GemmShape::smem(a.tokens, PER);
  // (the most any call asks for: calls of other threads may come between)
  const cudaError_t e = cudaFuncSetAttribute(fp8_product_kernel<W4, SWIGLU, PER>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             GemmShape::LIMIT);
  if (e != cudaSuccess) return cuda_fail(e);
  const long long tiles = tiles_at_most(a, SWIGLU);
  if (tiles > INT32_MAX - 65536) return MOE_ERR_UNSUPPORTED;
  const int pairs = n_sm / 2, groups = (a.kb + 3) / 4;
  a.fault = product_fault.load(std::memory_order_relaxed);
  a.wait_ns = a.fault ? product_wait_ns.load(std::memory_order_relaxed) : 0;
  if (!a.wait_ns) a.wait_ns = kWaitLimitNs;
  a.splits = 1;
  while (a.splits < kGemmMaxSplits && 2 * a.splits * tiles <= pairs && 2 * a.splits <= groups) {
    // (a cluster more than fit takes the call twice as long: one row times 4,096 x
    // 4,096, 16 tiles, by four pairs each 16.3 us, by two 9.5)
    int fit;
    const int rc = clusters_at_once(4 * a.splits, &fit);
    if (rc) return rc;
    if (tiles > fit) break;
    a.splits *= 2;
  }
  const int grid = 2 * a.splits * (int)std::min<long long>(pairs / a.splits, tiles);
  return launch(fp8_product_kernel<W4, SWIGLU, PER>, grid, 1, kGemmThreads, smem, 2 * a.splits, st,
                a, maps);
}

template <int WARPS, int ITER>
int launch_dispatch(const DispatchArgs& a, int ctas, int clusters, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(dispatch_kernel<WARPS, ITER>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       disp_smem<WARPS, ITER>(kDispMaxExperts));
  if (e == cudaSuccess && ctas > 8)
    e = cudaFuncSetAttribute(dispatch_kernel<WARPS, ITER>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return cuda_fail(e);
  return launch(dispatch_kernel<WARPS, ITER>, ctas * clusters, 1, kDispThreads,
                disp_smem<WARPS, ITER>(a.experts), ctas, st, a);
}

}  // namespace

extern "C" {

int moe_rms_norm(void* stream, const moe_rms_norm_t* args) {
  if (!args) return MOE_ERR_INVALID_ARG;
  const moe_rms_norm_t& t = *args;
  if (t.n_rows < 0 || t.d < 1 || !dtype16or32(t.dtype) || !dtype16or32(t.gamma_dtype) ||
      !(t.eps >= 0.f))
    return MOE_ERR_INVALID_ARG;
  if (t.n_rows == 0) return MOE_OK;
  if (!t.x || !t.gamma || (!t.out && !t.codes) || !t.codes != !t.scales ||
      (t.residual && overlap(t.n_rows, t.residual_stride, t.d)) ||
      (t.out && overlap(t.n_rows, t.out_stride, t.d)) ||
      (t.codes && (overlap(t.n_rows, t.codes_stride, t.d) ||
                   overlap(t.n_rows, t.scales_stride, (t.d + 127) / 128))))
    return MOE_ERR_INVALID_ARG;
  if (t.d % 8 || t.d > 16384 || misaligned(t.x, 16) || misaligned(t.residual, 16) ||
      misaligned(t.gamma, 16) || misaligned(t.out, 16) || misaligned(t.codes, 8) ||
      ((t.x_stride | (t.residual ? t.residual_stride : 0) | (t.out ? t.out_stride : 0) |
        (t.codes ? t.codes_stride : 0)) & 7))
    return MOE_ERR_UNSUPPORTED;
  NormArgs a{t.x,     t.x_stride,     t.residual, t.residual_stride, t.gamma,  t.out, t.out_stride,
             t.codes, t.codes_stride, t.scales,   t.scales_stride,   t.n_rows, t.d,
             t.dtype == MOE_DTYPE_F16, t.gamma_dtype, t.eps};
  return run_norm(a, t.dtype, stream);
}

int moe_fp8_quantize(void* stream, const void* x, int dtype, int64_t x_stride, int64_t n_rows,
                     int d, uint8_t* codes, int64_t codes_stride, uint8_t* scales,
                     int64_t scales_stride) {
  if (n_rows < 0 || d < 1 || !dtype16or32(dtype)) return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  if (!x || !codes || !scales || overlap(n_rows, codes_stride, d) ||
      overlap(n_rows, scales_stride, (d + 127) / 128))
    return MOE_ERR_INVALID_ARG;
  if (d % 8 || d > 16384 || misaligned(x, 16) || misaligned(codes, 8) ||
      ((x_stride | codes_stride) & 7))
    return MOE_ERR_UNSUPPORTED;
  NormArgs a{};
  a.x = x;
  a.xs = x_stride;
  a.codes = codes;
  a.cs = codes_stride;
  a.scales = scales;
  a.ss = scales_stride;
  a.rows = n_rows;
  a.d = d;
  a.f16 = dtype == MOE_DTYPE_F16;
  return run_norm(a, dtype, stream);
}

int moe_fp8_pack(void* stream, const void* w, int dtype, int64_t n_mat, int64_t n, int64_t k,
                 uint8_t* codes, uint8_t* scales) {
  if (n_mat < 0 || n < 1 || k < 1 || !dtype16or32(dtype)) return MOE_ERR_INVALID_ARG;
  if (n_mat == 0) return MOE_OK;
  if (!w || !codes || !scales) return MOE_ERR_INVALID_ARG;
  if (n > INT32_MAX || k > INT32_MAX || n_mat > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const long long blocks = (n + 127) / 128 * ((k + 127) / 128);
  if (blocks > INT32_MAX / n_mat || misaligned(w, dtype == MOE_DTYPE_F32 ? 4 : 2))
    return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  const int rc = begin(&dev);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)(blocks * n_mat);
  auto kernel = dtype == MOE_DTYPE_F32   ? fp8_pack_kernel<MOE_DTYPE_F32>
                : dtype == MOE_DTYPE_F16 ? fp8_pack_kernel<MOE_DTYPE_F16>
                                         : fp8_pack_kernel<MOE_DTYPE_BF16>;
  kernel<<<grid, 256, 0, st>>>(w, n, k, codes, scales);
  return end();
}

int moe_fp8_product(void* stream, const moe_fp8_product_t* args) {
  if (!args) return MOE_ERR_INVALID_ARG;
  const moe_fp8_product_t& t = *args;
  const bool w4 = t.w_format == MOE_WEIGHTS_MXFP4, swiglu = t.activation == MOE_ACT_SWIGLU;
  const bool codes = t.out_dtype == MOE_DTYPE_E4M3;
  if ((!w4 && t.w_format != MOE_WEIGHTS_E4M3) || (!swiglu && t.activation != MOE_ACT_NONE) ||
      (!codes && !dtype16or32(t.out_dtype)) || t.n_rows < 0 || t.x_rows < 0 || t.n < 1 || t.k < 1 ||
      t.n_experts < 1 || (!t.offsets && t.n_experts != 1) || (codes && !swiglu) ||
      (swiglu && t.n % 2) || (!t.rows && t.x_rows != t.n_rows))
    return MOE_ERR_INVALID_ARG;
  if (t.n_rows == 0) return MOE_OK;
  if (!t.x || !t.x_scales || !t.w || !t.w_scales || !t.out || (codes && !t.out_scales) ||
      t.x_rows == 0 || t.x_stride < t.k || t.w_stride < (w4 ? t.k / 2 : t.k) ||
      overlap(t.n_rows, t.out_stride, swiglu ? t.n / 2 : t.n) ||
      (codes && overlap(t.n_rows, t.out_scales_stride, (t.n / 2 + 127) / 128)))
    return MOE_ERR_INVALID_ARG;
  const int unit = w4 ? 32 : 16, size = codes ? 1 : t.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (t.k % (w4 ? 128 : 16) || t.n_experts > kGemmMaxExperts || misaligned(t.x, 16) ||
      (t.x_stride & 15) || t.x_stride > INT32_MAX || misaligned(t.w, unit) ||
      ((t.w_stride | t.w_expert_stride) & (unit - 1)) ||
      t.n_rows > INT32_MAX - 256 || t.n > INT32_MAX - 256 || t.k > INT32_MAX - kGemmK ||
      misaligned(t.out, size))
    return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  int rc = begin(&dev);
  if (rc) return rc;
  Encode fn;
  if ((rc = encoder(&fn))) return rc;
  // tokens of a tile: whole ones where there are many, of experts three times their
  // average (a smaller ring stage holds more of the weights in flight)
  const long long many = t.offsets ? 3 * (((long long)t.n_rows + t.n_experts - 1) / t.n_experts)
                                   : t.n_rows;
  const int tokens = (int)std::min<long long>(kGemmTokens, (std::max(many, 32ll) + 15) / 16 * 16);
  // Two blocks a copy where the copy engine bounds: MXFP4 weights, whose rows are
  // half as long, with few tokens; with more the coarser ring costs more.  Gates and
  // ups of 64 experts, 2,048 x 7,168, by the rows of each: 10 (tiles of 32 at most) 163
  // us, one by one 174; 42 (128) 185 and 187; 48 (144) 218 and 198; 160 (240) 303 and
  // 277.  One matrix, 10,240 x 7,168: 32 rows 14.9 and 17.1, 128 18.9 both, 129 22.0
  // and 20.0.  (K of 896: the same within 3% on both sides.)
  const int per = w4 && tokens <= 128 ? 2 : 1;
  GemmMaps maps;
  if (!t.rows) {
    // tiles of a dense call have one size, but for the last; an expert's any
    const int tiles = (t.n_rows + tokens - 1) / tokens;
    const int size = (int)(((long long)t.n_rows + tiles - 1) / tiles + 15) / 16 * 16;
    const int last = (t.n_rows - (tiles - 1) * size + 15) / 16 * 16;
    for (int n = 16; n <= tokens; n += 16)
      if ((t.offsets || n == size || n == last) &&
          (rc = encode_rows(fn, &maps.x[n / 16 - 1], t, per, n / 2)))
        return rc;
  }
  if ((rc = encode_weights(fn, &maps.w, t, per, swiglu))) return rc;
  GemmArgs a{};
  a.kb = (t.k + kGemmK - 1) / kGemmK;
  a.wide = t.n;
  a.n = swiglu ? t.n / 2 : t.n;
  a.rows = t.n_rows;
  a.tokens = tokens;
  a.x_rows = t.x_rows;
  a.experts = t.n_experts;
  a.offsets = t.offsets;
  a.src = t.rows;
  a.x = t.x;
  a.x_stride = t.x_stride;
  a.k = t.k;
  a.xs = t.x_scales;
  a.xs_stride = t.x_scales_stride;
  a.ws = t.w_scales;
  a.ws_stride = t.w_scales_stride;
  a.ws_expert = t.w_scales_expert_stride;
  a.out = static_cast<char*>(t.out);
  a.out_stride = t.out_stride * size;
  a.os = t.out_scales;
  a.os_stride = t.out_scales_stride;
  a.out_dtype = t.out_dtype;
  const int piece = codes ? 4 : 16;   // what a lane stores at a time
  a.vec = !misaligned(t.out, piece) && a.out_stride % piece == 0;
  auto align = [](const void* q, int64_t s) {
    const uintptr_t b = (uintptr_t)q | (uintptr_t)s;
    return b % 16 == 0 ? 16 : b % 8 == 0 ? 8 : b % 4 == 0 ? 4 : 1;
  };
  a.xs_align = align(t.x_scales, a.xs_stride);
  a.ws_align = align(t.w_scales, a.ws_stride | a.ws_expert);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int n_sm = dev->n_sm;
  if (per == 2) return swiglu ? launch_product<true, true, 2>(a, maps, n_sm, st)
                              : launch_product<true, false, 2>(a, maps, n_sm, st);
  if (w4) return swiglu ? launch_product<true, true, 1>(a, maps, n_sm, st)
                        : launch_product<true, false, 1>(a, maps, n_sm, st);
  return swiglu ? launch_product<false, true, 1>(a, maps, n_sm, st)
                : launch_product<false, false, 1>(a, maps, n_sm, st);
}

int moe_debug_set_product_fault(int fault, unsigned long long wait_ns) {
  if (fault < 0) return MOE_ERR_INVALID_ARG;
  product_wait_ns.store(wait_ns, std::memory_order_relaxed);
  product_fault.store(fault, std::memory_order_relaxed);
  return MOE_OK;
}

int moe_dispatch(void* stream, const int32_t* idx, int n_tokens, int top_k, int n_experts,
                 int32_t* offsets, int32_t* rows, int32_t* slots) {
  if (n_tokens < 0 || top_k < 1 || n_experts < 1 || !offsets) return MOE_ERR_INVALID_ARG;
  const long long n = (long long)n_tokens * top_k;
  if (n > 0 && (!idx || !rows || !slots)) return MOE_ERR_INVALID_ARG;
  if (n_experts > kDispMaxExperts || n > 1 << 24) return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  const int rc = begin(&dev);
  if (rc) return rc;
  // few choices (a decode batch's) to eight warps of one CTA (fewer counts to clear
  // and add); then 4,096 a CTA, up to 16 CTAs; then clusters of 16 with as many a
  // round, whose parts are 2,048 a CTA and up
  const DispatchArgs a{idx, (int)n, top_k, n_experts, offsets, rows, slots};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n <= 1024) return launch_dispatch<8, 4>(a, 1, 1, st);
  int ctas = 1;
  while (ctas < kDispMaxCtas && n > 4096ll * ctas) ctas *= 2;
  const int clusters = n <= 65536 ? 1 : (int)std::min<long long>(kDispMaxClusters, n / 32768);
  return launch_dispatch<32, 4>(a, ctas, clusters, st);
}

int moe_combine(void* stream, const moe_combine_t* args) {
  if (!args) return MOE_ERR_INVALID_ARG;
  const moe_combine_t& t = *args;
  if (t.n_tokens < 0 || t.top_k < 1 || t.y_rows < 0 || t.d < 1 || !dtype16or32(t.dtype))
    return MOE_ERR_INVALID_ARG;
  if (t.n_tokens == 0) return MOE_OK;
  if ((!t.y && t.y_rows > 0) || !t.w || !t.slots || !t.out ||
      overlap(t.n_tokens, t.out_stride, t.d))
    return MOE_ERR_INVALID_ARG;
  if (t.d % 8 || t.top_k > 32 || misaligned(t.y, 16) || misaligned(t.residual, 16) ||
      misaligned(t.out, 16) ||
      ((t.y_stride | (t.residual ? t.residual_stride : 0) | t.out_stride) & 7))
    return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  const int rc = begin(&dev);
  if (rc) return rc;
  const CombineArgs a{t.y, t.y_stride, t.w, t.slots, t.residual, t.residual_stride, t.out,
                      t.out_stride, t.n_tokens, t.top_k, t.y_rows, t.d, t.dtype == MOE_DTYPE_F16};
  const unsigned pieces = (t.d / 8 + kCombThreads - 1) / kCombThreads;
  return launch(t.dtype == MOE_DTYPE_F32 ? combine_kernel<true> : combine_kernel<false>, pieces,
                std::min(t.n_tokens, 65535), kCombThreads, 0, 1, static_cast<cudaStream_t>(stream),
                a);
}

}  // extern "C"
