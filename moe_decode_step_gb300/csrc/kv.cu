// The serving operators' C ABI: block tables, the 8-bit KV cache, expert
// routing from logits.
#include "host.cuh"
#include "kv_append.cuh"
#include "kv_attention.cuh"
#include "kv_attention_tc.cuh"
#include "kv_plan.cuh"
#include "moe_decode.h"
#include "route.cuh"

using namespace moe;

namespace {

// SMs that the attention kernels' joins and workspace count on.
int attention_sms(const Device* dev) { return std::min((int)dev->n_sm, kDecMaxCtas); }

int block_log2(int bs) {
  for (int l = 4; l <= 7; ++l)
    if (bs == 1 << l) return l;
  return -1;
}

int cache_view(const moe_kv_cache_t* c, KvView* v) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return MOE_ERR_INVALID_ARG;
  v->bs_log2 = block_log2(c->block_size);
  if (v->bs_log2 < 0 || c->n_blocks < 1 || c->n_kv_heads < 1) return MOE_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MOE_ERR_UNSUPPORTED;
  if ((long long)c->n_blocks * c->block_size > INT32_MAX || c->n_kv_heads > 32767)
    return MOE_ERR_UNSUPPORTED;
  if (misaligned(c->k, 16) || misaligned(c->v, 16) ||
      ((c->block_stride | c->head_stride | c->token_stride) & 15))
    return MOE_ERR_UNSUPPORTED;
  v->k = c->k;
  v->v = c->v;
  v->ks = c->k_scale;
  v->vs = c->v_scale;
  v->bstride = c->block_stride;
  v->hstride = c->head_stride;
  v->tstride = c->token_stride;
  v->sstride = c->scale_stride;
  v->n_blocks = c->n_blocks;
  v->heads = c->n_kv_heads;
  return MOE_OK;
}

// Workspace of an attention call: per CTA its counters and its slots.
size_t arrived_bytes(int n_sm) { return ((size_t)n_sm * 16 + 255) / 256 * 256; }
template <int D>
size_t dec_floats_of() {
  return std::max({DecShape<D, 1>::SLOTS * DecShape<D, 1>::SLOT,
                   DecShape<D, 2>::SLOTS * DecShape<D, 2>::SLOT, 2 * PrShape<D, true>::SLOT});
}
size_t dec_floats(int d) { return d == 64 ? dec_floats_of<64>() : dec_floats_of<128>(); }

template <int D, int NT>
int launch_decode(AttnArgs a, int n_sm, int max_q, cudaStream_t st) {
  using Sh = DecShape<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kv_attention_decode<D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return cuda_fail(e);
  // strips the call can have at most, as far as the host knows; any grid is right
  long long span = (long long)a.max_blocks << a.c.bs_log2;
  if (a.window > 0) span = std::min(span, (long long)a.window + max_q + 32);
  const long long tiles = std::max(1ll, ((long long)max_q * a.group + Sh::ROWS - 1) / Sh::ROWS);
  const double all = (double)a.rows * a.c.heads * tiles;
  const int grid = (int)std::min((double)n_sm, all * (double)((span + 31) / 32) / Sh::WARPS + all + 1);
  if ((e = cudaMemsetAsync(a.arrived, 0, (size_t)grid * 16, st)) != cudaSuccess)
    return cuda_fail(e);
  kv_attention_decode<D, NT><<<grid, Sh::THREADS, Sh::SMEM, st>>>(a);
  return end();
}

template <int D, bool PAIR>
int launch_tensor(const AttnArgs& a, int n_sm, cudaStream_t st) {
  using Sh = PrShape<D, PAIR>;
  cudaError_t e = cudaFuncSetAttribute(kv_attention_tc<D, PAIR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
  if (e != cudaSuccess) return cuda_fail(e);
  if ((e = cudaMemsetAsync(a.arrived, 0, (size_t)n_sm * 16, st)) != cudaSuccess)
    return cuda_fail(e);
  kv_attention_tc<D, PAIR><<<n_sm, kPrThreads, Sh::SMEM, st>>>(a);
  return end();
}

// The kernel by the rows (queries times heads) of a KV head in the longest batch
// row, as far as the host knows.  Measured on the device (us), 64 heads over 8
// of 128, 8 batch rows of 4,090 to 8,185 tokens where nothing else is said:
//  - up to 8 rows, one n-tile a warp: 47, two 52; to 32, two: 81 at 32 rows, on
//    tcgen05 89 (32 batch rows of 1,000 to 4,000 tokens 119 against 134); at 48
//    102 against 89.  Where the table says that rows are short the tcgen05
//    kernel's start counts, to 64 rows: with 500 to 900 tokens 44 against 53 at
//    48 rows, 49 against 56 at 64.
//  - then one row tile whose streams share its keys: 96 at 128 rows against 111
//    in pairs of row tiles.  Above that pairs, if the batch's rows fill them on
//    average and are enough for the SMs: 116 against 147 at 256 rows, 194 against
//    188 at 384, 198 against 231 at 512 (32 heads of 64: 103 against 116, 154
//    against 175); of one batch row the pairs are few: 118 against 73 at 256,
//    102 against 92 at 768, 106 against 109 at 1,024, 134 against 161 at 2,048.
template <int D>
int launch_attention(const AttnArgs& a, int n_sm, int max_q, cudaStream_t st) {
  const long long rows = (long long)max_q * a.group;
  const long long tokens = (long long)a.max_blocks << a.c.bs_log2;
  if (rows <= 8) return launch_decode<D, 1>(a, n_sm, max_q, st);
  if (rows <= 32 || (rows <= 64 && tokens <= 1024)) return launch_decode<D, 2>(a, n_sm, max_q, st);
  const long long pairs = (long long)a.rows * a.c.heads * ((rows + 255) / 256);
  const bool filled = (long long)a.n_tokens * a.group > 128ll * a.rows && pairs > n_sm / 4;
  if (rows <= 128 || (rows <= 65536 / D && !filled)) return launch_tensor<D, false>(a, n_sm, st);
  return launch_tensor<D, true>(a, n_sm, st);
}

// Shared memory only where groups go through it (sizes that are no power of
// two from 4 to 128, or experts one a load).
void launch_route(void (*kernel)(RouteArgs), const RouteArgs& a, int regs, bool vec,
                  unsigned grid, cudaStream_t st) {
  const int size = a.E / a.groups;
  const bool shuffles = vec && (size & (size - 1)) == 0 && size >= 4 && size <= 128;
  const int smem = a.groups > 1 && !shuffles ? kRouteWarps * regs * 32 * 4 : 0;
  kernel<<<grid, 32 * kRouteWarps, smem, st>>>(a);
}

}  // namespace

extern "C" {

int moe_kv_plan(void* stream, const int32_t* ctx_lens, const int32_t* q_lens, int n_rows,
                int32_t* block_table, int64_t table_stride, int max_blocks,
                const int32_t* free_list, int free_cap, const int32_t* n_free, int block_size,
                int32_t* seq_lens, int32_t* q_start, int32_t* slot_map, int n_slots,
                int32_t* n_free_out, int32_t* n_unserved) {
  if (!ctx_lens || !q_lens || !block_table || (!free_list && free_cap > 0) || !n_free ||
      !seq_lens || !q_start || (!slot_map && n_slots > 0) || !n_free_out || !n_unserved)
    return MOE_ERR_INVALID_ARG;
  const int bl = block_log2(block_size);
  if (n_rows < 1 || max_blocks < 1 || table_stride < max_blocks || free_cap < 0 || n_slots < 0 ||
      bl < 0 || n_free == n_free_out)
    return MOE_ERR_INVALID_ARG;
  if (n_rows > kPlanMaxRows) return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  int rc = begin(&dev);
  if (rc) return rc;
  // (past 48 KB with the kernel's static shared memory, for which there is room)
  const int smem = (2 * n_rows + 1) * 4;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (2 * kPlanMaxRows + 1) * 4);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  PlanArgs p{ctx_lens, q_lens,   n_rows,  block_table, table_stride, max_blocks, free_list, free_cap,
             n_free,   bl,       seq_lens, q_start,    slot_map,     n_slots,    n_free_out, n_unserved};
  // entries to write per thread: one slot, or one row's table entries per warp
  const long long work = std::max<long long>(n_slots, (long long)n_rows * 32);
  const int grid = (int)std::min<long long>(dev->n_sm, (work + kPlanThreads - 1) / kPlanThreads);
  kv_plan_kernel<<<grid, kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
  return end();
}

int moe_kv_release(void* stream, const uint8_t* finished, int n_rows, int32_t* seq_lens,
                   const int32_t* block_table, int64_t table_stride, int max_blocks,
                   int32_t* free_list, int free_cap, const int32_t* n_free, int block_size,
                   int32_t* n_free_out) {
  if (!finished) return MOE_ERR_INVALID_ARG;
  return moe_kv_release_past(stream, finished, nullptr, n_rows, seq_lens, block_table, table_stride,
                             max_blocks, free_list, free_cap, n_free, block_size, n_free_out);
}

int moe_kv_release_past(void* stream, const uint8_t* finished, const int32_t* keep_lens,
                        int n_rows, int32_t* seq_lens, const int32_t* block_table,
                        int64_t table_stride, int max_blocks, int32_t* free_list, int free_cap,
                        const int32_t* n_free, int block_size, int32_t* n_free_out) {
  if ((!finished && !keep_lens) || !seq_lens || !block_table || (!free_list && free_cap > 0) ||
      !n_free || !n_free_out)
    return MOE_ERR_INVALID_ARG;
  const int bl = block_log2(block_size);
  if (n_rows < 1 || max_blocks < 1 || table_stride < max_blocks || free_cap < 0 || bl < 0)
    return MOE_ERR_INVALID_ARG;
  if (n_rows > kPlanMaxRows) return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  int rc = begin(&dev);
  if (rc) return rc;
  ReleaseArgs p{finished,   keep_lens, n_rows,   seq_lens, block_table, table_stride,
                max_blocks, free_list, free_cap, n_free,   bl,          n_free_out};
  kv_release_kernel<<<1, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return end();
}

int moe_kv_append(void* stream, const moe_kv_cache_t* cache, const void* k, const void* v,
                  int dtype, int64_t k_token_stride, int64_t k_head_stride,
                  int64_t v_token_stride, int64_t v_head_stride, const int32_t* slot_map,
                  int n_tokens) {
  AppendArgs a{};
  int rc = cache_view(cache, &a.c);
  if (rc) return rc;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (n_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (n_tokens == 0) return MOE_OK;
  if (!k || !v || !slot_map) return MOE_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) ||
      ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 7) ||
      2 * (long long)cache->n_kv_heads > 65535)
    return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  if ((rc = begin(&dev))) return rc;
  a.src[0] = static_cast<const uint16_t*>(k);
  a.src[1] = static_cast<const uint16_t*>(v);
  a.ts[0] = k_token_stride;
  a.hs[0] = k_head_stride;
  a.ts[1] = v_token_stride;
  a.hs[1] = v_head_stride;
  a.f16 = dtype == MOE_DTYPE_F16;
  a.slot = slot_map;
  a.n_tokens = n_tokens;
  // short calls: few slots a CTA, so that a decode batch's tokens find a warp
  // each (64 tokens: 7.5 us, with 64 slots a CTA 16.4); long ones: a block's
  // worth (16 prompts of some 1,000 tokens: 32 us, with 8 slots a CTA 51)
  a.chunk = n_tokens <= 1024 ? 8 : 64;
  const dim3 grid((n_tokens - 1) / a.chunk + 1, 2 * cache->n_kv_heads);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cache->head_dim == 64) kv_append_kernel<64><<<grid, kAppendThreads, 0, st>>>(a);
  else kv_append_kernel<128><<<grid, kAppendThreads, 0, st>>>(a);
  return end();
}

size_t moe_kv_attention_workspace(int head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  const Device* dev;
  if (this_device(&dev)) return 0;
  const int n_sm = attention_sms(dev);
  return arrived_bytes(n_sm) + (size_t)n_sm * dec_floats(head_dim) * 4;
}

int moe_kv_attention(void* stream, const moe_kv_cache_t* cache, const moe_kv_attention_t* args) {
  AttnArgs a{};
  int rc = cache_view(cache, &a.c);
  if (rc) return rc;
  if (!args) return MOE_ERR_INVALID_ARG;
  const moe_kv_attention_t& t = *args;
  if (t.dtype != MOE_DTYPE_BF16 && t.dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (t.n_rows < 0 || t.n_tokens < 0 || t.n_heads < 1 || t.n_heads % cache->n_kv_heads ||
      t.max_blocks < 1 || t.table_stride < t.max_blocks || t.window < 0 || !(t.scale == t.scale))
    return MOE_ERR_INVALID_ARG;
  if (t.n_rows == 0 || t.n_tokens == 0) return MOE_OK;
  if (!t.q || !t.out || !t.block_table || !t.seq_lens || !t.q_start || !t.workspace)
    return MOE_ERR_INVALID_ARG;
  if (misaligned(t.q, 16) || misaligned(t.out, 16) || misaligned(t.workspace, 256) ||
      ((t.q_token_stride | t.q_head_stride | t.out_token_stride | t.out_head_stride) & 7))
    return MOE_ERR_UNSUPPORTED;
  if (t.n_rows > kPlanMaxRows) return MOE_ERR_UNSUPPORTED;
  if ((long long)t.max_blocks * cache->block_size > INT32_MAX - 128 ||
      (long long)t.n_tokens * t.n_heads > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  if ((rc = begin(&dev))) return rc;
  if (t.workspace_bytes < moe_kv_attention_workspace(cache->head_dim)) return MOE_ERR_ALLOC;
  a.q = static_cast<const uint16_t*>(t.q);
  a.q_ts = t.q_token_stride;
  a.q_hs = t.q_head_stride;
  a.out = static_cast<uint16_t*>(t.out);
  a.o_ts = t.out_token_stride;
  a.o_hs = t.out_head_stride;
  a.lse = t.lse;
  a.table = t.block_table;
  a.table_stride = t.table_stride;
  a.seq_lens = t.seq_lens;
  a.q_start = t.q_start;
  a.f16 = t.dtype == MOE_DTYPE_F16;
  a.rows = t.n_rows;
  a.n_tokens = t.n_tokens;
  a.heads = t.n_heads;
  a.group = t.n_heads / cache->n_kv_heads;
  a.max_blocks = t.max_blocks;
  a.causal = t.causal != 0;
  a.window = t.window;
  a.scale_log2 = t.scale * 1.4426950408889634f;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  a.arrived = static_cast<unsigned*>(t.workspace);
  const int n_sm = attention_sms(dev);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(t.workspace) + arrived_bytes(n_sm));
  const int max_q = std::max(t.max_q, 1);   // a hint, whatever it says
  return cache->head_dim == 64 ? launch_attention<64>(a, n_sm, max_q, st)
                               : launch_attention<128>(a, n_sm, max_q, st);
}

int moe_route(void* stream, const moe_route_t* cfg, const void* logits, int dtype,
              int64_t row_stride, int64_t n_rows, const float* bias, int32_t* idx, float* w) {
  if (!cfg) return MOE_ERR_INVALID_ARG;
  const moe_route_t& c = *cfg;
  if (c.n_experts < 1 || c.n_groups < 1 || c.n_experts % c.n_groups || c.topk_groups < 1 ||
      c.topk_groups > c.n_groups || c.top_k < 1 ||
      c.top_k > (long long)c.topk_groups * (c.n_experts / c.n_groups) ||
      (c.group_top != 1 && c.group_top != 2) || (c.scoring != 0 && c.scoring != 1) ||
      !(c.routed_scale == c.routed_scale) || n_rows < 0 || row_stride < 0 || dtype < 0 ||
      dtype > MOE_DTYPE_F32)
    return MOE_ERR_INVALID_ARG;
  if (c.n_experts > 1024 || c.top_k > 32 || c.n_groups > 32) return MOE_ERR_UNSUPPORTED;
  if (n_rows == 0) return MOE_OK;
  if (!logits || !idx || !w) return MOE_ERR_INVALID_ARG;
  if ((n_rows + kRouteWarps - 1) / kRouteWarps > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  const Device* dev;
  int rc = begin(&dev);
  if (rc) return rc;
  RouteArgs a{logits, row_stride, n_rows, bias, idx, w, dtype, c.n_experts, c.top_k, c.scoring,
              c.n_groups, c.topk_groups, c.group_top, c.renormalize != 0, c.routed_scale};
  const unsigned grid = (unsigned)((n_rows + kRouteWarps - 1) / kRouteWarps);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // four experts a load where every row allows it
  const int size = dtype == MOE_DTYPE_F32 ? 4 : 2;
  const bool vec = c.n_experts >= 128 && row_stride % 4 == 0 && !misaligned(logits, 4 * size) &&
                   !misaligned(bias, 16);
  const int n = c.n_experts;
  if (vec) {
    if (n <= 128) launch_route(route_kernel<1, 4>, a, 4, vec, grid, st);
    else if (n <= 256) launch_route(route_kernel<2, 4>, a, 8, vec, grid, st);
    else if (n <= 512) launch_route(route_kernel<4, 4>, a, 16, vec, grid, st);
    else launch_route(route_kernel<8, 4>, a, 32, vec, grid, st);
  } else {
    if (n <= 64) launch_route(route_kernel<2, 1>, a, 2, vec, grid, st);
    else if (n <= 256) launch_route(route_kernel<8, 1>, a, 8, vec, grid, st);
    else launch_route(route_kernel<32, 1>, a, 32, vec, grid, st);
  }
  return end();
}

}  // extern "C"
