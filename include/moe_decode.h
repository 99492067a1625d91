/*
 * moe_decode.h — C ABI of a single-GPU (GB300, sm_103a) mixture-of-experts
 * decode layer for 1..64 rows.
 *
 * The layer (one call of moe_decode_forward) is, for every row b of x:
 *   router      logits = x_b . W_r^T; s = sigmoid(logits); the top_k experts
 *               by s + bias (ties to the lower index); combine weights
 *               w = routed_scale * s_sel / sum(s_sel)
 *   routed      for each selected expert e: h = silu(W_gate,e x_b) * (W_up,e x_b),
 *               y_e = W_down,e h; y_routed = sum_j w_j y_{e_j}
 *               (expert weights are MXFP4: E2M1 nibbles, one E8M0 scale per
 *               32 contiguous K elements)
 *   shared      y_shared = W_sd (silu(W_sg x_b) * (W_su x_b)), bf16 weights
 *   tail        z = residual_b + y_routed + y_shared; residual_b <- bf16(z);
 *               out_b = bf16(z / sqrt(mean(z^2) + eps) * gamma)
 *
 * Sources: "Kimi K3 on GB300: 13 kernels a layer, and what 842 and 423 tokens
 * a second measure" — section "What one decode step of Kimi K3 does" (16 of
 * 896 experts per token, 17,547,264-byte MXFP4 experts), section "Why batch 1
 * on a rack is not only a bandwidth problem" (packed FP4 expert weights),
 * section "What the fused path changes" (router/MoE front, shared expert on a
 * side stream, one persistent routed-expert kernel for FC1 and FC2, a tail that
 * folds the down-projection reduction and the next norm together, L2 prefetch
 * of upcoming weights on a third stream; here the prefetch is issued by the
 * tail kernel).  The pages give the structure only;
 * the formulas above are the plainest reading of that structure.  Element and
 * scale encodings: OCP Microscaling Formats (MX) Specification v1.0.
 *
 * Conventions for every call:
 *  - Pointers marked "device" are CUDA device pointers on the device that was
 *    current at moe_layer_create; "host" pointers are ordinary host memory.
 *    The caller owns every buffer it passes; the library borrows weight
 *    pointers for the handle's lifetime and never frees them.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Forward calls are asynchronous on that stream, allocate nothing and never
 *    synchronise the host, so they may be captured into a CUDA graph.
 *  - Every call returns a moe_status (0 = MOE_OK).  Nothing aborts or throws
 *    across the ABI.  A handle must not be used from two streams at once.
 *  - bf16 tensors are row-major uint16 bit patterns (torch.bfloat16 layout).
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,   /* null pointer, bad size or dims */
  MOE_ERR_UNSUPPORTED = 2,   /* B outside [1, max_batch], device is not sm_103, misaligned
                                pointer: the caller should use another implementation */
  MOE_ERR_CUDA = 3,          /* a CUDA runtime call failed (the error is kept for
                                moe_last_cuda_error) */
  MOE_ERR_ALLOC = 4,         /* workspace allocation failed at create time */
  MOE_ERR_TIMEOUT = 5        /* a device-side bounded wait expired (see moe_layer_status) */
} moe_status;

typedef struct moe_layer* moe_layer_t;

/* Layer dimensions.  d % 256 == 0 and d <= 7680; f % 256 == 0 and f <= 3072;
 * f_shared % 256 == 0 and f_shared <= 4096; 1 <= top_k <= 32; top_k <= n_experts
 * <= 1024; 1 <= max_batch <= 64 (INVALID_ARG otherwise).
 *
 * expert_path picks how the routed experts run.  1: mma.sync tensor cores
 * with the weights converted to f16 in registers (the GEMV regime; the
 * kernels read the tiled layouts, FC1 matrices in layout 2 and FC2 matrices in
 * layout 1), the shared expert and the router on the CUDA cores.  2: tcgen05
 * tensor cores, block-scaled MXFP4 MMAs with tensor-memory accumulators (the
 * UMMA layouts, FC1 in layout 4 and FC2 in layout 3); the shared expert (and,
 * from 25 rows, the router) as bf16 MMAs on the same tensor cores, from bf16
 * copies of those weights in 128-row tiles that the handle owns (2 * (3 * d *
 * f_shared + 128 * ceil(E / 128) * d) bytes of extra device memory).  0
 * (default): the layer keeps both and takes path 1 for B = 1 and path 2 for
 * B >= 2, or only path 1 when max_batch is 1 (one copy of the expert bytes
 * instead of two).  Path 1's kernels hold a ring of shared-memory stages
 * sized for the dims; where it does not fit (large d with large f, or
 * f_shared above 3072, for example), path 1 returns UNSUPPORTED and path 0
 * keeps path 2 alone.  All give results within the same tolerance of the
 * exact layer.
 *
 * mxfp4_layout says how the caller's expert weights are laid out: 0
 * (canonical), 1 (tiled: FC1 layout 2, FC2 layout 1) or 3 (UMMA: FC1 layout 4,
 * FC2 layout 3); see mxfp4_pack.  Weights already in a kept path's layouts
 * are used in place; for every other kept path moe_layer_create relays them
 * into a copy the handle owns (E * 3 * d * f * 17/32 bytes of extra device
 * memory each). */
typedef struct {
  int32_t d;              /* hidden size */
  int32_t f;              /* routed-expert intermediate size */
  int32_t n_experts;      /* E */
  int32_t top_k;          /* k */
  int32_t f_shared;       /* shared-expert intermediate size */
  int32_t max_batch;      /* largest B forward will be called with */
  float routed_scale;     /* combine weights sum to this (2.5 for the Kimi-style router) */
  float rms_eps;          /* RMSNorm epsilon (1e-6) */
  int32_t mxfp4_layout;   /* 0: canonical, 1: tiled, 3: UMMA expert weights (see above) */
  int32_t expert_path;    /* 0: both (by batch), 1: mma.sync, 2: tcgen05 (see above) */
} moe_dims_t;

/* Device pointers to the layer's weights (borrowed, never freed).
 * Expert e's FC1 rows 0..f-1 are the gate projection and rows f..2f-1 the up
 * projection; row i of the gate pairs with row i of the up projection. */
typedef struct {
  const void* router_w;        /* device bf16 [E][d] */
  const float* router_bias;    /* device fp32 [E], used for selection only */
  const uint8_t* w_gu_q;       /* device [E][2f][d/2]  E2M1 nibbles (layout 0, 2 or 4) */
  const uint8_t* w_gu_s;       /* device [E][2f][d/32] E8M0 scale bytes (layout 0, 2 or 4) */
  const uint8_t* w_d_q;        /* device [E][d][f/2]  (layout 0, 1 or 3) */
  const uint8_t* w_d_s;        /* device [E][d][f/32] (layout 0, 1 or 3) */
  const void* shared_gu;       /* device bf16 [2 f_shared][d] (gate rows, then up rows) */
  const void* shared_d;        /* device bf16 [d][f_shared] */
  const void* rms_gamma;       /* device bf16 [d] */
} moe_weights_t;

/* Validate dims, device (must be sm_103) and pointer alignment (16 bytes),
 * allocate the workspace (routing tables, intermediates, timing events) on
 * the current device and return a handle in *out.
 * Errors: INVALID_ARG (null or bad dims), UNSUPPORTED (device/alignment),
 * ALLOC (workspace), CUDA. */
int moe_layer_create(const moe_dims_t* dims, const moe_weights_t* weights, moe_layer_t* out);

/* Free the workspace (synchronises the device first).  NULL is accepted. */
int moe_layer_destroy(moe_layer_t layer);

/* Router only: x device bf16 [B][d] -> idx device int32 [B][k] (descending by
 * score + bias, ties to the lower index) and w device fp32 [B][k] (combine
 * weights).  Same kernel as the first step of moe_decode_forward.
 * Errors: INVALID_ARG, UNSUPPORTED (B), CUDA. */
int moe_router_topk(moe_layer_t layer, void* stream, const void* x, int B, int32_t* idx, float* w);

/* The whole layer.  x device bf16 [B][d] (read only); residual device bf16
 * [B][d], read and overwritten with bf16(z); out device bf16 [B][d].  x, out
 * and residual must not overlap.  Asynchronous, allocation-free. */
int moe_decode_forward(moe_layer_t layer, void* stream, const void* x, int B, void* residual,
                       void* out);

/* The same layer with HOST buffers: copies x and residual host -> device on
 * `stream`, runs moe_decode_forward on the handle's own device staging
 * buffers, copies residual and out back, and synchronises `stream` before
 * returning.  x_host, residual_host, out_host: host bf16 [B][d] (pinned memory
 * gives asynchronous copies; pageable memory works but copies synchronously).
 * With pinned buffers and a stream other than the legacy default stream, the
 * first call captures the copies and the kernels as one CUDA graph, which
 * later calls with the same buffers, B and stream replay (one launch per call;
 * changing any of them captures again).  Overlapping calls on one layer race,
 * as for moe_decode_forward. */
int moe_decode_forward_host(moe_layer_t layer, void* stream, const void* x_host, int B,
                            void* residual_host, void* out_host);

/* moe_decode_forward that also exports intermediates (any may be NULL):
 * y_routed device fp32 [B][d], y_shared device fp32 [B][d],
 * h device fp32 [B][k][f] (h[b][j] belongs to expert idx[b][j]),
 * z device fp32 [B][d] (residual + y_routed + y_shared before bf16 rounding),
 * out_f32 device fp32 [B][d] (the normalised output before bf16 rounding). */
int moe_decode_forward_debug(moe_layer_t layer, void* stream, const void* x, int B, void* residual,
                             void* out, float* y_routed, float* y_shared, float* h, float* z,
                             float* out_f32);

/* Dequantise one expert matrix on the GPU from the handle's tiled copy, with
 * the kernels' element decode (cvt.rn.f16x2.e2m1x2) and the exact scale value:
 * which = 0 -> FC1 [2f][d], which = 1 -> FC2 [d][f], canonical row order;
 * out device fp32.  (The matmul kernels read scale code 0, 2^-127, as 0: the
 * products it scales are below 6 * 2^-127 * |activation|.) */
int moe_debug_dequant(moe_layer_t layer, void* stream, int expert, int which, float* out);

/* Activation format of the routed experts' products (the pages' routed-expert
 * kernel multiplies FP4 weights by MXFP8 activations: "Kimi K3 on GB300: 13
 * kernels a layer", "Why batch 1 on a rack is not only a bandwidth problem").
 * fmt 0 (default): x (bf16) and h (fp32) as they are, the exact layer within
 * the stated tolerance.  fmt 1: x and h rounded to MXFP8 (OCP MX v1.0: E4M3
 * elements, nearest with ties to even and saturation at 448, one E8M0 scale
 * 2^(floor(log2 max|v|) - 8) per 32 contiguous elements) before they meet the
 * MXFP4 weights; the router, shared expert and tail are unchanged.  The
 * one-row mma.sync kernel carries the rounded values exactly in its f16
 * operands; the tensor-core path builds its activation planes (E2M1 digits,
 * block-scaled MMAs) from them.  fmt 1 runs on the tensor-core path at any B
 * and on the mma.sync path at B = 1; a forward of B > 1 rows on the mma.sync
 * path returns MOE_ERR_UNSUPPORTED.  Errors: INVALID_ARG. */
int moe_set_act_format(moe_layer_t layer, int fmt);

/* Chain layers: this layer's tail kernel, whose CTAs start while the expert
 * kernels finish, issues L2 prefetches (prefetch.global.L2::evict_last) of
 * `next`'s router weights before it waits for them, so the next layer's
 * router, the first kernel of the next forward, finds them in L2.  No extra
 * launch or stream.  next may be NULL to switch it off.  Both handles must
 * live on the same device. */
int moe_set_prefetch_next(moe_layer_t layer, moe_layer_t next);

/* Synchronise the layer's streams and report the device status word
 * (0 = ok, else a moe_status such as MOE_ERR_TIMEOUT); clears it. */
int moe_layer_status(moe_layer_t layer, int* device_status);

/* Failure-detection test hook (the pages have no counterpart; it exists so a
 * test can watch a device-side wait expire without faulting anything).
 * fault = 1: in later forwards of one row on the mma.sync path (FC1 and FC2
 * in one launch, whose CTAs meet at a grid-wide barrier between the two
 * steps), CTA 0 does not count itself at that barrier, and every CTA's wait
 * there is limited to wait_ns nanoseconds (0: the default 2 s).  The waits
 * expire, FC2 runs on the FC1 results that are already written, the forward
 * completes, and moe_layer_status then reports MOE_ERR_TIMEOUT.  fault = 0
 * restores normal operation.
 * Nothing on the GPU traps, faults or hangs.  Errors: INVALID_ARG. */
int moe_debug_set_fault(moe_layer_t layer, int fault, unsigned long long wait_ns);

/* Per-phase timing of forward calls (CUDA events on the launching stream;
 * under stream capture they become event-record nodes of the graph).
 * enable != 0 records events around each phase from the next forward on.
 * moe_get_timing synchronises and writes up to n floats (microseconds) for
 * the last forward: [0] router + top-k, [1] FC1 (shared then routed gate/up),
 * [2] FC2 (shared then routed down), [3] always 0 (the shared expert has no
 * phase of its own), [4] tail, [5] whole layer. */
int moe_set_timing(moe_layer_t layer, int enable);
int moe_get_timing(moe_layer_t layer, float* us, int n);

/* Device-side kernel trace.  enable != 0 makes every later forward record,
 * per kernel, the earliest CTA start and the latest CTA end (globaltimer,
 * nanoseconds).  moe_get_trace synchronises the device and writes up to n
 * values: [start, end] of router, top-k, FC1, FC2, tail, in that order (ten
 * values); a kernel that did not run reports start > end. */
int moe_set_trace(moe_layer_t layer, int enable);
int moe_get_trace(moe_layer_t layer, unsigned long long* ns, int n);

/* Number of kernel launches one forward makes for batch B. */
int moe_launches_per_forward(moe_layer_t layer, int B);

/* ---- MXFP4 packing (OCP MX v1.0: E2M1 elements, E8M0 scale per 32 K) ---- */
/* Canonical layout 0: row-major; byte j of a row holds elements 2j (low
 * nibble) and 2j+1 (high nibble); scale byte b of a row covers elements
 * 32b..32b+31.  Scale exponent = floor(log2(amax)) - 2 clamped to [-127, 127]
 * (all-zero block: -127); element code = nearest E2M1 value to w / 2^exp,
 * ties to the even code, magnitudes past 6 saturate to 6, sign bit = sign of w. */

/* Tiled layouts 1 and 2 hold the same bytes for the tensor-core kernels.
 * Rows form tiles of 16 "mma rows": layout 1 puts rows 16T..16T+15 in tile T;
 * layout 2 (a [2n][k] gate/up matrix, row i pairing with row n + i) puts rows
 * 8T..8T+7 as mma rows 0..7 and rows n+8T..n+8T+7 as mma rows 8..15.  Tile T's
 * nibbles occupy bytes [8kT, 8k(T+1)): for K blocks 2P and 2P+1 (32 elements
 * each) and lane L = 4g + t (g < 8, t < 4), 16 bytes at 8kT + (32P + L) * 16
 * hold canonical bytes [4t, 4t+4) of block 2P of mma row g, then of mma row
 * g + 8, then the same two for block 2P+1.  Tile T's scales occupy bytes
 * [kT/2, k(T+1)/2): for block group Q (blocks 4Q..4Q+3) and g, 8 bytes at
 * kT/2 + (8Q + g) * 8 hold, per block 4Q+j, the scale of mma row g (byte 2j)
 * and of mma row g + 8 (byte 2j + 1).  Tiled layouts need k % 128 == 0 and
 * rows % 16 == 0. */

/* UMMA layouts 3 and 4 hold the same bytes as tcgen05 block-scaled operands
 * (no swizzle, K-major core matrices of 8 rows x 16 bytes).  Rows form tiles
 * of 128 "mma rows": layout 3 puts rows 128T..128T+127 in tile T; layout 4 (a
 * [2n][k] gate/up matrix) puts rows 64T..64T+63 as mma rows 0..63 and rows
 * n+64T..n+64T+63 as mma rows 64..127.  Tile T's nibbles occupy bytes
 * [64kT, 64k(T+1)): the 16 canonical bytes of K block b of mma row m at
 * 64kT + 2048b + 128(m/8) + 16(m%8).  Tile T's scales occupy bytes [4kT,
 * 4k(T+1)): the scale of (m, b) at 4kT + 512(b/4) + 16(m%32) + 4(m/32) + b%4.
 * UMMA layouts need k % 128 == 0 and rows % 128 == 0. */

/* Bytes of nibbles for rows x k (k % 32 == 0, and the layout's rules);
 * *scale_bytes gets the scale bytes when non-NULL.  The same for every
 * layout.  Returns 0 on bad arguments. */
size_t mxfp4_packed_bytes(int64_t rows, int64_t k, int layout, size_t* scale_bytes);

/* Host packer: w host fp32 [rows][k] -> q host [rows][k/2], s host [rows][k/32]. */
int mxfp4_pack(const float* w, int64_t rows, int64_t k, uint8_t* q, uint8_t* s, int layout);

/* Device packer, asynchronous on stream: w device fp32 -> q, s device. */
int mxfp4_pack_device(void* stream, const float* w, int64_t rows, int64_t k, uint8_t* q,
                      uint8_t* s, int layout);

/* Host conversion between layouts (0 to 4) of one rows x k matrix: q_in, s_in
 * host in layout `from`; q_out, s_out host in layout `to` (same sizes, must not
 * overlap the input).  Errors: INVALID_ARG, UNSUPPORTED (a layout's rules). */
int mxfp4_repack(const uint8_t* q_in, const uint8_t* s_in, int64_t rows, int64_t k, int from,
                 int to, uint8_t* q_out, uint8_t* s_out);

/* Canonical packed bytes -> tiled or UMMA layout 1 to 4, asynchronous on stream, for
 * n_mat matrices stored back to back (rows x k each): q_in, s_in device
 * canonical; q_out, s_out device, the same sizes, must not overlap the input.
 * Errors: INVALID_ARG, UNSUPPORTED (layout rules, 16-byte alignment), CUDA. */
int mxfp4_retile_device(void* stream, const uint8_t* q_in, const uint8_t* s_in, int64_t n_mat,
                        int64_t rows, int64_t k, int layout, uint8_t* q_out, uint8_t* s_out);

/* Router + top-k that allocates nothing (no counterpart in the paper: it
 * exists for callers that cannot call cudaMalloc, e.g. code running inside a
 * stream capture it does not own, runtimes that hand over a fixed memory pool,
 * or callers that must not synchronise the device).  It needs no layer handle:
 * router_w device bf16 [E][d], router_bias device fp32 [E], x device bf16
 * [B][d]; outputs idx device int32 [B][k] and w device fp32 [B][k], exactly
 * as moe_router_topk.  Its scratch (logits, ticket, status word, routing
 * tables; 284,416 bytes) is one static device array that every GPU loading
 * this library holds until the process exits; each call looks up the current
 * device's address of it.  Limits: B <= 64, E <= 1024, k <= 32, d % 256 == 0,
 * d <= 7680 (as for a layer); larger sizes return MOE_ERR_UNSUPPORTED.  The
 * first call on each device (and the first with a new d) sizes the launch
 * (host-side queries, no allocation): make that call before any stream
 * capture.  A CUDA error already pending when the call starts is returned
 * (MOE_ERR_CUDA, its code kept for moe_last_cuda_error) and nothing is
 * launched.  Every call shares the one array, so calls that overlap on the GPU
 * (two streams, or two threads) race; calls in one stream are safe. */
int moe_router_topk_noalloc(void* stream, const void* router_w, const float* router_bias,
                            const void* x, int B, int d, int n_experts, int top_k,
                            float routed_scale, int32_t* idx, float* w);

/* Status word of the allocation-free router on the current device: 0, or
 * MOE_ERR_TIMEOUT when a bounded device-side wait of an earlier call expired
 * (its outputs are then not valid).  Each call clears the word when it
 * starts, so this reports the calls since the last one started; synchronises
 * the device, then clears the word. */
int moe_router_topk_noalloc_status(int* device_status);

/* ---- Serving operators beside the layer ----
 * Block tables, an 8-bit KV cache with its attention, and expert routing from
 * logits, for the parts of a decode step around moe_decode_forward (no
 * counterpart in the pages, which describe the MoE half of a layer; the
 * formulas are the plain ones stated at each call).  They need no handle:
 * every call is asynchronous on `stream`, allocates nothing, never
 * synchronises the host and may be captured into a CUDA graph.  Lengths live
 * on the device, so a captured graph follows them.  A call checks what the
 * host can see (null pointers, sizes, alignment) and reports it as a status;
 * values it reads on the device (lengths, block ids, slots) are bounded there
 * as each call states, so that no value makes it read or write out of range.
 * A CUDA error already pending when a call starts is returned (MOE_ERR_CUDA)
 * and nothing is launched.  Limits: 16,384 rows (requests) per call; device
 * sm_103, else UNSUPPORTED. */

/* Element types: BF16 and F16, of moe_route's logits F32 too. */
typedef enum {
  MOE_DTYPE_BF16 = 0,
  MOE_DTYPE_F16 = 1,
  MOE_DTYPE_F32 = 2    /* only where a call says so */
} moe_dtype;

/* A paged KV cache in 8 bits.  Tokens live in blocks of block_size (16, 32,
 * 64 or 128); element (block b, KV head h, token t of the block, dim j) of K
 * is the E4M3 code at k[b * block_stride + h * head_stride + t * token_stride
 * + j] and stands for code * 2^(k_scale[b * scale_stride + h] - 127): one
 * E8M0 scale per (block, head), within 2^-60 .. 2^60 (bytes 67 .. 187; a byte
 * outside reads as the nearest of these).  V likewise.  Strides are in bytes;
 * block, head and token strides and the k and v pointers are multiples of 16,
 * so blocks may be head-major or token-major, or views of one larger tensor.
 * head_dim is 64 or 128; n_blocks * block_size < 2^31. */
typedef struct {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int64_t block_stride, head_stride, token_stride;
  int64_t scale_stride;
  int32_t n_blocks, n_kv_heads, block_size, head_dim;
} moe_kv_cache_t;

/* Block tables and slot maps of one step, from request lengths.  Row r holds
 * ctx_lens[r] cached tokens (in the first ceil(ctx / block_size) entries of
 * its block_table row, which are all it holds: a row that got shorter gives the
 * others back first, by moe_kv_release_past) and gets q_lens[r] new ones.  New blocks are taken in
 * row order from the top of the stack free_list[0 .. *n_free): the i-th new
 * block of the step is free_list[*n_free - 1 - i].  A row is served when its
 * blocks fit max_blocks and its length an int32, its tokens (if any) fit n_slots
 * and the stack still holds all
 * the new blocks it needs (once the stack is short, later rows that need
 * none are still served); a negative length leaves a row unserved, with no
 * tokens.  Writes, with q_start[r] the sum of the q_lens before r:
 *  - block_table: a served row's new entries; all others keep their values,
 *  - seq_lens [n_rows]: ctx + q of a served row, ctx (0 if negative) of others,
 *  - q_start [n_rows + 1],
 *  - slot_map [n_slots]: token i of row r goes to slot
 *    block * block_size + offset, at q_start[r] + i; -1 for the tokens of
 *    unserved rows, past the last row, and where a block id that the table
 *    holds is negative or gives no int32,
 *  - *n_free_out: blocks left on the stack, *n_unserved: rows not served.
 * Outputs must not overlap inputs (n_free_out is not n_free).  Rows of
 * block_table are table_stride entries apart.  *n_free is read as at most
 * free_cap, the entries of free_list.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int moe_kv_plan(void* stream, const int32_t* ctx_lens, const int32_t* q_lens, int n_rows,
                int32_t* block_table, int64_t table_stride, int max_blocks,
                const int32_t* free_list, int free_cap, const int32_t* n_free, int block_size,
                int32_t* seq_lens, int32_t* q_start, int32_t* slot_map, int n_slots,
                int32_t* n_free_out, int32_t* n_unserved);

/* Give back the blocks of finished rows: for every row with finished[r] != 0,
 * in row order, its ceil(seq_lens[r] / block_size) blocks are pushed on the
 * stack free_list[0 .. *n_free) and seq_lens[r] becomes 0.  *n_free_out is the
 * stack's new height (n_free_out may be n_free); pushes past free_cap are
 * dropped.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int moe_kv_release(void* stream, const uint8_t* finished, int n_rows, int32_t* seq_lens,
                   const int32_t* block_table, int64_t table_stride, int max_blocks,
                   int32_t* free_list, int free_cap, const int32_t* n_free, int block_size,
                   int32_t* n_free_out);

/* The same for rows that keep a part: a row that is not finished and has 0 <=
 * keep_lens[r] < seq_lens[r] gives back the blocks from entry
 * ceil(keep_lens[r] / block_size) of its block_table row on, and seq_lens[r]
 * becomes keep_lens[r]; a keep_lens[r] below 0 or not below seq_lens[r] leaves
 * the row as it is.  finished or keep_lens may be NULL, not both.  This is how
 * a row gets shorter (rejected drafts): moe_kv_plan takes a row to hold the
 * blocks of its ctx_lens and no more, so that a length lowered without this
 * call loses the blocks past it. */
int moe_kv_release_past(void* stream, const uint8_t* finished, const int32_t* keep_lens,
                        int n_rows, int32_t* seq_lens, const int32_t* block_table,
                        int64_t table_stride, int max_blocks, int32_t* free_list, int free_cap,
                        const int32_t* n_free, int block_size, int32_t* n_free_out);

/* Write the keys and values of n_tokens new tokens into the cache.  k, v
 * device [n_tokens][n_kv_heads][head_dim] of `dtype` (BF16 or F16), token and
 * head strides in elements (multiples of 8; pointers 16-byte aligned), rows
 * contiguous.  slot_map device [n_tokens]: block * block_size + offset per
 * token; -1 (or any slot outside the cache) skips the token.  The tokens a
 * step writes into one block follow one another in the slot map at consecutive
 * ascending offsets, with nothing but skipped tokens between them (then the
 * offsets need only ascend) and within block_size entries, and the block holds
 * the sequence's earlier tokens below them (what moe_kv_plan makes).  Per
 * block, head and side: e is the smallest
 * integer with max |finite value| <= 448 * 2^e, at least -60, at most 60; a
 * block that already held tokens keeps its exponent if that is larger, and
 * otherwise has their codes rounded to the new one.  Codes are value / 2^e
 * rounded to the nearest E4M3 (ties to even), past 448 (infinities too) to
 * 448; NaN stays NaN.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int moe_kv_append(void* stream, const moe_kv_cache_t* cache, const void* k, const void* v,
                  int dtype, int64_t k_token_stride, int64_t k_head_stride,
                  int64_t v_token_stride, int64_t v_head_stride, const int32_t* slot_map,
                  int n_tokens);

/* Attention of new tokens over the cache.  Row r's queries are tokens
 * q_start[r] .. q_start[r + 1) of q, the last of its seq_lens[r] cached tokens
 * (query i of n sits at position p = seq_len - n + i; their keys are in the
 * cache already).  Query head h reads KV head h / (n_heads / n_kv_heads).  A
 * query sees the keys j < seq_len with j <= p (causal != 0) and j > p - window
 * (window > 0), and not those of a block id outside the cache:
 *   out = sum_j softmax_j(scale * q . k_j) v_j,  lse = ln sum_j exp(scale * q . k_j)
 * (out 0 and lse -infinity when it sees none).  Keys and values it does not
 * see do not reach its result, whatever they hold.  Products and sums are
 * exact products summed in fp32; lse's sum takes its terms in fp32, whatever
 * the scales.  A key's weight in the second product, its probability times its
 * block's V scale, is rounded to f16 beside the row's largest: to 2^-11 of
 * itself down to 2^-21 of that one, to 2^-32 of that one below.
 * max_blocks * block_size and n_tokens * n_heads are below 2^31 - 128.  seq_lens is read as at most
 * max_blocks * block_size and q_start as within
 * [0, n_tokens], not descending; rows of q past q_start[n_rows] are left
 * alone.  max_q, the longest row's queries as the host knows it, only picks
 * the kernel: any value gives the same result up to rounding.  The tensor-core
 * kernel's waits between its warps are bounded: one that runs out (none does on a
 * device that works) leaves NaN in the rows it was for. */
typedef struct {
  const void* q;            /* device [n_tokens][n_heads][head_dim] */
  int64_t q_token_stride, q_head_stride;      /* elements, multiples of 8 */
  void* out;                /* device, the same shape and type */
  int64_t out_token_stride, out_head_stride;  /* elements, multiples of 8 */
  float* lse;               /* device [n_tokens][n_heads], or NULL */
  const int32_t* block_table;                 /* device [n_rows][max_blocks] */
  int64_t table_stride;
  const int32_t* seq_lens;  /* device [n_rows] */
  const int32_t* q_start;   /* device [n_rows + 1] */
  void* workspace;          /* device, moe_kv_attention_workspace bytes, 256-byte aligned */
  size_t workspace_bytes;
  int32_t dtype;            /* BF16 or F16 */
  int32_t n_rows, n_tokens, n_heads, max_blocks, max_q;
  int32_t causal;
  int32_t window;           /* 0: none */
  float scale;
} moe_kv_attention_t;

/* Errors: INVALID_ARG, UNSUPPORTED, ALLOC (workspace too small), CUDA.  The
 * workspace holds nothing between calls; calls that overlap need one each. */
int moe_kv_attention(void* stream, const moe_kv_cache_t* cache, const moe_kv_attention_t* args);

/* Bytes of workspace moe_kv_attention needs on the current device, whatever
 * the lengths (0 on error). */
size_t moe_kv_attention_workspace(int head_dim);

/* Expert routing from logits, for any number of rows.  Per row: score s_e =
 * sigmoid(l_e) or softmax(l)_e in fp32 (all of a softmax row at -infinity:
 * scores 0); experts are compared by s_e + bias_e (bias NULL: s_e), the sum
 * rounded to fp32, with the very s_e that the weights are made of.  With
 * n_groups > 1 the experts form n_groups equal consecutive groups, a group
 * counts with the sum of its group_top (1 or 2) best, and only the experts of
 * the topk_groups best groups are left.  The top_k best are written in
 * descending order; ties, of groups too, go to the lower index, and a NaN
 * comes after everything else.  Weights are the unbiased scores, divided by
 * their sum if renormalize (0 when the sum is 0), times routed_scale. */
typedef struct {
  int32_t n_experts;        /* <= 1024, a multiple of n_groups */
  int32_t top_k;            /* <= 32, <= topk_groups * (n_experts / n_groups) */
  int32_t scoring;          /* 0 sigmoid, 1 softmax */
  int32_t n_groups, topk_groups, group_top;   /* n_groups <= 32 */
  int32_t renormalize;
  float routed_scale;
} moe_route_t;

/* logits device [n_rows][n_experts] of `dtype`, rows row_stride elements
 * apart; bias device fp32 [n_experts] or NULL; idx device int32 and w device
 * fp32 [n_rows][top_k].  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int moe_route(void* stream, const moe_route_t* cfg, const void* logits, int dtype,
              int64_t row_stride, int64_t n_rows, const float* bias, int32_t* idx, float* w);

/* ---- 8-bit products, norms and the experts of any number of rows ----
 * What a prompt, or more than the layer's 64 rows, needs around the routing:
 * the norm with the residual's addition, 8-bit activations, products with
 * 8-bit or MXFP4 weights, dense or by expert, and the sorting of tokens by
 * expert and the weighted sum that go with them (no counterpart in the pages;
 * the formulas are stated at each call).  The rules of the serving operators
 * hold: no handle, asynchronous on `stream`, nothing allocated, no host
 * synchronisation, capturable; what the host can see is checked, values read
 * on the device are bounded there.  None of them needs a workspace.
 *
 * 8-bit activations are E4M3 codes [rows][d] with one E8M0 scale per (row, 128
 * columns), [rows][ceil(d / 128)]: code * 2^(scale - 127).  They are made so: e
 * is the smallest integer with max |finite value| <= 448 * 2^e over the 128, at
 * least -126 and at most 120 (an all-zero block: -126); a code is value / 2^e
 * rounded to the nearest E4M3 (ties to even), infinities to 448; NaN stays NaN.
 * 8-bit weights [n][k] have one scale per (128 rows, 128 columns).  The sums of
 * products are in fp32. */

/* More types, of outputs here only. */
enum { MOE_DTYPE_E4M3 = 3 };

/* Norm of rows, with a residual's addition: z = x + residual (fp32; x alone
 * where residual is NULL), residual <- z rounded to dtype, y = z / sqrt(mean(z^2)
 * + eps) * gamma from the unrounded z; out <- y rounded to dtype, codes and
 * scales <- y in 8 bits.  out may be NULL, or codes and scales, not all; out may
 * be x. */
typedef struct {
  const void* x;            /* device [n_rows][d] */
  int64_t x_stride;         /* elements, as all strides here; multiples of 8 */
  void* residual;           /* device [n_rows][d], read and written, or NULL */
  int64_t residual_stride;
  const void* gamma;        /* device [d] */
  void* out;                /* device [n_rows][d], or NULL */
  int64_t out_stride;
  uint8_t* codes;           /* device [n_rows][d], or NULL */
  int64_t codes_stride;
  uint8_t* scales;          /* device [n_rows][ceil(d / 128)] */
  int64_t scales_stride;    /* any */
  int64_t n_rows;
  int32_t d;                /* a multiple of 8, <= 16384 */
  int32_t dtype;            /* of x, residual and out: BF16, F16 or F32 */
  int32_t gamma_dtype;      /* BF16, F16 or F32 */
  float eps;
} moe_rms_norm_t;

/* Pointers 16-byte aligned (codes 8, scales any).  Errors: INVALID_ARG,
 * UNSUPPORTED, CUDA. */
int moe_rms_norm(void* stream, const moe_rms_norm_t* args);

/* The 8-bit form of x device [n_rows][d] of dtype BF16, F16 or F32. */
int moe_fp8_quantize(void* stream, const void* x, int dtype, int64_t x_stride, int64_t n_rows,
                     int d, uint8_t* codes, int64_t codes_stride, uint8_t* scales,
                     int64_t scales_stride);

/* The 8-bit form of weights: n_mat matrices w device [n][k] of dtype BF16, F16
 * or F32, back to back -> codes [n_mat][n][k], scales [n_mat][ceil(n / 128)]
 * [ceil(k / 128)], by the activations' rule over 128 x 128. */
int moe_fp8_pack(void* stream, const void* w, int dtype, int64_t n_mat, int64_t n, int64_t k,
                 uint8_t* codes, uint8_t* scales);

typedef enum {
  MOE_WEIGHTS_E4M3 = 0,     /* codes [n][k], scales [ceil(n / 128)][ceil(k / 128)] */
  MOE_WEIGHTS_MXFP4 = 1     /* canonical (layout 0): q [n][k / 2], scales [n][k / 32] */
} moe_weight_format;

typedef enum {
  MOE_ACT_NONE = 0,         /* out[., j] = p[., j] */
  MOE_ACT_SWIGLU = 1        /* out[., j] = silu(p[., j]) * p[., n / 2 + j]: gates, then ups
                             * (silu 0 below -87.3, where it is less than 1.1e-36) */
} moe_activation;

/* Products of 8-bit activations with 8-bit or MXFP4 weights: p[i, j] = sum_k
 * x[src(i), k] w[j, k].  With offsets NULL there is one matrix, n_experts is 1
 * and src(i) = i, or rows[i].  With offsets, output rows offsets[e] ..
 * offsets[e + 1) go through matrix e (a moe_dispatch's offsets); output rows
 * outside these are left alone, and offsets are read as within [0, n_rows], one
 * below an earlier one as that one.  rows[i], the row of x that output row i
 * reads, is read as within [0, x_rows).  out_dtype E4M3 (SWIGLU only) writes
 * the 8-bit form of the result: codes in out, scales in out_scales.  The
 * kernel's waits between its warps are bounded: one that runs out (none does on
 * a device that works) leaves NaN (8 bits: codes or scales of NaN) in its tile of
 * the output, 256 columns (SWIGLU: 128) of up to 240 rows, and in what the same
 * CTAs had still to do. */
typedef struct {
  const uint8_t* x;         /* device [x_rows][k], 16-byte aligned */
  int64_t x_stride;         /* a multiple of 16 */
  const uint8_t* x_scales;
  int64_t x_scales_stride;
  const uint8_t* w;         /* device [n_experts][n][k or k / 2], 16- (MXFP4: 32-) byte aligned */
  int64_t w_stride, w_expert_stride;   /* bytes, multiples of 16 (MXFP4: 32) */
  const uint8_t* w_scales;
  int64_t w_scales_stride, w_scales_expert_stride;
  const int32_t* offsets;   /* device [n_experts + 1], or NULL */
  const int32_t* rows;      /* device [n_rows], or NULL */
  void* out;                /* device [n_rows][n, or n / 2 with SWIGLU] */
  int64_t out_stride;       /* elements */
  uint8_t* out_scales;      /* E4M3: device [n_rows][ceil(n / 2 / 128)] */
  int64_t out_scales_stride;
  int32_t n_rows, x_rows, n, k;   /* k a multiple of 16 (MXFP4: 128) */
  int32_t n_experts;        /* <= 1024 */
  int32_t w_format, activation, out_dtype;   /* BF16, F16, F32 or E4M3 */
} moe_fp8_product_t;

/* Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int moe_fp8_product(void* stream, const moe_fp8_product_t* args);

/* Failure-detection test hook of moe_fp8_product: with fault = n > 0, in this
 * process's later calls pair n - 1 of the kernel's CTAs brings no weights (nor rows
 * that are not by index) to its tiles, and every wait is limited to wait_ns
 * nanoseconds (0: the default 2 s), so that the waits for them run out.  fault = 0
 * restores normal operation.  Nothing on the GPU traps, faults or hangs.  Errors:
 * INVALID_ARG. */
int moe_debug_set_product_fault(int fault, unsigned long long wait_ns);

/* Tokens by expert, from the choices idx device [n_tokens][top_k]: choice (t, j)
 * of an expert in [0, n_experts) is one entry; entries are ordered by expert,
 * and by t, then j, within one.  offsets [n_experts + 1]: each expert's first
 * entry; rows [n_tokens * top_k]: the token of each entry, -1 past the last;
 * slots [n_tokens][top_k]: the entry of each choice, -1 where idx names no
 * expert.  n_experts <= 1024, n_tokens * top_k <= 2^24.  Errors: INVALID_ARG,
 * UNSUPPORTED, CUDA. */
int moe_dispatch(void* stream, const int32_t* idx, int n_tokens, int top_k, int n_experts,
                 int32_t* offsets, int32_t* rows, int32_t* slots);

/* Weighted sums of the experts' rows: out[t] = residual[t] + sum_j w[t, j]
 * y[slots[t, j]], in fp32 in the order of j and rounded once; residual may be
 * NULL (0) or out; slots outside [0, y_rows) count 0.  y [y_rows][d], residual
 * and out [n_tokens][d] of dtype BF16, F16 or F32, 16-byte aligned, strides in
 * elements, multiples of 8, as is d; w fp32 and slots [n_tokens][top_k], top_k
 * <= 32.  Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
typedef struct {
  const void* y;
  int64_t y_stride;
  const float* w;
  const int32_t* slots;
  const void* residual;
  int64_t residual_stride;
  void* out;
  int64_t out_stride;
  int32_t n_tokens, top_k, y_rows, d, dtype;
} moe_combine_t;

int moe_combine(void* stream, const moe_combine_t* args);

/* Human-readable name of a status code (static string). */
const char* moe_status_string(int status);

/* The last CUDA error code a call saw (cudaError_t as int), 0 if none. */
int moe_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DECODE_H */
