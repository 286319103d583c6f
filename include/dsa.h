/*
 * dsa.h - C ABI of the GB300 (sm_103a) DSA sparse MLA attention library (libdsa_gb300.so).
 *
 * What the library computes is defined by sglang PR #38547 "Enable zero-RoPE TileLang DSA on
 * gfx950":
 *   - Summary / Contract table: the 256+0 latent geometry (256-wide NoPE latent, zero-width
 *     RoPE tail; Q [tokens, 64, 256], KV [slots, 1, 256], output BF16 [tokens, 64, 256]) and
 *     the DeepSeek-style 512+64 layout kept as a control (d_v = 512, 64-wide RoPE tail);
 *   - Contract table, "scaled FP8 cache row": 264 bytes = 256 e4m3 + 2 fp32 scales + 0 RoPE,
 *     656 bytes = 512 e4m3 + 4 fp32 scales + 64 bf16 RoPE values;
 *   - Scope list: quant_k_cache (pack rows), dequant_k_cache (direct, paged, gather/dequant);
 *   - Direct GLM geometry coverage list: top-k widths 2048 / 2112, rows padded with -1, the
 *     reference computation (gather the rows, mask padding, score, softmax, weight the rows),
 *     and repeated runs that agree bit for bit.
 *
 * Conventions for every entry point:
 *   - All pointers are DEVICE pointers unless stated otherwise; the caller owns all memory.
 *     The library allocates nothing and keeps no per-call state, so calls on different
 *     streams may run concurrently when they use different output/workspace buffers.
 *   - Work is enqueued on `stream` (a cudaStream_t passed as void*; NULL = legacy default
 *     stream) and runs asynchronously. The return value reports host-side argument checks and
 *     launch errors only. Problems found on the device (an index that addresses no slot, a
 *     bounded wait that timed out) are OR-ed into the optional device word `error_word`
 *     (DSA_DEVERR_* bits), which the caller reads after synchronising.
 *   - bf16 tensors are IEEE bfloat16 bit patterns (uint16); all strides are in elements.
 *   - On error nothing is launched and no output is written.
 */
#ifndef DSA_GB300_H
#define DSA_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define DSA_API __attribute__((visibility("default")))
#else
#define DSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARGUMENT = 1,   /* null pointer, negative size, bad stride or alignment */
  DSA_ERR_UNSUPPORTED = 2,        /* a geometry or head count this build has no kernel for */
  DSA_ERR_WORKSPACE_TOO_SMALL = 3,
  DSA_ERR_CUDA = 4,               /* a CUDA runtime/driver call failed (see dsa_last_cuda_error) */
  DSA_ERR_NO_DEVICE = 5           /* the current device is not an sm_103 GPU */
} dsa_status_t;

/* Bits OR-ed into the optional device error word. */
#define DSA_DEVERR_INDEX_OUT_OF_RANGE 0x1  /* an index / page addressed no slot: entry masked */
#define DSA_DEVERR_TIMEOUT 0x2             /* a bounded device-side wait gave up */
#define DSA_DEVERR_SLOT_OUT_OF_RANGE 0x4   /* quant_k_cache: out_loc outside [0, num_slots): row skipped */
#define DSA_DEVERR_REQUEST_ORDER 0x8       /* paged_attn_mass: a request named twice or out of order: token skipped */
#define DSA_DEVERR_OUT_OF_PAGES 0x10       /* batch_plan: the free pages do not suffice: request refused */
#define DSA_DEVERR_TOKEN_CAPACITY 0x20     /* batch_plan: more new tokens than room for them: request refused */

typedef enum {
  DSA_CACHE_BF16 = 0,        /* bf16 latent rows [num_slots, d_nope + d_rope] */
  DSA_CACHE_FP8_SCALED = 1   /* packed rows [num_slots, dsa_packed_row_bytes(d_nope, d_rope)] uint8 */
} dsa_cache_kind_t;

/* Human-readable name of a status code (static string). */
DSA_API const char* dsa_status_string(dsa_status_t status);

/* The CUDA error code (cudaError_t as int) behind the last DSA_ERR_CUDA of this thread. */
DSA_API int dsa_last_cuda_error(void);

/* Bytes of one packed scaled-FP8 row: d_nope codes + 4 * (d_nope / 128) scale bytes +
 * 2 * d_rope RoPE bytes (Contract table: 264 for 256+0, 656 for 512+64). Returns -1 when
 * d_nope is not a positive multiple of 128 or d_rope < 0. */
DSA_API int64_t dsa_packed_row_bytes(int d_nope, int d_rope);

/* Bytes of one cache row of the given kind (bf16 rows: 2 * (d_nope + d_rope)). */
DSA_API int64_t dsa_cache_row_bytes(dsa_cache_kind_t kind, int d_nope, int d_rope);

/*
 * dsa_quant_k_cache - pack latent rows into the scaled-FP8 cache (quant_k_cache, Scope list;
 * memory_pool write sites). For row i and each 128-element tile j of its NoPE part:
 *   amax = max |x|, scale = amax / 448 (fp32), code = e4m3_rne_satfinite(x / scale) (one IEEE
 *   fp32 division per element; an all-zero tile stores scale 0 and codes 0),
 * written to slot out_loc[i] (or slot i when out_loc is NULL) as
 *   [d_nope codes][d_nope/128 fp32 scales, little endian][d_rope bf16 RoPE values, copied].
 *   k_nope        bf16 [n, d_nope], row i at k_nope + i * k_nope_row_stride (stride >= d_nope, even)
 *   k_rope        bf16 [n, d_rope], row i at k_rope + i * k_rope_row_stride; NULL iff d_rope == 0
 *   out_loc       int64 [n] destination slots, or NULL; a slot outside [0, num_slots) skips the row
 *                 and sets DSA_DEVERR_SLOT_OUT_OF_RANGE
 *   cache         uint8 [num_slots, row_bytes], 8-byte aligned base
 * Supported: d_nope in {256, 512}, d_rope in {0, 64}. n == 0 is a no-op.
 */
DSA_API dsa_status_t dsa_quant_k_cache(const void* k_nope, int64_t k_nope_row_stride, const void* k_rope,
                               int64_t k_rope_row_stride, int64_t n, int d_nope, int d_rope,
                               const int64_t* out_loc, void* cache, int64_t num_slots,
                               int32_t* error_word, void* stream);

/*
 * dsa_gather_dequant - gather latent rows by index and widen them to bf16 (dequant_k_cache:
 * direct, paged and gather/dequant paths; Contract table "paged dequant/gather").
 *   indices       int32 [n]; an entry < 0 yields a zero row
 *   block_table   int32 [R, bt_stride] physical page of each logical page, or NULL (direct mode:
 *                 the index is the slot). Paged: slot = block_table[r, i / page_size] * page_size
 *                 + i % page_size with r = req_of_index[k] (0 when req_of_index is NULL) and
 *                 i < max_pages * page_size.
 *   out           bf16 [n, d_nope + d_rope] (contiguous). FP8 rows: bf16_rne(fp32(e4m3(code)) * scale),
 *                 RoPE bits copied; BF16 rows: copied.
 * An index that addresses no slot yields a zero row and sets DSA_DEVERR_INDEX_OUT_OF_RANGE.
 */
DSA_API dsa_status_t dsa_gather_dequant(const void* cache, dsa_cache_kind_t kind, int64_t num_slots,
                                int d_nope, int d_rope, const int32_t* indices, int64_t n,
                                const int32_t* block_table, int64_t bt_stride, int page_size,
                                int max_pages, const int32_t* req_of_index, void* out,
                                int32_t* error_word, void* stream);

/*
 * dsa_gather_requant - gather packed scaled-FP8 rows by index and pack them again
 * (dequant_k_cache: the gather/dequant/requant path; PR #38547, its production-file list). Row i
 * of the result is exactly dsa_quant_k_cache applied to the bf16 row dsa_gather_dequant returns
 * for indices[i]: each gathered tile is widened to bf16_rne(fp32(e4m3(code)) * scale), then
 * re-packed (new amax, scale = amax / 448, codes = e4m3_rne_satfinite(x / scale)); RoPE bits are
 * copied. A masked index (< 0), or one that addresses no slot (which also sets
 * DSA_DEVERR_INDEX_OUT_OF_RANGE), packs the all-zero row.
 *   cache         uint8 [num_slots, row_bytes] packed rows (8-byte aligned base)
 *   indices, block_table, bt_stride, page_size, max_pages, req_of_index: as for dsa_gather_dequant
 *   out_loc       int64 [n] destination row of each result in `out`, or NULL (row i); a row
 *                 outside [0, out_slots) is skipped and sets DSA_DEVERR_SLOT_OUT_OF_RANGE
 *   out           uint8 [out_slots, row_bytes] (8-byte aligned base); may not overlap `cache`
 * Supported: d_nope in {256, 512}, d_rope in {0, 64}. n == 0 is a no-op.
 */
DSA_API dsa_status_t dsa_gather_requant(const void* cache, int64_t num_slots, int d_nope, int d_rope,
                                const int32_t* indices, int64_t n, const int32_t* block_table,
                                int64_t bt_stride, int page_size, int max_pages,
                                const int32_t* req_of_index, const int64_t* out_loc, void* out,
                                int64_t out_slots, int32_t* error_word, void* stream);

/*
 * dsa_topk_select - the top-k position list of each query token from its index-logits, the
 * input dsa_sparse_attn gathers by (FreeToken PR #270 "glm5_next: support GLM-5.3-Flash",
 * Summary, the DSA key-pooling bullet: pooled keys are scored and the best-scoring positions
 * read; PR #38547, Direct GLM geometry coverage list: top-k widths 2048 and 2112, lists padded
 * with -1). The pages give the scoring itself no formula: the scores are an input.
 *   scores        fp32 [T, S], row t at scores + t * score_stride_t (stride >= S); finite or
 *                 +-inf (NaN is outside the contract); may be NULL when S == 0
 *   lengths       int32 [T] positions each row considers (0 .. n_t - 1, n_t = lengths[t]
 *                 clamped to [0, S]: a causal limit), or NULL (n_t = S)
 *   K             result width, 1 .. 16384
 *   indices       int32 [T, K] at indices + t * idx_stride_t (stride >= K): the positions of the
 *                 min(K, n_t) largest scores of row t in descending score order, equal scores
 *                 in ascending position order (-0.0 equals +0.0), then -1 up to K
 * The result depends only on the inputs (integer decisions on order-preserving keys). T == 0 is
 * a no-op; errors: DSA_ERR_INVALID_ARGUMENT (sizes, strides, null or misaligned pointers),
 * DSA_ERR_UNSUPPORTED (S above 2^31 - 1).
 */
DSA_API dsa_status_t dsa_topk_select(const float* scores, int64_t T, int64_t S, int64_t score_stride_t,
                             const int32_t* lengths, int K, int32_t* indices, int64_t idx_stride_t,
                             void* stream);

/* Arguments of dsa_sparse_attn. Zero-initialise, then fill. */
typedef struct dsa_attn_args {
  const void* q;                 /* bf16 [T, H, d_nope + d_rope]; element (t,h,d) at
                                    q + t*q_stride_t + h*q_stride_h + d; 16-byte aligned base,
                                    strides multiples of 8 elements */
  int64_t q_stride_t, q_stride_h;
  int64_t T;                     /* query tokens (0 = no-op) */
  int H;                         /* heads: 64 */
  const void* cache;             /* BF16 rows or packed FP8 rows, see dsa_cache_kind_t */
  dsa_cache_kind_t kind;
  int64_t num_slots;
  int d_nope, d_rope, d_v;       /* (256, 0, 256) or (512, 64, 512) */
  const int32_t* indices;        /* int32 [T, topk] at indices + t*idx_stride_t; < 0 = masked */
  int64_t idx_stride_t;
  int topk;                      /* 1 .. 16384 */
  const int32_t* block_table;    /* int32 [R, bt_stride] or NULL (direct slots) */
  int64_t bt_stride;
  int page_size, max_pages;
  const int32_t* req_of_token;   /* int32 [T] request of each token, or NULL (request 0) */
  float sm_scale;                /* softmax scale applied to q.k: any finite value (0 gives the
                                    mean of the valid rows, a negative value is allowed) */
  void* out;                     /* bf16 [T, H, d_v]; (t,h,d) at out + t*out_stride_t + h*out_stride_h + d */
  int64_t out_stride_t, out_stride_h;
  float* lse;                    /* optional fp32 [T, H] natural-log sum of exp(scores); NULL ok */
  void* workspace;               /* device scratch of dsa_sparse_attn_workspace_size bytes,
                                    zero-filled before its first use. A call tags the merge flags
                                    it sets with a per-workspace counter and clears every flag it
                                    consumes before it ends, so the workspace needs no clearing
                                    between calls (zero-fill it again after a call that reported
                                    DSA_DEVERR_TIMEOUT). One call at a time per workspace. */
  size_t workspace_bytes;
  int32_t* error_word;           /* optional device int32; DSA_DEVERR_* bits are OR-ed in */
} dsa_attn_args_t;

/*
 * dsa_sparse_attn_workspace_size - bytes of workspace dsa_sparse_attn needs for these arguments
 * on the current device (depends on the device's SM count and d_v only).
 */
DSA_API dsa_status_t dsa_sparse_attn_workspace_size(const dsa_attn_args_t* args, size_t* bytes);

/*
 * dsa_sparse_attn - DSA sparse MLA attention forward (the TileLang BF16 "partial" kernel and
 * the FP8 kernel of the Scope list, re-designed for sm_103a). For every token t and head h:
 *   valid entries j: indices[t, j] >= 0 (translated through block_table in paged mode);
 *   k_j = the latent row (BF16 as stored; FP8: e4m3 code * tile scale, RoPE bf16 as stored);
 *   s_j = sm_scale * dot(q[t,h,:], k_j), p = softmax_j(s), out[t,h,:] = sum_j p_j * k_j[0:d_v];
 *   lse[t,h] = log(sum_j exp(s_j)). A token with no valid entry gets out = 0 and lse = -inf.
 * Duplicate indices are separate terms. The result is bit-identical across repeated calls with
 * the same inputs on the same device.
 * Arithmetic. BF16 rows: products of bf16 operands accumulated in fp32 (tensor cores);
 * probabilities enter the value product as bf16. 256+0 FP8 rows: 8-bit tensor-core products
 * accumulated in fp32; the e4m3 codes enter exactly, the bf16 query as two e4m3 terms per head
 * and 128-column tile (a power-of-two scale each; exact for every component within 2^9 of the
 * tile's largest), the fp32 tile scales multiply the score accumulators, and the probabilities
 * (times each key's tile scale) enter the value product as two e4m3 terms, 8 significant bits.
 * The keys are thus the exact products code * scale (never rounded to bf16). 512+64 FP8 rows:
 * keys are bf16_rne(code * scale), the rows dsa_gather_dequant returns.
 */
DSA_API dsa_status_t dsa_sparse_attn(const dsa_attn_args_t* args, void* stream);

/*
 * dsa_sparse_attn_static_ws - dsa_sparse_attn for callers that cannot allocate device memory.
 * (The pages have no counterpart: this is a deployment variant of the same computation.)
 *
 * Who needs it: callers that have no device allocator to offer, or may not use one when they
 * call: serving engines that reserve all device memory up front for their KV page pool and
 * hand libraries only input and output buffers, runtimes that work from a fixed memory plan,
 * and latency-critical paths where an allocation could stall or synchronise the device. This
 * entry point takes no workspace (args->workspace and workspace_bytes are ignored): its
 * split-token scratch lives in a fixed device array inside the library, about 10.6 MB, enough
 * for the partial results of up to 160 CTAs. Every GPU that loads the library holds that array
 * until the process exits. The call allocates nothing.
 *
 * Arguments, results and errors are those of dsa_sparse_attn; the result is identical to
 * dsa_sparse_attn's on GPUs with at most 160 SMs. On a GPU with more SMs the kernel runs on 160
 * CTAs; if the array could not hold the scratch of the launch the call returns
 * DSA_ERR_WORKSPACE_TOO_SMALL without launching.
 *
 * The first call on each device does one-time set-up: it looks up the array's device address
 * (cudaGetSymbolAddress) and sets the attention kernels' shared-memory limits on that device.
 * All calls share the one array,
 * which keeps what the last call left there: a call tags the flags it sets with a fresh value
 * and clears every flag it consumes, so nothing has to be cleared between calls. Two calls
 * whose kernels overlap on the GPU (different streams, no ordering between them) race on the
 * array: order such calls, or use dsa_sparse_attn with separate workspaces.
 */
DSA_API dsa_status_t dsa_sparse_attn_static_ws(const dsa_attn_args_t* args, void* stream);

/*
 * FP8 block-scaled projection GEMM, for the dense MLA projections around the attention
 * (sglang PR #31955 "Opt-in prefill-only FP8 dense projection GEMM for MLA q_b/o_proj",
 * Motivation and Modifications: weights repacked into e4m3 with one UE8M0 (power-of-two) scale
 * per 128x128 block, activations quantised per token and 128-column group, "a8w8 blockscale").
 *
 * dsa_blockscale_bytes - bytes of the scale tensor of a [rows, cols] matrix (cols a multiple of
 * 128): ceil(rows / 128) * (cols / 128) * 512; -1 for invalid sizes.
 *
 * dsa_quant_fp8_blockscale - quantise bf16 x [rows, cols] (row stride in elements, a multiple
 * of 8; cols a multiple of 128) into e4m3 codes [rows, cols] (uint8, contiguous) and scales.
 * block_rows = 128 (weights: 128 x 128 blocks) or 1 (activations: 1 x 128 blocks). Per block,
 * e = the smallest integer in [-127, 127] with 448 * 2^e >= max |x| (0 for an all-zero block) and
 * code = e4m3 round-to-nearest-even of x / 2^e (exact; nothing saturates). The UE8M0 bytes e + 127
 * are stored in the GEMM's 32-element block-scale layout: each 128-column block is four equal
 * 32-column scales; tiles of 128 rows x 4 scale columns (512 bytes; row r, scale column c at
 * (r % 32) * 16 + ((r % 128) / 32) * 4 + c % 4) in row-tile-major order. Scales of rows past
 * `rows` in the last tile read 127 (scale 1). Inputs must be finite. Pointers 16-byte aligned.
 *
 * dsa_proj_gemm - y[m, n] = sum_k x[m, k] w[n, k] over the dequantised operands (x from
 * block_rows = 1, w [N, K] from block_rows = 128), fp32 accumulation, bf16 output y [M, N] with
 * row stride y_stride (elements, a multiple of 8). N and K multiples of 128. The product runs in
 * cuBLASLt (e4m3 operands with 32-element UE8M0 block scales); `workspace` (256-byte aligned,
 * may be NULL with workspace_bytes 0) is its scratch. Calls on one device are serialised on the
 * host (the library keeps one cuBLASLt handle and a plan cache per device).
 */
DSA_API int64_t dsa_blockscale_bytes(int64_t rows, int64_t cols);
DSA_API dsa_status_t dsa_quant_fp8_blockscale(const void* x, int64_t rows, int64_t cols, int64_t row_stride,
                                              int block_rows, void* codes, void* scales, void* stream);
DSA_API dsa_status_t dsa_proj_gemm(const void* x_codes, const void* x_scales, const void* w_codes,
                                   const void* w_scales, int64_t M, int64_t N, int64_t K, void* y, int64_t y_stride,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Dense attention over the paged latent cache: one new token per request (decode), over every
 * position of a range instead of a top-k list, with the two operators that shrink a cache by the
 * attention its positions receive. Geometry 256+0 (d_nope = d_v = 256), both cache kinds.
 *
 * Positions. Request r's position j is the cache row slot(r, j) = block_table[r, j / page_size] *
 * page_size + j % page_size, or slot j when block_table is NULL (direct mode). Token t reads the
 * positions starts[t] <= j < lengths[t] of request req_of_token[t]. A range past the addressable
 * positions (max_pages * page_size; num_slots in direct mode; the row width of key_positions or
 * of the mass), a page that addresses no slot, or a request outside [0, num_requests) sets
 * DSA_DEVERR_INDEX_OUT_OF_RANGE, and the positions concerned are masked. Rows outside the range
 * are never used, whatever they hold.
 *
 * Scores, natural units, for head h and position j:
 *   u = sm_scale * dot(q[t,h,:], k_j)
 *   u = logit_cap * tanh(u / logit_cap)                       when logit_cap > 0
 *   u = u - slopes[h] * |qpos_t - kpos_rj|                    when slopes != NULL
 * with qpos_t = q_positions[t] (lengths[t] - 1 when NULL) and kpos_rj = key_positions[r, j] (j
 * when NULL; a cache that evicted positions keeps them out of order, dsa_cache_evict).
 * A document mask is a range (starts[t] = the document's first position); a causal or a prefix
 * mask over several tokens of a request is lengths[t].
 * Arithmetic: keys are exact (bf16 as stored; FP8 code * tile scale, the codes exact in the
 * products and the fp32 scales applied to the fp32 accumulators); with an FP8 cache the bf16 query
 * enters as two e4m3 terms per head (a power-of-two scale each; exact for every component within 2^9
 * of the head's largest, and within 2^-17 of the largest otherwise); scores, softmax statistics and
 * sums in fp32; the probabilities enter the value product as bf16 (FP8: times the key's tile scale,
 * as f16: 11 bits down to 2^-22 of the largest such weight of the head and tile so far; largest weights
 * below 2^-80, or 2^40 below that of another of the same 16 heads, count as that). The value products'
 * fp32 sums truncate: within n * 2^-22 of sum p |k| for n positions. Results are
 * bit-identical across repeated calls with the same inputs on one device.
 */
typedef struct dsa_paged_args {
  const void* q;                 /* bf16 [T, H, 256], 16-byte aligned, strides multiples of 8 */
  int64_t q_stride_t, q_stride_h;
  int64_t T;                     /* query tokens, at most 2^24 (0 = no-op); T * ceil(H / 64) *
                                    (addressable positions / 128 + 2) below 2^31 */
  int H;                         /* heads: 1 .. 128 */
  const void* cache;             /* contiguous rows, 16-byte aligned */
  dsa_cache_kind_t kind;
  int64_t num_slots;
  int d_nope, d_rope, d_v;       /* (256, 0, 256) */
  const int32_t* block_table;    /* int32 [num_requests, bt_stride] or NULL (direct slots) */
  int64_t bt_stride;
  int page_size, max_pages;
  int64_t num_requests;          /* rows of block_table, key_positions and mass */
  const int32_t* req_of_token;   /* int32 [T], or NULL: token t belongs to request t */
  const int32_t* starts;         /* int32 [T], or NULL: 0; a negative entry counts as 0 */
  const int32_t* lengths;        /* int32 [T]; lengths[t] <= starts[t]: nothing to read */
  const int32_t* q_positions;    /* int32 [T] or NULL */
  const int32_t* key_positions;  /* int32 [num_requests, kp_stride] or NULL */
  int64_t kp_stride;
  int64_t kp_width;              /* entries of a key_positions row */
  float sm_scale;                /* any finite value */
  float logit_cap;               /* 0: none; else positive and finite; the capped score errs by less than
                                    2^-20 of itself, whatever the cap's size */
  const float* slopes;           /* fp32 [H] or NULL */
  void* out;                     /* bf16 [T, H, 256], 16-byte aligned, strides multiples of 8 */
  int64_t out_stride_t, out_stride_h;
  float* lse;                    /* fp32 [T, H] natural log sum of exp(u): optional output of
                                    dsa_paged_attn, input of dsa_paged_attn_mass */
  void* workspace;               /* device scratch of dsa_paged_attn_workspace_size bytes, 256-byte
                                    aligned, of any content. Calls whose kernels may overlap on
                                    the GPU need separate ones (two captured graphs included). */
  size_t workspace_bytes;
  int32_t* error_word;           /* optional device int32; DSA_DEVERR_* bits are OR-ed in */
} dsa_paged_args_t;

/* Bytes of workspace dsa_paged_attn needs on the current device (T and H of the args count). */
DSA_API dsa_status_t dsa_paged_attn_workspace_size(const dsa_paged_args_t* args, size_t* bytes);

/*
 * dsa_paged_attn - out[t,h,:] = sum_j softmax_j(u) k_j over the token's range, and lse[t,h] when
 * asked for. A token with nothing to read gets out = 0 and lse = -inf. Tokens may share a request.
 */
DSA_API dsa_status_t dsa_paged_attn(const dsa_paged_args_t* args, void* stream);

/*
 * dsa_paged_attn_mass - the attention weight each cached position received, summed over heads:
 *   mass_out[r, j] = mass[r, j] + sum_h exp(u[h, j] - lse[t, h])   for the positions j of token t's range,
 * r its request; every other entry of mass_out is left as it is. args->lse [T, H] is the input
 * (dsa_paged_attn's on the same arguments); out and workspace are not used.
 *   mass          fp32 [num_requests, mass_width], row stride mass_stride
 *   mass_out      the same shape, row stride mass_out_stride: equal to mass (in place) or disjoint
 * Each request at most once and in ascending order (req_of_token strictly ascending, or NULL):
 * a token whose request does not exceed every earlier one is skipped and sets
 * DSA_DEVERR_REQUEST_ORDER. Masked positions add nothing, but are copied.
 */
DSA_API dsa_status_t dsa_paged_attn_mass(const dsa_paged_args_t* args, const float* mass, int64_t mass_stride,
                                         float* mass_out, int64_t mass_out_stride, int64_t mass_width, void* stream);

/*
 * dsa_cache_evict - shrink every request to its budget, keeping the positions of largest mass, in
 * place in the paged cache. For request r with n = lengths[r] and b = budgets[r] (budget when
 * budgets is NULL; a negative one counts as 0), n > b:
 *   kept        the b positions of the largest mass, ties to the lower position; the first `sink`
 *               token positions (kpos < sink) and the `recent` newest (kpos > max kpos - recent)
 *               rank as +inf. kpos_j = positions[r, j], j when positions is NULL. NaN is outside
 *               the contract (any order, but b are kept).
 *   moved       the i-th kept position >= b, in ascending order, moves to the i-th evicted
 *               position < b: its cache row, mass and kpos. Nothing else moves, so the rows of
 *               [0, b) hold the kept positions, not in order of age.
 *   mass_out    [r, 0 .. b): the kept masses; [r, b .. n): 0
 *   positions_out [r, 0 .. b): the kept kpos (optional when positions is NULL)
 *   lengths_out [r] = b
 * A request with n <= b keeps all: mass_out and positions_out [r, 0 .. n) are copies, lengths_out
 * n. Entries at or past n are left as they are. Each output may be its input (in place) or disjoint.
 * A request whose n exceeds `width` or the addressable positions, or with a page among its n
 * positions that addresses no slot, keeps all as well and sets DSA_DEVERR_INDEX_OUT_OF_RANGE
 * (only its first min(n, width) entries are copied).
 * The pages of a request that is shrunk must be its own, each named once among its n positions: a
 * page that another request also names would change under it, and rows of a page named twice would
 * move over one another (give such a request a budget of at least its length).
 * Cache rows of both kinds and both geometries (256+0, 512+64). Direct mode (block_table NULL)
 * takes one request. Bit-identical across repeated calls.
 */
typedef struct dsa_evict_args {
  void* cache;                   /* contiguous rows, 8-byte aligned */
  dsa_cache_kind_t kind;
  int64_t num_slots;
  int d_nope, d_rope;
  const int32_t* block_table;    /* int32 [num_requests, bt_stride] or NULL (direct slots) */
  int64_t bt_stride;
  int page_size, max_pages;
  int64_t num_requests;          /* at most 65535 (0 = no-op) */
  const int32_t* lengths;        /* int32 [num_requests] */
  const int32_t* budgets;        /* int32 [num_requests] or NULL */
  int budget;                    /* used when budgets is NULL: >= 0 (0 evicts every position) */
  int sink, recent;              /* >= 0 */
  int64_t width;                 /* entries of a row of mass and positions: 1 .. 2^30 */
  const float* mass;             /* fp32 [num_requests, width] */
  int64_t mass_stride;
  const int32_t* positions;      /* int32 [num_requests, width] or NULL */
  int64_t positions_stride;
  float* mass_out;
  int64_t mass_out_stride;
  int32_t* positions_out;
  int64_t positions_out_stride;
  int32_t* lengths_out;          /* int32 [num_requests] */
  void* workspace;               /* dsa_cache_evict_workspace_size bytes, any content; one call at
                                    a time per workspace */
  size_t workspace_bytes;
  int32_t* error_word;
} dsa_evict_args_t;

DSA_API dsa_status_t dsa_cache_evict_workspace_size(int64_t num_requests, int64_t width, size_t* bytes);
DSA_API dsa_status_t dsa_cache_evict(const dsa_evict_args_t* args, void* stream);

/*
 * A serving step around the paged cache: the batch plan that brings block tables to the requests'
 * lengths, the norms and the rotation of queries and keys with the cache write, and the selection
 * of the blocks (a block = a page of positions) that each token attends to. In turn: dsa_batch_plan
 * -> dsa_qk_norm_rope -> dsa_block_pool -> dsa_block_scores -> dsa_block_select -> dsa_paged_attn
 * over the selected table; dsa_cache_evict shrinks lengths, and the next plan takes its pages back.
 * An eviction closes the gaps it leaves, so the j-th cached position of a request holds its j-th token
 * only until the first one. Where the cache is told by its positions (means, scores, choice, lengths),
 * the plan's `positions` and `token_lengths` say it; where a token's place in its sequence counts (the
 * rotation, the attention's q_positions and key_positions), `token_positions` does, with `seen`.
 * Results are bit-identical across repeated calls with the same inputs on one device.
 */

/*
 * dsa_batch_plan - block tables and slot maps of a step, from request lengths on the device. For
 * request r with l = lengths[r] cached positions, h = held[r] pages in its table row and
 * n = new_tokens[r]:
 *   n < 0       the request ends: its length becomes 0
 *   n >= 0      its length becomes l + n
 *   need        ceil(new length / page_size) pages
 *   need < h    pages block_table[r, need .. h) go onto the free stack (the entries stay as they are)
 *   need > h    block_table[r, h .. need) are taken from the top of the free stack
 * The free stack is free_pages[0 .. *num_free), its last entry the top. Pages given back are put on
 * it first, requests in order and pages in order, so this call may take them; then pages are taken,
 * requests in order and pages in order. A request is refused when need > max_pages or l + n exceeds
 * 2^31 - 1 (DSA_DEVERR_INDEX_OUT_OF_RANGE); or, of the requests not refused by that, when it takes
 * pages and it and those before it want more pages than there are (DSA_DEVERR_OUT_OF_PAGES), or
 * when it adds tokens and it and those before it add more than T (DSA_DEVERR_TOKEN_CAPACITY). A
 * refused request adds no token and takes no page; its length and seen stay, and pages past need still
 * go back. What it wanted still counts for those behind it: a request too large for the step holds up
 * every later one that takes a page or adds a token, until the caller leaves it out (new_tokens 0).
 * Negative lengths and held count as 0, held past max_pages as max_pages, *num_free as clamped to
 * [0, free_capacity]. Pages that find no room on the stack are dropped and set
 * DSA_DEVERR_SLOT_OUT_OF_RANGE.
 * Pages that go back must be the request's own. The plan does not look for one that another request
 * holds too (a shared prefix): each would give it back, and it would be handed out twice, to requests
 * that then write over each other's rows, with no error bit. A request whose first s pages are shared
 * must keep at least s * page_size positions; to end it, set its length to that with new_tokens 0, which
 * gives the pages behind them back, then set its length and held to 0. The shared pages go back with
 * the last request that holds them.
 * The tokens that requests add are numbered in order of requests and positions, i = 0, 1, ...:
 *   cu_tokens     [R + 1]: the first token of each request, and the number of all
 *   req_of_token  [T], positions [T] (the token's position among its request's cached ones),
 *                 token_lengths [T] (position + 1: what the token attends to), out_loc int64 [T] (the
 *                 cache slot of its position; -1 for a page < 0). Entries behind the last token: request
 *                 0, position -1, length 0, slot -1, which every operator skips (dsa_quant_k_cache
 *                 with its error bit for such a slot).
 * Where an eviction has shortened requests, a token's place in its sequence is not its position any
 * more. `seen` counts the tokens that each request has been given: the i-th of this step's has place
 * seen + i, and seen becomes seen + n (0 when the request ends; a negative one counts as 0; l + i and
 * l when NULL). A request whose seen + n exceeds 2^31 - 1, or that adds tokens to more than kp_width
 * positions, is refused (DSA_DEVERR_INDEX_OUT_OF_RANGE).
 *   token_positions  [T]: the token's place, -1 behind the last token
 *   key_positions    [r, position] = place of every new token (the other entries stay: dsa_cache_evict
 *                    moves them with the rows as its positions, in place)
 * Each of lengths_out, held_out, num_free_out and seen_out may be its input (in place) or disjoint; the
 * block table and the free stack change in place. Zero-initialise the struct, then fill.
 */
typedef struct dsa_plan_args {
  int64_t num_requests;          /* at most 2^20 */
  const int32_t* lengths;        /* int32 [num_requests] */
  const int32_t* new_tokens;     /* int32 [num_requests] */
  const int32_t* held;           /* int32 [num_requests] */
  int32_t* block_table;          /* int32 [num_requests, bt_stride] */
  int64_t bt_stride;
  int page_size, max_pages;
  int32_t* free_pages;           /* int32 [free_capacity] */
  int64_t free_capacity;         /* at most 2^31 - 1 */
  const int32_t* num_free;       /* int32 [1] */
  int32_t* lengths_out;          /* int32 [num_requests] */
  int32_t* held_out;             /* int32 [num_requests] */
  int32_t* num_free_out;         /* int32 [1] */
  int64_t T;                     /* room for tokens: at most 2^30 */
  int32_t* cu_tokens;            /* int32 [num_requests + 1] */
  int32_t* req_of_token;         /* int32 [T] */
  int32_t* positions;            /* int32 [T] */
  int32_t* token_lengths;        /* int32 [T] */
  int64_t* out_loc;              /* int64 [T] */
  int32_t* error_word;
  const int32_t* seen;           /* int32 [num_requests] or NULL */
  int32_t* seen_out;             /* int32 [num_requests]; unused without seen */
  int32_t* token_positions;      /* int32 [T] or NULL */
  int32_t* key_positions;        /* int32 [num_requests, kp_width] or NULL */
  int64_t kp_stride;
  int64_t kp_width;
} dsa_plan_args_t;

DSA_API dsa_status_t dsa_batch_plan(const dsa_plan_args_t* args, void* stream);

/*
 * dsa_qk_norm_rope - the norm of every query head and of the latent key, the rotation of their
 * RoPE columns and the key's cache row, in one pass. A row x of d_nope + d_rope columns becomes
 *   y_d = x_d * rsqrt(mean_{d < n} x_d^2 + eps) * weight_d      for the first n columns
 * (n = q_norm for queries, k_norm for keys: 0 leaves them as they are, d_nope, or all; weight 1
 * when NULL), then, when cos_sin is given, the last d_rope columns turn by the token's angles
 * (positions: its place in the sequence, the plan's token_positions where the cache evicts):
 *   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs (i, i + d_rope / 2), or (2 i, 2 i + 1) when interleaved,
 * with cos = cos_sin[positions[t], i] and sin = cos_sin[positions[t], d_rope / 2 + i]. Everything is
 * in fp32 and rounded once: queries to bf16, the key's row as the cache holds it (bf16, or packed as
 * dsa_quant_k_cache packs, from the unrounded row; but a tile of NaN, or of zeros and NaN, keeps its
 * NaN as codes: a NaN under the norm makes all normalised columns NaN; and a tile whose scale rounds
 * to zero, largest value below 448 * 2^-150, is zeros). Sums of squares must stay below the fp32 range.
 * A token with a negative position is padding: nothing of it is read or written. A position at or
 * past num_positions skips the token and sets DSA_DEVERR_INDEX_OUT_OF_RANGE. A key whose out_loc is
 * negative is not written; one at or past num_slots is not either and sets
 * DSA_DEVERR_SLOT_OUT_OF_RANGE. Slots of one call must differ.
 * Geometries 256+0 and 512+64. q_out may be q (in place, equal strides) or disjoint.
 */
typedef struct dsa_qk_args {
  int64_t T;                     /* tokens, at most 2^24 (0 = no-op) */
  int d_nope, d_rope;
  const void* q;                 /* bf16 [T, H, d_nope + d_rope], 16-byte aligned, strides multiples
                                    of 8; NULL: keys only */
  int64_t q_stride_t, q_stride_h;
  int H;                         /* 1 .. 128 (unused without q) */
  void* q_out;                   /* bf16, the shape of q */
  int64_t q_out_stride_t, q_out_stride_h;
  int q_norm;
  const void* q_weight;          /* bf16 [q_norm], 16-byte aligned, or NULL */
  const void* k;                 /* bf16 [T, d_nope + d_rope], 16-byte aligned, stride a multiple of
                                    8; NULL: queries only */
  int64_t k_stride_t;
  int k_norm;
  const void* k_weight;          /* bf16 [k_norm], 16-byte aligned, or NULL */
  void* cache;                   /* contiguous rows, 16-byte aligned (unused without k) */
  dsa_cache_kind_t kind;
  int64_t num_slots;
  const int64_t* out_loc;        /* int64 [T], or NULL: token t's key goes to slot t */
  float eps;                     /* positive and finite */
  const int32_t* positions;      /* int32 [T], or NULL (not with cos_sin): no padding */
  const float* cos_sin;          /* fp32 [num_positions, cs_stride], or NULL: no rotation */
  int64_t cs_stride;             /* >= d_rope */
  int64_t num_positions;
  int interleaved;
  int32_t* error_word;
} dsa_qk_args_t;

DSA_API dsa_status_t dsa_qk_norm_rope(const dsa_qk_args_t* args, void* stream);

/*
 * dsa_block_pool - the mean row of each block that tokens of this step lie in (geometry 256+0):
 *   summary[page] = bf16(mean of the cached rows of the block's positions below lengths[r])
 * for the block positions[t] / page_size of request r = req_of_token[t] (request t when NULL) of
 * every token t, page = block_table[r, block]. Rows in fp32 (FP8: code * tile scale), summed in a
 * fixed order. Negative positions are skipped. A request or page that does not exist, a position
 * at or past max_pages * page_size, a block without a position below lengths[r] or with rows past
 * num_slots sets DSA_DEVERR_INDEX_OUT_OF_RANGE and is skipped. Requests of one call that share a page
 * must have equally many positions in it: it has one summary.
 *   cache         contiguous rows, 16-byte aligned; num_slots below 2^31
 * (dsa_cache_evict moves rows between blocks: make the summaries of what is left anew, by positions 0 .. length - 1.)
 *   lengths       int32 [num_requests], with this step's tokens
 *   summary       bf16 [num_pages, 256], 16-byte aligned; the summaries of other pages stay as they are
 */
DSA_API dsa_status_t dsa_block_pool(const void* cache, dsa_cache_kind_t kind, int64_t num_slots,
                                    const int32_t* block_table, int64_t bt_stride, int page_size, int max_pages,
                                    int64_t num_requests, const int32_t* positions, const int32_t* req_of_token,
                                    int64_t T, const int32_t* lengths, void* summary, int64_t num_pages,
                                    int32_t* error_word, void* stream);

/*
 * dsa_block_scores - a cheap score of each block for each token:
 *   scores[t, b] = sum_h w[t,h] * max(0, sm_scale * dot(q[t,h,:], summary[block_table[r, b]]))
 * for the blocks b < ceil(lengths[t] / page_size) of the token's request r; other entries of scores
 * are left as they are. w = weights, or 1 when NULL. bf16 products (exact) accumulated in fp32 on
 * the tensor cores, the sum over heads in fp32 (of w * sm_scale times the products' positive
 * part). The tensor cores' sums truncate: a score is within 2^-15 * sum_h |w| sm_scale sum_d |q_d s_d|
 * + (H + 2) * 2^-24 * sum_h |w| sm_scale max(0, q.s) of its formula. NaN passes through the maximum. A block whose page does not
 * exist scores -inf and sets DSA_DEVERR_INDEX_OUT_OF_RANGE, as do blocks at or past max_pages or
 * width (not scored) and a request that does not exist (its token is skipped).
 * Causality: a token's own block, and with several tokens of a request in one call the blocks after
 * it, hold rows the token must not see. Blocks after it are not scored (lengths[t]); its own block
 * has to be selected whatever its score (recent >= 1 below).
 *   q             bf16 [T, H, 256], 16-byte aligned, strides multiples of 8; H 1 .. 128, T <= 2^24
 *   summary       bf16 [num_pages, 256], 16-byte aligned
 *   req_of_token  int32 [T], or NULL: token t belongs to request t. Neighbouring tokens of one
 *                 request share the reads of its summaries.
 *   lengths       int32 [T]: the positions each token attends to
 *   sm_scale      positive and finite
 *   weights       fp32 [T, H] or NULL
 *   scores        fp32 [T, width], row stride score_stride >= width; width 1 .. 2^24
 */
DSA_API dsa_status_t dsa_block_scores(const void* q, int64_t q_stride_t, int64_t q_stride_h, int64_t T, int H,
                                      const void* summary, int64_t num_pages, const int32_t* block_table,
                                      int64_t bt_stride, int page_size, int max_pages, int64_t num_requests,
                                      const int32_t* req_of_token, const int32_t* lengths, float sm_scale,
                                      const float* weights, float* scores, int64_t score_stride, int64_t width,
                                      int32_t* error_word, void* stream);

/*
 * dsa_block_select - the K best blocks of each token, as a block table of the token's own. Of the
 * n = ceil(lengths[t] / page_size) blocks of token t, m = min(K, n) are chosen: the first `sink`,
 * the last `recent`, and of the others those of the largest score (ties to the lower block; -0.0
 * equals +0.0; NaN is outside the contract, but m are chosen).
 *   blocks        int32 [T, K]: the chosen blocks in ascending order, then -1 (NULL: not wanted)
 *   table         int32 [T, K]: their pages, block_table[r, block], then -1
 *   lengths_out   int32 [T]: the positions of the chosen blocks, where the token's last block counts
 *                 those below lengths[t] only: it comes last, so dsa_paged_attn(q, cache, table,
 *                 lengths_out) with one table row per token attends to exactly these positions. (Its
 *                 distance bias wants key_positions of the same order.)
 * A request that does not exist chooses nothing; it and a token with more blocks than max_pages or
 * width (the excess is left out, its last block then counting as full) set
 * DSA_DEVERR_INDEX_OUT_OF_RANGE.
 *   scores        fp32 [T, width], row stride score_stride >= width; width 1 .. 2^24
 *   K             1 .. 16384; sink, recent >= 0 with sink + recent <= K
 *   T             at most 2^24 (0 = no-op)
 */
DSA_API dsa_status_t dsa_block_select(const float* scores, int64_t score_stride, int64_t width, int64_t T,
                                      const int32_t* block_table, int64_t bt_stride, int page_size, int max_pages,
                                      int64_t num_requests, const int32_t* req_of_token, const int32_t* lengths, int K,
                                      int sink, int recent, int32_t* blocks, int64_t blocks_stride, int32_t* table,
                                      int64_t table_stride, int32_t* lengths_out, int32_t* error_word, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_GB300_H */
