/*
 * qkvp.h - C ABI of libqkvp: paged MLA decode attention that reads a quantized latent KV cache
 * (FP8 E4M3 or NVFP4) directly, for NVIDIA GB300 (sm_103a). Next to it: the appends that apply the
 * rotary position embedding on the way into a cache, and decode attention over a paged 8-bit cache of
 * K and V heads (gqa_*), whole or through a sliding window with sink tokens.
 *
 * The problem, as the source pages state it:
 *  - Each token stores one 576-wide latent: kv_lora_rank 512 ("nope") + qk_rope_head_dim 64. All
 *    query heads share it. Attention uses K = the whole latent and V = its first 512 dims ("The
 *    Smoking Gun: Tracing the FP8-to-BF16 KV Cache Cast", section "The Investigation Leading to This
 *    Message": pool shape [495552, 1, 576]).
 *  - The pool is paged and addressed through a CSR page table (qo_indptr, kv_indptr, kv_indices,
 *    kv_len_arr), with num_heads, kv_lora_rank, qk_rope_head_dim, page_size, sm_scale and the KV
 *    dtype given to a host-side plan() before a device-side run() ("The Smoking Gun", section
 *    "What Message 1408 Actually Reveals").
 *  - The KV cache is FP8 E4M3 (float8_e4m3fn; "The FP8 KV Cache Wall", section "Context and
 *    Motivation") or NVFP4: E2M1 values, one E4M3 scale per 16 values, one FP32 global scale per
 *    tensor ("SGLang x Qwen x NVIDIA ... NVFP4 KV Cache", section "NVFP4 format").
 *  - Decode reads the quantized pages directly and dequantizes inside the kernel; nothing casts the
 *    pool to BF16 first (same page, section "SGLang implementation", item 3).
 *
 * Memory layout (all device buffers are caller-owned; the library allocates no device memory. Its
 * only global state: per device, four pinned host staging buffers and events for the work table
 * upload of mla_decode_plan, and the fixed device scratch array of mla_decode_noalloc with its
 * static host table):
 *  - slot s = page * page_size + offset; page_size must be 64.
 *  - FP8 pool  : kv_data uint8 [num_pages][64][576], one E4M3 byte per latent element. The decode
 *                entry points read kv_data (any pool type) with 32-byte loads: it must be 32-byte aligned.
 *  - NVFP4 pool: kv_data uint8 [num_pages][64][288] packed E2M1 pairs (element 2k in the low nibble
 *                of byte k, 2k+1 in the high nibble) and kv_scale uint8 [num_pages][64][36] E4M3
 *                block scales (block j covers elements 16j..16j+15). 324 bytes per token = 9/16 of
 *                FP8. An element decodes to global_scale * scale(block) * e2m1(code).
 *  - FP8 pool with per-token scales (QKVP_KV_FP8_PER_TOKEN): kv_data uint8 [num_pages][37120]:
 *                page p holds the 64 token rows of 576 E4M3 codes (bytes 0..36863), then the 64
 *                FP32 token scales (bytes 36864..37119, little-endian). 580 bytes per token. An
 *                element decodes to scale(token) * e4m3(code). The layout is the pages' indexer key
 *                cache (FP8 elements + 4 scale bytes per token in a paged [npages, page_bytes] uint8
 *                buffer, 64 tokens per page: "The Precision Frontier: Implementing bf16 Index Keys",
 *                section "The Message: Planning the bf16-K Implementation") carrying the latent.
 *  - BF16 pool : kv_data uint16 [num_pages][64][576] (the cast-then-attend baseline only).
 *  - head pool (gqa_*): kv_data uint8 [num_pages][2][num_kv_heads][64][head_dim], the K blocks of a
 *                page and then its V blocks, one code per element (qkvp_cache_dtype), and kv_scale
 *                float [num_pages][2][num_kv_heads], one scale per (page, K or V, head). An element
 *                decodes to kv_scale(block) * value(code). 2 * num_kv_heads * (64 * head_dim + 4)
 *                bytes per page.
 *  - q         : bf16 [batch][num_heads][576], row-major, contiguous.
 *  - out       : bf16 [batch][num_heads][512], 16-byte aligned (the attend kernels store 16-byte
 *                vectors); lse: float [batch][num_heads] (natural log), or NULL.
 *
 * Errors: every call returns an int status (qkvp_status). Arguments are checked before anything is
 * launched; a failed check launches nothing. QKVP_E_CUDA reports a CUDA error from a launch or copy
 * issued by the call. Faults that occur asynchronously inside a kernel surface at the caller's next
 * synchronisation. Indices read from device memory (slot ids, page ids) are bounds-checked in the
 * kernels: out-of-range entries are skipped (append) or read as masked tokens (decode); they never
 * cause an out-of-bounds access.
 *
 * Streams: `stream` is a cudaStream_t (NULL = the legacy default stream). Calls are asynchronous
 * with respect to the host unless stated. The library is re-entrant across distinct streams and
 * workspaces.
 */
#ifndef QKVP_H_
#define QKVP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* qkvp_stream_t; /* identical to cudaStream_t */

typedef enum {
  QKVP_OK = 0,
  QKVP_E_INVALID = -1,     /* bad argument: null pointer, negative size, inconsistent page table */
  QKVP_E_UNSUPPORTED = -2, /* valid but not supported: page size, head count, dtype combination */
  QKVP_E_WORKSPACE = -3,   /* workspace missing or smaller than plan->workspace_bytes */
  QKVP_E_CUDA = -4         /* a CUDA runtime call or launch failed */
} qkvp_status;

typedef enum {
  QKVP_KV_FP8_E4M3 = 1,
  QKVP_KV_NVFP4 = 2,
  QKVP_KV_BF16 = 3,
  QKVP_KV_FP8_PER_TOKEN = 4
} qkvp_kv_dtype;
typedef enum { QKVP_SRC_FP8_E4M3 = 1, QKVP_SRC_BF16 = 2 } qkvp_src_dtype;

/* Decode kernel families. AUTO lets the planner choose. */
typedef enum {
  QKVP_ALGO_AUTO = 0,
  QKVP_ALGO_MMA_SYNC = 1,  /* warp-level mma.sync split-KV kernel, any supported head count */
  QKVP_ALGO_TCGEN05 = 2,   /* tcgen05/TMEM CTA-pair split-KV kernel: always 128 head rows (fewer heads
                              ride as zero rows), so its cost does not shrink with the heads; AUTO picks
                              it above 64 heads (from 64 for BF16 pools) */
  QKVP_ALGO_MMA_FP8 = 3,   /* the mma.sync kernel with Q.K^T on the FP8 tensor-core path, for FP8 and
                              per-token-scaled FP8 pools (others: QKVP_E_UNSUPPORTED): K is the page's
                              E4M3 bytes as stored, Q is split per head row into two E4M3 terms,
                              q ~ (hi + lo / 16) / sc with sc = 2^floor(log2(448 / max|q|)),
                              hi = E4M3(q sc), lo = E4M3(16 (q sc - hi)), and the two products are
                              summed in FP32; P.V stays FP16. The pages' decode dequantizes "to FP8 or
                              BF16" ("SGLang x Qwen x NVIDIA ... NVFP4 KV Cache", section "SGLang
                              implementation", item 3); a single E4M3 term for Q (or for P) misses
                              the output tolerance on the outlier-channel workloads, two terms for Q
                              meet it. 16 or 32 heads per CTA. On GB300 it takes 1.5-1.8x the
                              time of QKVP_ALGO_MMA_SYNC (two MMAs per 32 dims, and the legacy FP8
                              MMA path gains no rate over FP16), so AUTO never picks it. */
  QKVP_ALGO_TCGEN05_TOKENS = 4 /* tcgen05/TMEM kernel with the page's tokens as the rows of both
                              products (M = 64 tokens for Q.K^T, M = 128 output dims for P.V) and the
                              heads as the columns (N = 16, 32 or 64; 48 heads ride in 64): 16 to 64
                              heads, FP8, NVFP4 and per-token-scaled FP8 pools (others:
                              QKVP_E_UNSUPPORTED); one CTA per SM. Same arithmetic and tolerance as
                              the other families. AUTO picks it for quantized pools at 32 to 64 heads,
                              where it measured fastest on GB300 (FP8 44 x 32K at 32 / 64 heads:
                              287 / 405 us against 311 / 495 us for the other families; NVFP4 1M:
                              236 / 333 against 347 / 361 us). At 16 heads the mma.sync kernel is
                              faster. */
} qkvp_algo;

/* Code type of a head pool. E4M3: as in the FP8 pools. INT8: two's complement codes in [-127, 127]. */
typedef enum { QKVP_CACHE_E4M3 = 1, QKVP_CACHE_INT8 = 2 } qkvp_cache_dtype;
/* Which dims of a head's first r dims the rotary embedding turns as pair i (i < r / 2):
 * HALVES (x[i], x[i + r/2]), PAIRS (x[2i], x[2i + 1]). */
typedef enum { QKVP_ROPE_HALVES = 0, QKVP_ROPE_PAIRS = 1 } qkvp_rope_style;

#define QKVP_LATENT_DIM 576
#define QKVP_V_DIM 512
#define QKVP_PAGE_SIZE 64

/* Host-side plan produced by mla_decode_plan and consumed by mla_decode_run. Plain data: it may be
 * copied, and one plan serves any number of runs (e.g. one per layer) with the same page table,
 * lengths, head count and KV dtype, as long as the workspace it was uploaded to is left intact. */
typedef struct {
  int32_t batch, num_heads, page_size, kv_dtype;
  int32_t algo;              /* the kernel family the plan was made for */
  int32_t num_workers;       /* independent split-KV workers (one CTA pair or CTA group each) */
  int32_t ctas_per_worker;   /* CTAs that cooperate on one worker's token ranges */
  int32_t num_segments;      /* (request, page range) pieces; each writes one partial or output */
  int32_t num_split_requests;/* requests whose pages span more than one segment (need a combine) */
  int32_t num_empty_requests;/* requests with no tokens (output 0, lse -inf) */
  int32_t max_worker_pages;  /* most pages given to one worker (load balance) */
  int32_t min_worker_pages;  /* fewest pages given to one worker */
  int32_t num_partials;      /* FP32 split partials held in the workspace */
  int32_t max_request_segments; /* most segments one request is cut into */
  int32_t num_wide_requests; /* requests cut into more than 8 segments: the combine gives each of
                                them several CTAs per head instead of one thread per 8 output dims */
  int64_t total_pages;       /* sum over requests of ceil(len / 64) */
  int64_t total_tokens;      /* sum of lengths */
  uint64_t workspace_bytes;  /* device workspace the run needs (table + split partials) */
  uint64_t table_bytes;      /* bytes of the work table at the start of the workspace */
  uint64_t partial_o_offset; /* byte offset of the FP32 partial outputs in the workspace */
  uint64_t partial_lse_offset;
  uint64_t status_offset;    /* int32 device status word in the workspace: 0 after planning; a
                                decode kernel that gave up waiting on its own pipeline (a bug, never
                                expected) sets bits in it, and its outputs are then undefined */
  uint64_t magic;            /* set by a successful plan; checked by run */
} qkvp_plan;

/*
 * kv_append_quant - quantize-on-append: write n_tokens new latent rows into the paged pool.
 *
 * Source: "SGLang x Qwen x NVIDIA ... NVFP4 KV Cache", section "SGLang implementation", items 1-2
 * (quantize KV from FP8 into NVFP4 and write it to the persistent cache); section "NVFP4 format"
 * (two-level scaling). For an FP8 pool: E4M3 storage of the latent ("The FP8 KV Cache Wall").
 *
 *  src          device, [n_tokens][576]: E4M3 bytes (src_dtype QKVP_SRC_FP8_E4M3) or BF16
 *               (QKVP_SRC_BF16).
 *  slot_mapping device int64 [n_tokens]: destination slot page * page_size + offset; a negative slot
 *               skips the token; a slot >= num_pages * page_size is skipped too.
 *  kv_data      device pool (layout above) for kv_dtype QKVP_KV_FP8_E4M3, QKVP_KV_NVFP4 or
 *               QKVP_KV_FP8_PER_TOKEN.
 *  kv_scale     device NVFP4 block-scale pool; must be NULL for the FP8 pools.
 *  global_scale NVFP4 decode multiplier g (> 0, finite): an element decodes to g * s * e. Must be
 *               1.0 for the FP8 pools.
 *
 * FP8 pool: FP8 sources are copied; BF16 sources round to nearest even, saturating at +-448; NaN
 * gives 0x7F. NVFP4 pool, per block of 16 consecutive elements x (FP32 arithmetic, one rounding per
 * operation): amax = max|x| (NaN if any x is NaN); s8 = E4M3(amax / (6 g)) rounded to nearest even
 * and saturated; sd = value(s8) * g; codes = 0 where sd == 0, else E2M1(x / sd) rounded to nearest
 * even and saturated at +-6 (NaN gives 0). FP8 pool with per-token scales, per token x (FP32
 * arithmetic, one rounding per operation): amax = max|x|; scale = amax / 448, or the NaN 0x7FC00000
 * if any x is NaN; codes = E4M3(x / scale) rounded to nearest even and saturated (NaN gives 0x7F),
 * or E4M3(x) (a signed zero) when scale == 0. The stored bytes are bit-identical to the CPU oracle.
 * If two tokens of one call name the same slot, that row is unspecified: it may mix what they bring.
 */
int kv_append_quant(const void* src, int32_t src_dtype, int64_t n_tokens,
                    const int64_t* slot_mapping, void* kv_data, uint8_t* kv_scale,
                    int32_t kv_dtype, float global_scale, int32_t page_size, int64_t num_pages,
                    qkvp_stream_t stream);

/*
 * mla_decode_plan - split the batch's pages into balanced work for the decode kernel.
 *
 * Source: the plan/run split and CSR page table of the pages' plan() call ("The Smoking Gun",
 * section "What Message 1408 Actually Reveals"). The split-KV decomposition itself is not on the
 * pages; its partial results are merged by log-sum-exp in mla_decode_run.
 *
 *  kv_indptr_host host int32 [batch + 1], in pages: request r owns kv_indices[kv_indptr[r] ..
 *                 kv_indptr[r+1]). Must start at 0 and be non-decreasing.
 *  kv_len_host    host int32 [batch], tokens per request; ceil(len / 64) must not exceed the
 *                 request's page count. len 0 is allowed (output 0, lse -inf).
 *  num_heads      query heads: a multiple of 16 in [16, 128].
 *  page_size      must be 64.
 *  num_sms        streaming multiprocessors to plan for; <= 0 queries the current device (a CUDA
 *                 runtime call, also in query mode).
 *  min_splits     lower bound on the number of segments (e.g. 148 to spread one long request over
 *                 every SM); 0 for none.
 *  algo           a qkvp_algo; QKVP_ALGO_AUTO picks the fastest supported family.
 *  workspace      device buffer that receives the work table; NULL makes this a pure host query
 *                 that only fills *plan (including plan->workspace_bytes) and touches no device.
 *  stream         stream of the table upload: an asynchronous copy from one of four library-owned
 *                 pinned buffers (per device, reused once its previous copy has completed), so the
 *                 call does not wait for earlier work on the stream and the host arrays may be
 *                 reused as soon as it returns. If pinned memory is refused it copies from
 *                 pageable memory instead (staged by the runtime before the call returns).
 *
 * Returns QKVP_E_WORKSPACE (with plan->workspace_bytes filled) when workspace is non-NULL but
 * smaller than needed, and QKVP_E_UNSUPPORTED when workspace is non-NULL and `stream` is being
 * captured into a CUDA graph: the upload reads host memory that belongs to this call only, so a
 * replayed graph would read it after it is gone. Plan outside capture; mla_decode_run,
 * mla_decode_attend and mla_decode_combine only launch kernels and may be captured.
 */
int mla_decode_plan(const int32_t* kv_indptr_host, const int32_t* kv_len_host, int32_t batch,
                    int32_t num_heads, int32_t page_size, int32_t kv_dtype, int32_t num_sms,
                    int32_t min_splits, int32_t algo, void* workspace, uint64_t workspace_bytes,
                    qkvp_stream_t stream, qkvp_plan* plan);

/*
 * mla_decode_run - paged MLA decode attention over the quantized pool, for one layer.
 *
 * Computes, per request r and head h over its tokens t < len_r (in natural-log terms),
 *   z_t = sm_scale * g * sum_{d<576} q[r,h,d] * k_t[d]
 *   out[r,h,v] = g * sum_t softmax(z)_t * k_t[v] (v < 512),   lse[r,h] = log sum_t exp(z_t)
 * where k_t is the dequantized latent without the global scale g (g = 1 for FP8 and BF16 pools;
 * "SGLang x Qwen x NVIDIA ... NVFP4 KV Cache", section "SGLang implementation", item 3: the global
 * scale enters through the matrix-multiply scaling, not per element). The kernels dequantize in
 * registers and run Q.K^T and P.V on the tensor cores with FP16 operands and FP32 accumulation:
 * every dequantized K/V value is exact in FP16, Q is converted from BF16 exactly (a row holding a
 * value of 2^15 or more is first scaled by a power of two, folded into the logit scale), and the
 * probabilities P keep 11 mantissa bits. The softmax runs online in FP32; each segment writes one
 * partial, and partials are merged by log-sum-exp.
 *
 *  plan       from mla_decode_plan with the same kv_dtype, uploaded into this workspace.
 *  q          device bf16 [batch][num_heads][576].
 *  kv_data    device pool for plan->kv_dtype; kv_scale the NVFP4 scale pool (NULL otherwise).
 *  num_pages  pages in the pool; page ids outside [0, num_pages) read as masked tokens.
 *  kv_indices device int32 page ids addressed by the plan's kv_indptr.
 *  sm_scale   logit scale (finite); global_scale: NVFP4 g (> 0, finite), must be 1.0 otherwise.
 *  out, lse   outputs (lse may be NULL).
 *  workspace  the buffer given to mla_decode_plan, at least plan->workspace_bytes.
 */
int mla_decode_run(const qkvp_plan* plan, const void* q, const void* kv_data,
                   const uint8_t* kv_scale, int64_t num_pages, const int32_t* kv_indices,
                   float sm_scale, float global_scale, void* out, float* lse, void* workspace,
                   uint64_t workspace_bytes, qkvp_stream_t stream);

/*
 * mla_decode_attend / mla_decode_combine - the two halves of mla_decode_run, for callers that
 * schedule or time them separately. attend runs the split-KV decode kernel: requests covered by a
 * single segment get their final out/lse, the others leave FP32 partials (normalised output and
 * base-2 log-sum-exp) in the workspace. combine merges those partials by log-sum-exp into out/lse
 * and writes zeros / -inf for empty requests. combine must follow attend on the same stream with
 * the same plan, workspace, global_scale, out and lse. Arguments as for mla_decode_run.
 */
int mla_decode_attend(const qkvp_plan* plan, const void* q, const void* kv_data,
                      const uint8_t* kv_scale, int64_t num_pages, const int32_t* kv_indices,
                      float sm_scale, float global_scale, void* out, float* lse, void* workspace,
                      uint64_t workspace_bytes, qkvp_stream_t stream);
int mla_decode_combine(const qkvp_plan* plan, float global_scale, void* out, float* lse,
                       void* workspace, uint64_t workspace_bytes, qkvp_stream_t stream);

/*
 * mla_decode_noalloc - mla_decode_plan (algo QKVP_ALGO_MMA_SYNC) followed by mla_decode_run, for callers
 * that cannot allocate device memory: a serving loop that has already given every free byte of the
 * GPU to a pre-sized KV pool, or a latency-critical decode step that must not risk the device-wide
 * synchronisation an allocation can bring. The source pages have no counterpart for this call.
 *
 * The work table and the split partials live in one fixed device array of
 * QKVP_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads the library holds until
 * the process exits. The call allocates nothing (no cudaMalloc or cudaFree, no allocating library
 * routine, no host heap). Problems that do not fit return QKVP_E_WORKSPACE before any device work:
 * more than QKVP_NOALLOC_MAX_BATCH requests, more than QKVP_NOALLOC_MAX_SEGMENTS segments, or a
 * table plus partials above the array size (at 128 heads, about 250 split partials).
 *
 * The first call on each device looks up the array's device address (cudaGetSymbolAddress) with
 * that device current, and later calls on that device reuse it: a cudaDeviceReset between calls
 * would leave that address stale, so do not reset a device between calls. Every call shares the
 * one array and leaves its partials there; calls whose GPU work overlaps (different streams or host
 * threads) race on it, so the caller must serialise them. Nothing in the array needs to start at
 * zero: each call uploads its own table and writes every partial before reading it.
 * The table is copied from static, pageable host memory, so the call returns only after the work
 * already queued on `stream` has drained. It returns QKVP_E_UNSUPPORTED while `stream` is being
 * captured into a CUDA graph (a replay would read a host table that later calls overwrite).
 * It runs the mma.sync kernel family with the same split as mla_decode_plan for that family and
 * the same SM count, so its output equals that of plan + run bit for bit.
 * Arguments as for mla_decode_plan and mla_decode_run (page size 64).
 */
#define QKVP_NOALLOC_SCRATCH_BYTES (64ull << 20)
#define QKVP_NOALLOC_MAX_BATCH 8192
#define QKVP_NOALLOC_MAX_SEGMENTS 16384
int mla_decode_noalloc(const int32_t* kv_indptr_host, const int32_t* kv_len_host, int32_t batch,
                       int32_t num_heads, int32_t kv_dtype, int32_t num_sms, int32_t min_splits,
                       const void* q, const void* kv_data, const uint8_t* kv_scale,
                       int64_t num_pages, const int32_t* kv_indices, float sm_scale,
                       float global_scale, void* out, float* lse, qkvp_stream_t stream);

/*
 * kv_pool_cast_bf16 - the cast-then-attend baseline's pool-wide cast: every E4M3 byte of an FP8
 * pool to its BF16 value (exact; NaN bytes 0x7F/0xFF become 0x7FC0). Source: "The Smoking Gun",
 * section "The Investigation Leading to This Message" (k_buffer = pool.to(q.dtype) over the whole
 * [495552, 1, 576] pool, every layer). Used only to measure that baseline.
 *  in  device uint8 [n_elems]; out device uint16 [n_elems]; both 16-byte aligned.
 */
int kv_pool_cast_bf16(const uint8_t* in, int64_t n_elems, void* out, qkvp_stream_t stream);

/*
 * kv_gather_fp8 - the extend path's gather: each request's cached tokens into one contiguous FP8
 * E4M3 workspace, the buffer a chunked-prefill step attends over and that every layer reuses.
 * Source: "SGLang x Qwen x NVIDIA ... NVFP4 KV Cache", section "SGLang implementation", item 2 (the
 * cached prefix is gathered and dequantized into an FP8 workspace shared across layers, then joined
 * with the current chunk's KV for FP8 attention).
 *   Workspace row tok_indptr[r] + t (t < tok_indptr[r+1] - tok_indptr[r]) is token t of request r,
 *   read from page kv_indices[kv_indptr[r] + t / 64], offset t % 64.
 *   FP8 pool: the bytes are copied. NVFP4 pool: element i becomes E4M3_RNE_satfinite(v) with
 *   v = fp32(scale(block) * e2m1(code)) * global_scale (the first product is exact; the second is one
 *   FP32 rounding): the workspace holds the E4M3 domain the cache was quantized from. The page does
 *   not say how the workspace is scaled; this is the plain reading.
 *  kv_data, kv_scale  device pool as for mla_decode_run (kv_scale NULL for FP8); 16-byte aligned.
 *  kv_dtype           QKVP_KV_FP8_E4M3 or QKVP_KV_NVFP4; global_scale 1 for FP8, finite > 0 for NVFP4.
 *  kv_indptr          device int32 [batch + 1] (pages); kv_indices device int32 [nnz] page ids.
 *  tok_indptr         device int64 [batch + 1], non-decreasing, tok_indptr[0] = 0,
 *                     tok_indptr[batch] = total_tokens (the caller's contract; rows are matched to
 *                     requests by binary search over it).
 *  out                device uint8 [total_tokens][576], 16-byte aligned; every row is written.
 * Every table entry is bounds-checked on the device: a row whose entry lies outside the request's
 * pages, the table (nnz) or the pool (num_pages) is written as zeros. Errors: QKVP_E_INVALID for
 * bad arguments, QKVP_E_UNSUPPORTED for page_size != 64, a BF16 pool or a per-token-scaled pool
 * (whose scale has no place in a plain E4M3 workspace).
 */
int kv_gather_fp8(const void* kv_data, const uint8_t* kv_scale, int32_t kv_dtype, float global_scale,
                  int32_t page_size, int64_t num_pages, const int32_t* kv_indptr, const int32_t* kv_indices,
                  int64_t nnz, const int64_t* tok_indptr, int32_t batch, int64_t total_tokens, uint8_t* out,
                  qkvp_stream_t stream);

/*
 * kv_gather_pages_bf16 - the gather-then-cast baseline: only the pages a batch reads, cast to BF16
 * into a compact pool that a BF16 decode then reads with page ids 0..n_pages-1. Source: "The FP8 KV
 * Cache Wall", sections "The Message" and "Aftermath" (Option B: cast only the active tokens, not
 * the whole pool; measured there at +29%). Used only to measure that baseline.
 *  kv_data   device FP8 pool [num_pages][64][576], 16-byte aligned.
 *  page_ids  device int32 [n_pages]; out device BF16 [n_pages][64][576], 16-byte aligned.
 * Page i of out is pool page page_ids[i] cast exactly (NaN bytes become 0x7FC0); an id outside the
 * pool gives a zero page. Errors: QKVP_E_INVALID for bad arguments, QKVP_E_UNSUPPORTED for
 * page_size != 64.
 */
int kv_gather_pages_bf16(const uint8_t* kv_data, int32_t page_size, int64_t num_pages, const int32_t* page_ids,
                         int64_t n_pages, void* out, qkvp_stream_t stream);

/*
 * mla_append_rope - one MLA step's append with the rotary position embedding on the way: token t's
 * latent row [c_kv(t) | R(p) k_pe(t)] goes into the pool as by kv_append_quant, p = positions[t], and the
 * query's rope parts go, rotated, into the last 64 dims of the q that mla_decode_run reads. The
 * source pages name the operation (a fused norm, rotation and store for indexer keys: "The Precision
 * Frontier: Implementing bf16 Index Keys") but give no arithmetic.
 *   R(p) turns each pair (a, b) of the 64 rope dims (rope_style) into (a c - b s, b c + a s), c =
 *   cos_sin[p][i], s = cos_sin[p][32 + i], in FP32 with one rounding per operation. The rotated values
 *   are quantized from FP32 (no rounding to BF16 in between), by the formulas of kv_append_quant.
 *  c_kv         device bf16, row t at c_kv + t * c_kv_stride (elements), 512 values.
 *  k_pe         device bf16, row t at k_pe + t * k_pe_stride, 64 values. May be a slice of a wider row.
 *  n_tokens     rows of c_kv, k_pe, slot_mapping, positions, q_pe and q.
 *  slot_mapping device int64 [n_tokens], as for kv_append_quant: slots outside the pool skip the row.
 *  positions    device int64 [n_tokens]. A position outside [0, max_positions) skips the token: neither
 *               its row nor its q is written.
 *  cos_sin      device float [max_positions][64]: the 32 cosines of a position, then the 32 sines.
 *  q_pe         device bf16, head h of token t at q_pe + t * q_pe_token_stride + h * q_pe_head_stride,
 *               64 values; NULL: no query is rotated (q must be NULL, num_heads 0).
 *  q            device bf16 [n_tokens][num_heads][576]; dims 512..575 of every head are written, the
 *               others are left as they are. q_pe may be q + 512 itself (strides num_heads * 576 and
 *               576): rotation in place. Other overlaps are not supported.
 *  kv_data, kv_scale, kv_dtype, global_scale, page_size, num_pages: as for kv_append_quant (an FP8,
 *               NVFP4 or per-token-scaled FP8 pool).
 * Row strides are multiples of 8 elements, c_kv, k_pe, q_pe, q, kv_data and cos_sin 16-byte aligned.
 * If two tokens of one call name the same slot, that row is unspecified: it may mix what they bring.
 */
int mla_append_rope(const void* c_kv, int64_t c_kv_stride, const void* k_pe, int64_t k_pe_stride,
                    int64_t n_tokens, const int64_t* slot_mapping, const int64_t* positions,
                    const float* cos_sin, int64_t max_positions, int32_t rope_style, const void* q_pe,
                    int64_t q_pe_token_stride, int64_t q_pe_head_stride, int32_t num_heads, void* q,
                    void* kv_data, uint8_t* kv_scale, int32_t kv_dtype, float global_scale,
                    int32_t page_size, int64_t num_pages, qkvp_stream_t stream);

/*
 * gqa_append_rope - append new tokens' K and V heads to a paged head pool (layout above), K rotated on
 * the way, and rotate the query heads in the same launch. Every array below is on the device, so a
 * captured call replays with new lengths.
 *   Request r brings the tokens tok_indptr[r] .. tok_indptr[r+1] - 1 and holds kv_len[r] tokens already;
 *   its j-th new token goes to cache position kv_len[r] + j, i.e. offset (kv_len[r] + j) % 64 of page
 *   kv_indices[kv_indptr[r] + (kv_len[r] + j) / 64]. Rows behind tok_indptr[batch] are padding: nothing
 *   of them is read or written.
 *   Block scale, per (page, K or V, head): need = amax / m, m = 448 (E4M3) or 127 (INT8), amax the
 *   largest finite |x| of the new elements that the call puts into the block. If the call writes the
 *   block's offset 0, or its scale is 0, the scale becomes need. Otherwise it becomes scale * 2^j with the
 *   smallest j >= 0 for which that is at least need, and if j > 0 the codes of the block's older tokens
 *   (the offsets before the call's first) become round(code * 2^-j): exact for E4M3 but for codes that
 *   become subnormal, and for INT8 each growth halves the errors before it, so that they stay below one
 *   step of the final scale. Codes are round(x / scale), or round(x) when scale is 0: E4M3 to nearest
 *   even, saturating at +-448, NaN gives 0x7F; INT8 to nearest even, held in [-127, 127], NaN gives 0.
 *   FP32 arithmetic with one rounding per operation; the rotation as for mla_append_rope, over the first
 *   rot_dim dims of a head, the others unchanged.
 *  k, v         device bf16, head h of token t at k + t * k_stride + h * head_dim (elements).
 *  n_tokens     rows of k, v, positions, q and q_out (tok_indptr entries beyond it are cut to it).
 *  tok_indptr   device int32 [batch + 1], non-decreasing from 0. kv_len device int32 [batch].
 *  kv_indptr, kv_indices, nnz: page table on the device, as for kv_gather_fp8 (kv_indices may be NULL if nnz is 0).
 *  positions    device int64 [n_tokens], the positions that rotate K and Q; NULL: the cache positions.
 *  cos_sin      device float [max_positions][rot_dim], cosines then sines; rot_dim a multiple of 16 up to
 *               head_dim, or 0 (no rotation, cos_sin NULL).
 *  q, q_out     device bf16 [.][num_heads][head_dim], token t at q + t * q_stride, q_out contiguous; the
 *               same buffer (q_stride = num_heads * head_dim) rotates in place. NULL, NULL, num_heads 0:
 *               none.
 * Skipped on the device: a token whose page lies outside the request's pages, the table or the pool
 * (its query is still rotated), and a token whose position lies outside [0, max_positions) (so is its
 * query). A page must not be appended to by two requests of one call.
 * head_dim 64, 128 or 256; num_kv_heads 1 to 256; row strides multiples of 8; k, v, q, q_out, kv_data and
 * cos_sin 16-byte aligned.
 */
int gqa_append_rope(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t n_tokens,
                    const int32_t* tok_indptr, const int32_t* kv_len, int32_t batch,
                    const int32_t* kv_indptr, const int32_t* kv_indices, int64_t nnz,
                    const int64_t* positions, const float* cos_sin, int64_t max_positions,
                    int32_t rot_dim, int32_t rope_style, int32_t num_kv_heads, int32_t head_dim,
                    void* kv_data, float* kv_scale, int32_t cache_dtype, int32_t page_size,
                    int64_t num_pages, const void* q, int64_t q_stride, int32_t num_heads, void* q_out,
                    qkvp_stream_t stream);

/* Host-side plan produced by gqa_decode_plan and consumed by gqa_decode_run; plain data, used as a
 * qkvp_plan is. */
typedef struct {
  int32_t batch, num_heads, num_kv_heads, head_dim, page_size, cache_dtype;
  int32_t window, sinks;       /* as given; window 0: every token is visible */
  int32_t num_workers;         /* independent workers of the decode kernel */
  int32_t warps_per_worker;    /* warps that share a worker's segments: 4 (a CTA) or 1 */
  int32_t num_segments;        /* (request, KV head, page range) pieces */
  int32_t num_split_groups;    /* (request, KV head) pairs cut into more than one segment */
  int32_t max_group_segments;  /* most segments of one pair */
  int32_t num_partials;        /* FP32 split partials held in the workspace */
  int32_t max_worker_pages, min_worker_pages;
  int32_t table_entries;       /* entries of kv_indices that the plan may address: kv_indptr[batch] */
  int32_t reserved;
  int64_t total_pages;         /* visible pages, summed over requests (of one KV head) */
  int64_t total_tokens;        /* visible tokens, summed over requests */
  uint64_t workspace_bytes, table_bytes, partial_o_offset, partial_lse_offset;
  uint64_t status_offset;      /* int32 status word, as in qkvp_plan; after a run that left it non-zero,
                                  plan again before the next */
  uint64_t magic;
} gqa_plan;

/*
 * gqa_decode_plan - split the visible pages of a batch into balanced work for gqa_decode_run.
 *  kv_indptr_host, kv_len_host, batch, page_size, num_sms, min_splits, workspace, workspace_bytes, stream:
 *               as for mla_decode_plan (also its return values, the size query with workspace NULL, and
 *               the refusal under stream capture). kv_len counts the token that asks: the query of
 *               request r sits at position kv_len[r] - 1.
 *  num_heads    a multiple of num_kv_heads; query heads h * G .. h * G + G - 1, G = num_heads /
 *               num_kv_heads, read KV head h. Any G: the kernel takes up to 16 of them in one pass over
 *               the pages and reads the pages again for each further 16.
 *  num_kv_heads 1 to 256. head_dim 64, 128 or 256. cache_dtype a qkvp_cache_dtype.
 *  window       tokens that a query sees back from its own, itself included; 0: all of them.
 *  sinks        with a window, the first tokens that stay visible as well; without one it must be 0.
 *               Token t of len is visible if t >= len - window or t < sinks. Pages with no visible token
 *               are never read: their table entries may be anything.
 * Host memory that runs out is reported as QKVP_E_WORKSPACE, too.
 */
int gqa_decode_plan(const int32_t* kv_indptr_host, const int32_t* kv_len_host, int32_t batch,
                    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                    int32_t cache_dtype, int32_t window, int32_t sinks, int32_t num_sms,
                    int32_t min_splits, void* workspace, uint64_t workspace_bytes, qkvp_stream_t stream,
                    gqa_plan* plan);

/*
 * gqa_decode_run - decode attention of one layer over a head pool. Per request r and query head a with
 * KV head h = a / G, over the visible tokens t,
 *   z_t = sm_scale * sum_d q[r,a,d] * sk * kcode_t[d],  out[r,a,d] = sum_t softmax(z)_t * sv * vcode_t[d],
 *   lse[r,a] = log sum_t exp(z_t),
 * sk, sv the scales of the token's K and V block. A request with no visible token (kv_len 0, or every
 * page id out of the pool) gives out 0 and lse -inf. One kernel launch: requests that are split are
 * joined by the last of their CTAs to finish, in a fixed order, so equal inputs give equal bits.
 * Codes of tokens that are not visible take no part, whatever they hold (NaN too).
 *  q            device bf16 [batch][num_heads][head_dim]. Held as FP16 times a power of two per head. The softmax's weights
 *               enter the product with V as FP16 (off by up to 2^-11); its sum and lse are taken from FP32 weights.
 *  kv_data, kv_scale, num_pages: the head pool; kv_data 128-byte aligned (TMA reads it), scales finite
 *               and not negative. Page ids outside [0, num_pages) read as tokens that are not visible.
 *               V scales and logits may be any powers of two apart, in any order; a token's weight below 2^-70
 *               of the request's largest may count as zero.
 *  kv_indices   device int32 page ids addressed by the plan's kv_indptr.
 *  out          device bf16 [batch][num_heads][head_dim], 16-byte aligned; lse float [batch][num_heads]
 *               or NULL.
 *  workspace    the buffer given to gqa_decode_plan. It holds partials and counters during the run: two
 *               runs that use one workspace must not overlap (nor two graphs that captured them).
 */
int gqa_decode_run(const gqa_plan* plan, const void* q, const void* kv_data, const float* kv_scale,
                   int64_t num_pages, const int32_t* kv_indices, float sm_scale, void* out, float* lse,
                   void* workspace, uint64_t workspace_bytes, qkvp_stream_t stream);

/*
 * qkvp_encode_f32 - the device rounding routines of kv_append_quant applied to raw FP32 values:
 * fmt 1 -> E4M3 (nearest even, saturating at +-448, NaN -> 0x7F); fmt 2 -> E2M1 (nearest even,
 * saturating at +-6, NaN -> 0x0). One code byte per input. Exposed so the rounding can be checked
 * exhaustively against the CPU oracle.
 */
int qkvp_encode_f32(const float* x, int64_t n, int32_t fmt, uint8_t* codes, qkvp_stream_t stream);

/* Static description of a status code; never NULL. */
const char* qkvp_status_string(int status);

/* Library ABI version (major * 100 + minor). */
int qkvp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QKVP_H_ */
