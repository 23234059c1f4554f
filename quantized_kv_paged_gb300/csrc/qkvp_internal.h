// Internal declarations shared by the translation units of libqkvp (not part of the ABI).
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/qkvp.h"

namespace qkvp {

constexpr int kLatent = 576;            // 512 nope + 64 rope
constexpr int kDv = 512;                // V = the first 512 latent dims
constexpr int kPage = 64;               // tokens per page
constexpr int kPacked = kLatent / 2;    // NVFP4 data bytes per token (two E2M1 codes per byte)
constexpr int kScales = kLatent / 16;   // NVFP4 E4M3 block scales per token
constexpr uint64_t kPlanMagic = 0x716b76702d706c31ull;

enum : int { KV_FP8 = 1, KV_NVFP4 = 2, KV_BF16 = 3, KV_FP8PT = 4 };
// Per-token-scaled FP8 page: 64 rows of 576 E4M3 codes, then 64 FP32 token scales.
constexpr int kPtScaleOff = kPage * kLatent;              // 36,864
constexpr int kPtPageBytes = kPage * (kLatent + 4);       // 37,120
enum : int { SRC_FP8 = 1, SRC_BF16 = 2 };
enum : int { ALGO_AUTO = 0, ALGO_MMA = 1, ALGO_TC = 2 };

// One piece of one request's page list, processed by one worker from start to end. Segments are
// stored in request order; a request whose pages form a single segment is written straight to the
// output (partial < 0), otherwise each segment writes a normalised FP32 partial and its
// log2-sum-exp, merged by the combine kernel.
struct Segment {
  int32_t req;
  int32_t page_begin;   // index into kv_indices of the first page
  int32_t num_pages;
  int32_t num_tokens;   // tokens covered (the last page may be partial)
  int32_t partial;      // partial slot, or -1 for a direct write
  int32_t pad[3];
};
static_assert(sizeof(Segment) == 32, "segment layout");

struct DecodeArgs {
  const uint16_t* q;          // bf16 [B][H][576]
  const uint8_t* kv;          // pool (fp8 / nvfp4 data / bf16)
  const uint8_t* kv_scale;    // nvfp4 block scales
  int64_t num_pages;
  const int32_t* kv_indices;
  const Segment* segs;
  const int32_t* worker_ptr;  // [num_workers + 1]
  const int32_t* req_seg_ptr; // [batch + 1]
  const int32_t* wide_req;    // [num_wide] requests with more than kCombineWideSegs segments
  float* part_o;              // [num_segments][H][512]
  float* part_lse;            // [num_segments][H], log2 domain
  uint16_t* out;              // bf16 [B][H][512]
  float* lse;                 // [B][H] natural log, may be null
  int* status;                // device status word (timeouts), inside the workspace
  int batch, heads, num_workers, ctas_per_worker, num_segments, kv_dtype;
  int fp8_qk;                 // mma.sync kernel: FP8 Q.K^T (two-term E4M3 Q) instead of FP16
  float scale_log2;           // sm_scale * g * log2(e)
  float out_scale;            // g
};

// Workspace layout of a plan: the segment table, the per-worker segment ranges, the per-request
// segment ranges and the list of wide requests, each 256-byte aligned, followed by the FP32 partials.
constexpr uint64_t kTableAlign = 256;
inline uint64_t align_up(uint64_t x) { return (x + kTableAlign - 1) / kTableAlign * kTableAlign; }

// The status word is zero after planning; a kernel that gives up waiting sets bits in it.
struct TableLayout {
  uint64_t segs, wptr, rptr, wide, status, bytes;
};

// A request cut into more segments than this is merged by the combine's wide CTAs (eight segment
// groups per quarter head) instead of one thread per 8 output dims walking every segment; the
// planner lists such requests in the table.
constexpr int kCombineWideSegs = 8;

inline TableLayout table_layout(int64_t segments, int64_t workers, int64_t batch) {
  TableLayout t;
  t.segs = 0;
  t.wptr = align_up(static_cast<uint64_t>(segments) * sizeof(Segment));
  t.rptr = t.wptr + align_up(static_cast<uint64_t>(workers + 1) * 4);
  t.wide = t.rptr + align_up(static_cast<uint64_t>(batch + 1) * 4);
  t.status = t.wide + align_up(static_cast<uint64_t>(batch) * 4);
  t.bytes = t.status + kTableAlign;
  return t;
}

// The split-KV planner (split.cu), shared by mla_decode_plan and mla_decode_noalloc. It writes into
// the caller's arrays: segs [max_segs], wptr [workers + 1], rptr [batch + 1], wide [batch]. With
// segs == nullptr it only counts (num_segments, page totals and per-worker page counts); the
// per-request fields of SplitInfo need the segments. Returns false when more than max_segs
// segments would be written.
struct SplitOut {
  Segment* segs = nullptr;
  int64_t max_segs = 0;
  int32_t* wptr = nullptr;
  int32_t* rptr = nullptr;
  int32_t* wide = nullptr;
};
struct SplitInfo {
  int64_t num_segments = 0;
  int32_t split_reqs = 0, empty_reqs = 0, max_pages = 0, min_pages = 0, partials = 0, max_req_segs = 0,
          num_wide = 0;
  int64_t total_pages = 0, total_tokens = 0;
};
// seg_cost > 0 balances pages + seg_cost per request each worker starts (the tcgen05 kernel loads a
// new request's Q and refills its pipeline at each); 0 gives every worker an equal page quota.
bool split_pages(const int32_t* indptr, const int32_t* len, int batch, int workers, int min_splits,
                 const SplitOut& out, SplitInfo& info, int seg_cost = 0);
// The argument checks of mla_decode_plan that need no device (status code, QKVP_OK if they pass).
int check_plan_args(const int32_t* indptr, const int32_t* len, int batch, int num_heads, int page_size,
                    int kv_dtype, int min_splits);
// Sets every field of *plan except magic from a split (table layout, offsets and workspace size).
void fill_plan(qkvp_plan* plan, const SplitInfo& info, int batch, int num_heads, int kv_dtype, int algo,
               int workers, int ctas_per_worker);
// Writes the work table of a filled split into blob [table_layout(...).bytes], zeros elsewhere.
void write_table(uint8_t* blob, const SplitOut& s, const SplitInfo& info, int workers, int batch);

// Arguments of the extend-path gather (kv_gather_fp8).
struct GatherArgs {
  const uint8_t* kv;
  const uint8_t* kv_scale;
  int64_t num_pages;
  const int32_t* kv_indptr;   // [batch + 1], pages
  const int32_t* kv_indices;  // [nnz] page ids
  int64_t nnz;
  const int64_t* tok_indptr;  // [batch + 1], workspace rows
  uint8_t* out;               // [total_tokens][576] E4M3
  int64_t total_tokens;
  int batch, kv_dtype;
  float g;
};

// Arguments of mla_append_rope.
struct MlaAppendArgs {
  const uint16_t* c_kv;       // bf16 [n][512], row stride c_kv_stride
  const uint16_t* k_pe;       // bf16 [n][64], row stride k_pe_stride
  const int64_t* slots;
  const int64_t* positions;
  const float* cos_sin;       // [max_pos][64]
  const uint16_t* q_pe;       // bf16 [n][heads][64], strides q_pe_tok, q_pe_head
  uint16_t* q;                // bf16 [n][heads][576]
  uint8_t* kv;
  uint8_t* kv_scale;
  int64_t c_kv_stride, k_pe_stride, q_pe_tok, q_pe_head, n, max_pos, num_slots;
  int heads, style, kv_dtype;
  float g;
};

// Arguments of gqa_append_rope.
struct GqaAppendArgs {
  const uint16_t* k;          // bf16 [n][kv_heads][dim], row stride k_stride
  const uint16_t* v;
  const int32_t* tok_indptr;  // [batch + 1]
  const int32_t* kv_len;      // [batch]
  const int32_t* kv_indptr;   // [batch + 1]
  const int32_t* kv_indices;  // [nnz]
  const int64_t* positions;   // [n] or null
  const float* cos_sin;       // [max_pos][rot]
  const uint16_t* q;          // bf16 [n][heads][dim], row stride q_stride
  uint16_t* q_out;            // bf16 [n][heads][dim]
  uint8_t* kv;                // [num_pages][2][kv_heads][64][dim]
  float* kv_scale;            // [num_pages][2][kv_heads]
  int64_t k_stride, v_stride, q_stride, n, nnz, max_pos, num_pages;
  int batch, rot, style, kv_heads, dim, heads, cache_dtype;
  int head_parts;             // CTAs that share a page's K (or V) heads (set by the launcher)
  uint32_t kv_ctas;           // CTAs of the K and V blocks; the query's follow (set by the launcher)
};

// One piece of the visible pages of one (request, KV head, pass of 16 query heads), processed by one worker
// of the head-pool decode, a CTA or a warp. Visible page v of a request is page v of its list below sink_pages, and page
// win_page + (v - sink_pages) from there on.
struct GqaSegment {
  int32_t req, kv_head;
  int32_t head0, heads;        // first query head and how many (1 to 16)
  int32_t page0;               // index into kv_indices of the request's first page
  int32_t len;                 // tokens of the request
  int32_t sink_pages, win_page;
  int32_t win_begin, sink_end; // token t is visible if t < sink_end or win_begin <= t < len
  int32_t page_begin, num_pages;  // visible pages [page_begin, page_begin + num_pages)
  int32_t partial;             // partial slot, or -1 for a direct write
  // Arrivals at `counter` are joined by the last of `group_count`, from the slots group_first ... A group of
  // many segments joins in two levels: subgroups first, each into sub_slot, and the last subgroup joins the
  // top_count slots from top_first. top_counter -1: one level.
  int32_t group_first, group_count, counter;
  int32_t top_first, top_count, top_counter, sub_slot;
};
static_assert(sizeof(GqaSegment) == 80, "segment layout");

// What a worker starts from, in one read: the range of its segments and the first of them.
struct GqaWorker {
  GqaSegment first;
  int32_t begin, end;
  int32_t pad[2];
};
static_assert(sizeof(GqaWorker) == 96, "worker layout");

constexpr uint64_t kGqaMagic = 0x716b76702d677161ull;
constexpr int kGqaPassHeads = 16;   // query heads of one pass over the pages
// CTAs of the head-pool decode that one SM holds: what registers allow, and at D = 128 no more than two (its comment).
constexpr int gqa_ctas_per_sm(int dim, int group) { return dim == 64 && group <= 8 ? 3 : 2; }

struct GqaDecodeArgs {
  const uint16_t* q;          // bf16 [B][H][D]
  const uint8_t* kv;
  const float* kv_scale;
  int64_t num_pages;
  const int32_t* kv_indices;
  const GqaSegment* segs;
  const GqaWorker* workers;   // [num_workers]
  uint32_t* counters;         // arrival counters of the joins, zero between runs
  int* status;
  float* part_o;              // [num_partials][16][D], normalised
  float* part_lse;            // [num_partials][16], log2 domain
  uint16_t* out;              // bf16 [B][H][D]
  float* lse;                 // [B][H] or null
  int heads, kv_heads, dim, cache_dtype, num_workers;
  int team;                   // warps of a worker: 4 (a CTA) or 1
  float scale_log2;           // sm_scale * log2(e)
};

// Work table of a head-pool plan: segments, workers, then the status word and the joins' counters.
struct GqaTable {
  uint64_t segs, workers, status, counters, bytes;
};
inline GqaTable gqa_table(int64_t segments, int64_t workers, int64_t counters) {
  GqaTable t;
  t.segs = 0;
  t.workers = align_up(static_cast<uint64_t>(segments) * sizeof(GqaSegment));
  t.status = t.workers + align_up(static_cast<uint64_t>(workers) * sizeof(GqaWorker));
  t.counters = t.status + kTableAlign;
  t.bytes = t.counters + align_up(static_cast<uint64_t>(counters) * 4);
  return t;
}

// One piece of the pages that one block of query rows of a tree attention sees. Row i of a (request, KV head) is drafted
// token i / G, query head kv_head * G + i % G; a block holds up to 128 consecutive rows. Page v of the request's
// visible ones is page v of its list below sink_pages, and page win_page + (v - sink_pages) from there on.
struct TreeSegment {
  int32_t kv_head, row0, rows;    // rows [row0, row0 + rows) of the KV head
  int32_t tok0;                   // the request's first drafted token among the call's
  int32_t page0;                  // index into kv_indices of the request's first page
  int32_t cached, len;            // tokens before the drafted ones, and with them
  int32_t sink_pages, win_page;
  int32_t page_begin, num_pages;  // visible pages [page_begin, page_begin + num_pages)
  int32_t partial;                // partial slot, or -1 for a direct write
};
static_assert(sizeof(TreeSegment) == 48, "segment layout");

// A block that was cut into segments: its partials are slots [first, first + count).
struct TreeJoin {
  int32_t first, count, kv_head, row0, rows, tok0;
  int32_t pad[2];
};
static_assert(sizeof(TreeJoin) == 32, "join layout");

constexpr uint64_t kTreeMagic = 0x716b76702d747265ull;
constexpr int kTreeTile = 128;         // rows of a block: the lanes of tensor memory
constexpr int kTreeMaxDrafted = 256;   // drafted tokens of a request
struct TreeWorker {
  int32_t begin, end;             // its segments
  int32_t pages;                  // of all of them
  int32_t pad;
};

struct TreeArgs {
  const uint16_t* q;          // bf16 [n][H][D]
  const uint8_t* kv;
  const float* kv_scale;
  int64_t num_pages;
  const int32_t* kv_indices;
  const uint32_t* mask;       // [n][words], or null: a chain
  const TreeSegment* segs;
  const TreeWorker* workers;  // [num_workers]
  const TreeJoin* joins;
  int* status;
  float* part_o;              // [num_partials][D / 4][128][4], normalised
  float* part_lse;            // [num_partials][128], log2 domain; with row_copies the lanes are [row_copies][128 / row_copies]
  uint16_t* out;              // bf16 [n][H][D]
  float* lse;                 // [n][H] or null
  int heads, kv_heads, dim, cache_dtype, words, window, sinks;
  int num_workers, num_joins, row_copies;
  float scale_log2;           // |sm_scale| log2(e)
  uint32_t flip;              // 0x80008000 where sm_scale is negative: turns Q's signs
};

// Work table of a tree plan.
struct TreeTable {
  uint64_t segs, workers, joins, status, bytes;
};
inline TreeTable tree_table(int64_t segments, int64_t workers, int64_t joins) {
  TreeTable t;
  t.segs = 0;
  t.workers = align_up(static_cast<uint64_t>(segments) * sizeof(TreeSegment));
  t.joins = t.workers + align_up(static_cast<uint64_t>(workers) * sizeof(TreeWorker));
  t.status = t.joins + align_up(static_cast<uint64_t>(joins) * sizeof(TreeJoin));
  t.bytes = t.status + kTableAlign;
  return t;
}

// Arguments of gqa_tree_commit.
constexpr int kMaxLayers = 128;
struct TreeCommitArgs {
  uint8_t* kv[kMaxLayers];    // [num_pages][2][kv_heads][64][dim] of each layer
  float* scale[kMaxLayers];   // [num_pages][2][kv_heads]
  const int32_t* kv_len;      // [batch] tokens before the drafted ones
  const int32_t* kv_indptr;   // [batch + 1]
  const int32_t* kv_indices;  // [nnz]
  const int32_t* path;        // [batch][max_path]
  const int32_t* path_len;    // [batch]
  int64_t nnz, num_pages;
  int layers, batch, max_path, kv_heads, dim, cache_dtype;
};

// The pools that a page is copied in, cut into units of kCopyUnit bytes.
constexpr int kMaxPools = 256;
constexpr int kCopyUnit = 4096;
struct PagePools {
  uint8_t* base[kMaxPools];
  uint32_t bytes[kMaxPools];       // of a page
  uint32_t first_unit[kMaxPools];  // of the pool's units within a page's
  uint32_t units;                  // of a page, all pools
  int count;
};

// Page tables, counts and the free list (qkvp_page_state).
struct PageState {
  int32_t *table, *held, *lens, *refs, *free_list, *free_count;
  int rows, row_pages;
  int64_t num_pages;
};

// A page call's workspace. arrived, claim and marks are zero between calls; the rest is scratch.
struct PageWork {
  int32_t *arrived, *moves;
  int32_t* claim;      // [rows]
  uint32_t* marks;     // [num_pages / 32]
  int32_t *src, *dst;  // [max(n, num_pages)]
  int32_t* rank;       // [num_pages]
};

// Limits of the head pool's entry points.
constexpr int kMaxKvHeads = 256;
constexpr int kMaxHeads = 4096;
inline bool dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }
inline bool cache_ok(int32_t c) { return c == QKVP_CACHE_E4M3 || c == QKVP_CACHE_INT8; }

// The visible pages of one request: its sink pages, then the pages of its window.
struct Visible {
  int32_t sink_pages = 0, win_page = 0, win_begin = 0, sink_end = 0;
  int32_t pages = 0;
  int64_t tokens = 0;
};
inline Visible visible_pages(int32_t len, int32_t window, int32_t sinks) {
  Visible v;
  const int32_t pages = static_cast<int32_t>((static_cast<int64_t>(len) + kPage - 1) / kPage);
  if (window == 0 || len <= window) {
    v.pages = pages;
    v.tokens = len;
    return v;
  }
  v.win_begin = len - window;
  v.sink_end = std::min(sinks, v.win_begin);
  v.win_page = v.win_begin / kPage;
  // a page that holds both sinks and window is counted once
  v.sink_pages = std::min(static_cast<int32_t>((static_cast<int64_t>(v.sink_end) + kPage - 1) / kPage), v.win_page);
  v.pages = v.sink_pages + pages - v.win_page;
  v.tokens = static_cast<int64_t>(window) + v.sink_end;
  return v;
}

// Copies a work table to the device in stream order, through pinned staging where it can (capi.cu).
cudaError_t upload_table(void* dst, const void* src, size_t n, cudaStream_t st);
int query_sms();
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Launches a kernel that calls dev::wait_for_previous() before it touches anything that the kernel before it in the
// stream may have written, so that it may start while that one ends.
template <class... Params, class... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

cudaError_t launch_mla_append_rope(const MlaAppendArgs& a, cudaStream_t s);
cudaError_t launch_gqa_append_rope(const GqaAppendArgs& a, cudaStream_t s);
cudaError_t launch_gqa_decode(const GqaDecodeArgs& a, cudaStream_t s);
cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s);
cudaError_t launch_tree_commit(const TreeCommitArgs& a, cudaStream_t s);
cudaError_t launch_pages_copy(const PagePools& p, const int32_t* src, const int32_t* dst, int64_t n, int64_t num_pages, int sms, cudaStream_t s);
cudaError_t launch_pages_fork(const PagePools& p, const PageState& t, const int32_t* parents, const int32_t* children, int n, int32_t* status,
                              const PageWork& ws, int sms, cudaStream_t s);
cudaError_t launch_pages_grow(const PageState& t, const int32_t* list, const int32_t* tokens, int n, int32_t* status, const PageWork& ws,
                              cudaStream_t s);
cudaError_t launch_pages_free(const PageState& t, const int32_t* list, int n, const PageWork& ws, cudaStream_t s);
cudaError_t launch_pages_compact(const PagePools& p, const PageState& t, const PageWork& ws, int sms, cudaStream_t s);
cudaError_t launch_gather_fp8(const GatherArgs& a, cudaStream_t s);
cudaError_t launch_gather_pages_bf16(const uint8_t* pool, int64_t num_pages, const int32_t* ids, int64_t n,
                                     void* out, cudaStream_t s);
cudaError_t launch_append(const void* src, int src_dtype, int64_t n, const int64_t* slots,
                          void* kv_data, uint8_t* kv_scale, int kv_dtype, float g,
                          int64_t num_slots, cudaStream_t s);
cudaError_t launch_encode(const float* x, int64_t n, int fmt, uint8_t* codes, cudaStream_t s);
cudaError_t launch_cast(const uint8_t* in, int64_t n, uint16_t* out, cudaStream_t s);
cudaError_t launch_decode_mma(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_tc(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_tm(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_combine(const DecodeArgs& a, int num_wide, cudaStream_t s);

// Heads per CTA of the mma.sync kernel for a head count (0 if unsupported), and of its FP8 Q.K^T
// variant (16 or 32).
int mma_heads_per_cta(int heads);
int mma_fp8_heads_per_cta(int heads);
// Head columns of the token-major tcgen05 kernel for a head count (16, 32 or 64; 0 if unsupported).
int tm_heads_padded(int heads);
// CTA pairs of the tcgen05 kernel that the current device runs at once (-1 on error).
int tc_max_active_clusters();

}  // namespace qkvp
