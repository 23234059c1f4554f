// C entry points of the rotated appends and of the head-pool decode: argument checks, the plan, dispatch.
//
// The plan reuses the split-KV planner: each (request, KV head, pass of up to 16 query heads) is a row of
// pages to it, the visible ones only, so the workers share out exactly the pages that are read.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/qkvp.h"
#include "qkvp_internal.h"

using namespace qkvp;

namespace {

constexpr int kMaxKvHeads = 256;
constexpr int kMaxHeads = 4096;
// Workers (CTAs) per SM of the decode kernel, and the pages of work that starting a segment costs.
constexpr int kCtasPerSm = 2;
constexpr int kSegmentCost = 2;

// Row strides in elements: multiples of 8 (16-byte vectors), at least one row wide.
bool stride_ok(int64_t s, int64_t width) { return s >= width && s % 8 == 0; }

// The visible pages of one request: its sink pages, then the pages of its window.
struct Visible {
  int32_t sink_pages = 0, win_page = 0, win_begin = 0, sink_end = 0;
  int32_t pages = 0;
  int64_t tokens = 0;
};
Visible visible_pages(int32_t len, int32_t window, int32_t sinks) {
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
  v.sink_pages = std::min((v.sink_end + kPage - 1) / kPage, v.win_page);
  v.pages = v.sink_pages + pages - v.win_page;
  v.tokens = static_cast<int64_t>(window) + v.sink_end;
  return v;
}

bool dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }
bool cache_ok(int32_t c) { return c == QKVP_CACHE_E4M3 || c == QKVP_CACHE_INT8; }

}  // namespace

extern "C" {

int mla_append_rope(const void* c_kv, int64_t c_kv_stride, const void* k_pe, int64_t k_pe_stride, int64_t n_tokens,
                    const int64_t* slot_mapping, const int64_t* positions, const float* cos_sin, int64_t max_positions,
                    int32_t rope_style, const void* q_pe, int64_t q_pe_token_stride, int64_t q_pe_head_stride,
                    int32_t num_heads, void* q, void* kv_data, uint8_t* kv_scale, int32_t kv_dtype, float global_scale,
                    int32_t page_size, int64_t num_pages, qkvp_stream_t stream) {
  if (n_tokens < 0 || num_pages < 0 || max_positions < 0 || num_heads < 0) return QKVP_E_INVALID;
  if (kv_dtype != QKVP_KV_FP8_E4M3 && kv_dtype != QKVP_KV_NVFP4 && kv_dtype != QKVP_KV_FP8_PER_TOKEN)
    return QKVP_E_UNSUPPORTED;
  if (rope_style != QKVP_ROPE_HALVES && rope_style != QKVP_ROPE_PAIRS) return QKVP_E_UNSUPPORTED;
  if (page_size != QKVP_PAGE_SIZE || num_heads > kMaxHeads) return QKVP_E_UNSUPPORTED;
  if (kv_dtype != QKVP_KV_NVFP4) {
    if (kv_scale != nullptr || global_scale != 1.0f) return QKVP_E_INVALID;
  } else {
    if (kv_scale == nullptr || !std::isfinite(global_scale) || !(global_scale > 0.0f)) return QKVP_E_INVALID;
    if (!aligned(kv_scale, 16)) return QKVP_E_INVALID;
  }
  if ((q_pe != nullptr) != (q != nullptr) || (q_pe != nullptr) != (num_heads > 0)) return QKVP_E_INVALID;
  if (n_tokens == 0) return QKVP_OK;
  if (!c_kv || !k_pe || !slot_mapping || !positions || !cos_sin || !kv_data) return QKVP_E_INVALID;
  if (!aligned(c_kv, 16) || !aligned(k_pe, 16) || !aligned(slot_mapping, 8) || !aligned(positions, 8) ||
      !aligned(cos_sin, 16) || !aligned(kv_data, 16))
    return QKVP_E_INVALID;
  if (!stride_ok(c_kv_stride, kDv) || !stride_ok(k_pe_stride, kLatent - kDv)) return QKVP_E_INVALID;
  if (q) {
    if (!aligned(q, 16) || !aligned(q_pe, 16)) return QKVP_E_INVALID;
    if (!stride_ok(q_pe_head_stride, kLatent - kDv) || !stride_ok(q_pe_token_stride, kLatent - kDv)) return QKVP_E_INVALID;
  }
  if (num_pages > INT64_MAX / page_size) return QKVP_E_INVALID;
  if (n_tokens > (int64_t(1) << 32)) return QKVP_E_UNSUPPORTED;
  MlaAppendArgs a{};
  a.c_kv = static_cast<const uint16_t*>(c_kv);
  a.k_pe = static_cast<const uint16_t*>(k_pe);
  a.slots = slot_mapping;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.q_pe = static_cast<const uint16_t*>(q_pe);
  a.q = static_cast<uint16_t*>(q);
  a.kv = static_cast<uint8_t*>(kv_data);
  a.kv_scale = kv_scale;
  a.c_kv_stride = c_kv_stride;
  a.k_pe_stride = k_pe_stride;
  a.q_pe_tok = q_pe_token_stride;
  a.q_pe_head = q_pe_head_stride;
  a.n = n_tokens;
  a.max_pos = max_positions;
  a.num_slots = num_pages * page_size;
  a.heads = num_heads;
  a.style = rope_style;
  a.kv_dtype = kv_dtype;
  a.g = global_scale;
  cudaError_t e = launch_mla_append_rope(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QKVP_OK : e == cudaErrorInvalidValue ? QKVP_E_UNSUPPORTED : QKVP_E_CUDA;
}

int gqa_append_rope(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t n_tokens,
                    const int32_t* tok_indptr, const int32_t* kv_len, int32_t batch, const int32_t* kv_indptr,
                    const int32_t* kv_indices, int64_t nnz, const int64_t* positions, const float* cos_sin,
                    int64_t max_positions, int32_t rot_dim, int32_t rope_style, int32_t num_kv_heads, int32_t head_dim,
                    void* kv_data, float* kv_scale, int32_t cache_dtype, int32_t page_size, int64_t num_pages,
                    const void* q, int64_t q_stride, int32_t num_heads, void* q_out, qkvp_stream_t stream) {
  if (n_tokens < 0 || batch < 0 || nnz < 0 || num_pages < 0 || max_positions < 0 || num_heads < 0) return QKVP_E_INVALID;
  if (page_size != QKVP_PAGE_SIZE || !dim_ok(head_dim) || !cache_ok(cache_dtype)) return QKVP_E_UNSUPPORTED;
  if (num_kv_heads < 1 || num_kv_heads > kMaxKvHeads || num_heads > kMaxHeads) return QKVP_E_UNSUPPORTED;
  if (rope_style != QKVP_ROPE_HALVES && rope_style != QKVP_ROPE_PAIRS) return QKVP_E_UNSUPPORTED;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16) return QKVP_E_UNSUPPORTED;
  if ((rot_dim > 0) != (cos_sin != nullptr)) return QKVP_E_INVALID;
  if ((q != nullptr) != (q_out != nullptr) || (q != nullptr) != (num_heads > 0)) return QKVP_E_INVALID;
  if (n_tokens > INT32_MAX) return QKVP_E_UNSUPPORTED;
  if (n_tokens == 0 || batch == 0) return QKVP_OK;
  if (!k || !v || !tok_indptr || !kv_len || !kv_indptr || !kv_indices || !kv_data || !kv_scale) return QKVP_E_INVALID;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kv_data, 16) || !aligned(tok_indptr, 4) || !aligned(kv_len, 4) ||
      !aligned(kv_indptr, 4) || !aligned(kv_indices, 4) || !aligned(kv_scale, 4) || !aligned(positions, 8) ||
      !aligned(cos_sin, 16) || !aligned(q, 16) || !aligned(q_out, 16))
    return QKVP_E_INVALID;
  const int64_t width = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (!stride_ok(k_stride, width) || !stride_ok(v_stride, width)) return QKVP_E_INVALID;
  const int64_t q_width = static_cast<int64_t>(num_heads) * head_dim;
  if (q && !stride_ok(q_stride, q_width)) return QKVP_E_INVALID;
  if (q && q == q_out && q_stride != q_width) return QKVP_E_INVALID;
  if (num_pages > INT64_MAX / (2 * width * page_size)) return QKVP_E_INVALID;
  GqaAppendArgs a{};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.tok_indptr = tok_indptr;
  a.kv_len = kv_len;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.kv = static_cast<uint8_t*>(kv_data);
  a.kv_scale = kv_scale;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.n = n_tokens;
  a.nnz = nnz;
  a.max_pos = max_positions;
  a.num_pages = num_pages;
  a.batch = batch;
  a.rot = rot_dim;
  a.style = rope_style;
  a.kv_heads = num_kv_heads;
  a.dim = head_dim;
  a.heads = num_heads;
  a.cache_dtype = cache_dtype;
  cudaError_t e = launch_gqa_append_rope(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QKVP_OK : e == cudaErrorInvalidValue ? QKVP_E_UNSUPPORTED : QKVP_E_CUDA;
}

int gqa_decode_plan(const int32_t* kv_indptr_host, const int32_t* kv_len_host, int32_t batch, int32_t num_heads,
                    int32_t num_kv_heads, int32_t head_dim, int32_t page_size, int32_t cache_dtype, int32_t window,
                    int32_t sinks, int32_t num_sms, int32_t min_splits, void* workspace, uint64_t workspace_bytes,
                    qkvp_stream_t stream, gqa_plan* plan) try {
  if (!plan) return QKVP_E_INVALID;
  std::memset(plan, 0, sizeof(*plan));
  if (page_size != QKVP_PAGE_SIZE || !dim_ok(head_dim) || !cache_ok(cache_dtype)) return QKVP_E_UNSUPPORTED;
  if (num_kv_heads < 1 || num_kv_heads > kMaxKvHeads) return QKVP_E_UNSUPPORTED;
  if (num_heads < 1 || num_heads > kMaxHeads || num_heads % num_kv_heads) return QKVP_E_UNSUPPORTED;
  if (window < 0 || sinks < 0 || (window == 0 && sinks != 0)) return QKVP_E_INVALID;
  // the page table's checks, with a head count that they accept
  const int st = check_plan_args(kv_indptr_host, kv_len_host, batch, 16, page_size, QKVP_KV_FP8_E4M3, min_splits);
  if (st != QKVP_OK) return st;
  const int group = num_heads / num_kv_heads;
  const int passes = (group + kGqaPassHeads - 1) / kGqaPassHeads;
  const int64_t rows = static_cast<int64_t>(batch) * num_kv_heads * passes;
  if (rows > (1 << 24)) return QKVP_E_UNSUPPORTED;
  if (num_sms <= 0) {
    num_sms = query_sms();
    if (num_sms <= 0) return QKVP_E_CUDA;
  }
  if (num_sms > 65536) return QKVP_E_INVALID;
  const int workers = num_sms * kCtasPerSm;

  // one row of visible pages per (request, KV head, pass)
  std::vector<Visible> vis(batch);
  std::vector<int32_t> len(rows), indptr(rows + 1);
  int64_t pages = 0, tokens = 0, row_pages = 0;
  for (int r = 0; r < batch; ++r) {
    vis[r] = visible_pages(kv_len_host[r], window, sinks);
    pages += vis[r].pages;
    tokens += vis[r].tokens;
  }
  if (pages * num_kv_heads * passes > INT32_MAX) return QKVP_E_UNSUPPORTED;
  for (int64_t i = 0; i < rows; ++i) {
    const Visible& v = vis[i / (num_kv_heads * passes)];
    indptr[i] = static_cast<int32_t>(row_pages);
    if (static_cast<int64_t>(v.pages) * kPage > INT32_MAX) return QKVP_E_UNSUPPORTED;
    len[i] = v.pages * kPage;
    row_pages += v.pages;
  }
  indptr[rows] = static_cast<int32_t>(row_pages);

  SplitInfo info;
  split_pages(indptr.data(), len.data(), static_cast<int>(rows), workers, min_splits, SplitOut{}, info, kSegmentCost);
  std::vector<Segment> cut(static_cast<size_t>(std::max<int64_t>(1, info.num_segments)));
  std::vector<int32_t> wptr(workers + 1), rptr(rows + 1), wide(std::max<int64_t>(1, rows));
  const SplitOut out{cut.data(), info.num_segments, wptr.data(), rptr.data(), wide.data()};
  if (!split_pages(indptr.data(), len.data(), static_cast<int>(rows), workers, min_splits, out, info, kSegmentCost))
    return QKVP_E_INVALID;
  // rows without a visible page get a segment of no pages, which writes zeros: appended to the workers in turn
  const int64_t empty = info.empty_reqs;
  const int64_t total = info.num_segments + empty;
  const GqaTable t = gqa_table(total, workers, info.split_reqs);

  plan->batch = batch;
  plan->num_heads = num_heads;
  plan->num_kv_heads = num_kv_heads;
  plan->head_dim = head_dim;
  plan->page_size = page_size;
  plan->cache_dtype = cache_dtype;
  plan->window = window;
  plan->sinks = sinks;
  plan->num_workers = workers;
  plan->num_segments = static_cast<int32_t>(total);
  plan->num_split_groups = info.split_reqs;
  plan->max_group_segments = info.max_req_segs;
  plan->num_partials = info.partials;
  plan->max_worker_pages = info.max_pages;
  plan->min_worker_pages = info.min_pages;
  plan->total_pages = pages;
  plan->total_tokens = tokens;
  plan->table_bytes = t.bytes;
  plan->status_offset = t.status;
  plan->partial_o_offset = t.bytes;
  plan->partial_lse_offset = t.bytes + align_up(static_cast<uint64_t>(info.partials) * kGqaPassHeads * head_dim * 4);
  plan->workspace_bytes = plan->partial_lse_offset + align_up(static_cast<uint64_t>(info.partials) * kGqaPassHeads * 4);
  if (workspace == nullptr) return QKVP_OK;
  if (workspace_bytes < plan->workspace_bytes || !aligned(workspace, kTableAlign)) {
    const uint64_t need = plan->workspace_bytes;
    std::memset(plan, 0, sizeof(*plan));
    plan->workspace_bytes = need;
    return QKVP_E_WORKSPACE;
  }
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(reinterpret_cast<cudaStream_t>(stream), &cap) != cudaSuccess) return QKVP_E_CUDA;
  if (cap != cudaStreamCaptureStatusNone) {
    std::memset(plan, 0, sizeof(*plan));
    return QKVP_E_UNSUPPORTED;
  }

  std::vector<uint8_t> blob(t.bytes);
  GqaSegment* segs = reinterpret_cast<GqaSegment*>(blob.data() + t.segs);
  int32_t* ptr = reinterpret_cast<int32_t*>(blob.data() + t.wptr);
  std::vector<int32_t> counter(rows, 0);
  for (int64_t i = 0, c = 0; i < rows; ++i)
    if (rptr[i + 1] - rptr[i] > 1) counter[i] = static_cast<int32_t>(c++);
  auto fill = [&](GqaSegment& g, int64_t row) {
    const int r = static_cast<int>(row / (num_kv_heads * passes));
    const int h = static_cast<int>(row / passes % num_kv_heads), pass = static_cast<int>(row % passes);
    const Visible& v = vis[r];
    g.req = r;
    g.kv_head = h;
    g.head0 = h * group + pass * kGqaPassHeads;
    g.heads = std::min(kGqaPassHeads, group - pass * kGqaPassHeads);
    g.page0 = kv_indptr_host[r];
    g.len = kv_len_host[r];
    g.sink_pages = v.sink_pages;
    g.win_page = v.win_page;
    g.win_begin = v.win_begin;
    g.sink_end = v.sink_end;
    g.partial = -1;
  };
  int64_t n = 0, next_empty = 0, given = 0;
  for (int w = 0; w < workers; ++w) {
    ptr[w] = static_cast<int32_t>(n);
    for (int32_t i = wptr[w]; i < wptr[w + 1]; ++i) {
      const Segment& s = cut[i];
      GqaSegment& g = segs[n++];
      fill(g, s.req);
      g.page_begin = s.page_begin - indptr[s.req];
      g.num_pages = s.num_pages;
      g.partial = s.partial;
      if (s.partial >= 0) {
        g.group_first = cut[rptr[s.req]].partial;
        g.group_count = rptr[s.req + 1] - rptr[s.req];
        g.counter = counter[s.req];
      }
    }
    for (const int64_t share = empty * (w + 1) / workers; given < share; ++given) {
      while (len[next_empty] > 0) ++next_empty;
      fill(segs[n++], next_empty++);
    }
  }
  ptr[workers] = static_cast<int32_t>(n);
  if (upload_table(workspace, blob.data(), blob.size(), reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return QKVP_E_CUDA;
  plan->magic = kGqaMagic;
  return QKVP_OK;
} catch (const std::bad_alloc&) {
  return QKVP_E_WORKSPACE;
} catch (...) {
  return QKVP_E_INVALID;
}

int gqa_decode_run(const gqa_plan* plan, const void* q, const void* kv_data, const float* kv_scale, int64_t num_pages,
                   const int32_t* kv_indices, float sm_scale, void* out, float* lse, void* workspace,
                   uint64_t workspace_bytes, qkvp_stream_t stream) {
  if (!plan || plan->magic != kGqaMagic) return QKVP_E_INVALID;
  if (!workspace || workspace_bytes < plan->workspace_bytes || !aligned(workspace, kTableAlign)) return QKVP_E_WORKSPACE;
  if (num_pages < 0 || !std::isfinite(sm_scale)) return QKVP_E_INVALID;
  if (plan->batch == 0) return QKVP_OK;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4))) return QKVP_E_INVALID;
  if (plan->total_pages > 0) {
    if (!kv_data || !kv_scale || !kv_indices) return QKVP_E_INVALID;
    if (!aligned(kv_data, 128) || !aligned(kv_scale, 4) || !aligned(kv_indices, 4)) return QKVP_E_INVALID;
  }
  const int64_t page_bytes = 2ll * plan->num_kv_heads * kPage * plan->head_dim;
  if (num_pages > (int64_t(1) << 31) * 128 / page_bytes) return QKVP_E_UNSUPPORTED;   // 256 GiB: TMA row coordinates
  const GqaTable t = gqa_table(plan->num_segments, plan->num_workers, plan->num_split_groups);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  GqaDecodeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.kv = static_cast<const uint8_t*>(kv_data);
  a.kv_scale = kv_scale;
  a.num_pages = num_pages;
  a.kv_indices = kv_indices;
  a.segs = reinterpret_cast<const GqaSegment*>(ws + t.segs);
  a.worker_ptr = reinterpret_cast<const int32_t*>(ws + t.wptr);
  a.counters = reinterpret_cast<uint32_t*>(ws + t.counters);
  a.status = reinterpret_cast<int*>(ws + t.status);
  a.part_o = reinterpret_cast<float*>(ws + plan->partial_o_offset);
  a.part_lse = reinterpret_cast<float*>(ws + plan->partial_lse_offset);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.heads = plan->num_heads;
  a.kv_heads = plan->num_kv_heads;
  a.dim = plan->head_dim;
  a.cache_dtype = plan->cache_dtype;
  a.num_workers = plan->num_workers;
  a.scale_log2 = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
  return launch_gqa_decode(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? QKVP_OK : QKVP_E_CUDA;
}

}  // extern "C"
