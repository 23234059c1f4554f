// C entry points of the rotated appends and of the head-pool decode: argument checks, the plan, dispatch.
//
// The plan reuses the split-KV planner: each (request, KV head, pass of up to 16 query heads) is a row of
// pages to it, the visible ones only, so the workers share out exactly the pages that are read.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/qkvp.h"
#include "qkvp_internal.h"

using namespace qkvp;

namespace {

// The split, from decode times on one GB300 over 256 to 4,096 rows (a row: the visible pages of one request and
// KV head, or of 16 of its query heads) of 128 to 2,048 tokens, D 64 to 256, 4 to 16 query heads per KV head:
// - Rows per SM from which a worker is a warp: 512 rows of 512 tokens (D 64) 9.8 us against 11.4 with CTAs (ragged ones of 128
//   to 1,024 tokens 9.0 against 8.8), 1,024 of 2,048 (D 128) 81 against 88; below it CTAs: 352 of 32,768 429 against 444, 256
//   ragged ones (16 heads, INT8) 80 against 88. From one row per SM already where a row has no more than 8 units: 256
//   ragged ones of 32 to 256 tokens 11.3 against 12.3 (D 256), 7.4 against 8.7 (D 128); equal ones of 128 (D 256) 11.2 / 10.1.
// - Pages below which a CTA is not worth its start: 8 rows of 16 pages (D 128) 6.9 us with 1, 5.8 with 2, 6.4 with 4; a
//   sweep of 15 other shapes does not tell 2 and 4 apart (8 rows of 4 pages stay whole, 4.3 us).
// - Pages of work that starting a row counts as, some 128 KB for a CTA and 32 to 48 KB for a warp. Warps, 2 against 4
//   against 8 pages: 24.8 / 23.4 / 22.5 us in the window case of D 64 (128 requests), 28.9 / 30.5 / 35.1 at 1,280 rows of
//   128 to 1,024 tokens of D 128, 55.2 / 59.7 / 69.6 of D 256 (52.6 with 1). CTAs, 4 against 8: 15.2 / 14.1 at 256 rows of 512
//   to 4,096 tokens of D 64, 23.8 / 23.3 at 32 requests of 512 to 4,096 tokens of D 128, 24.8 / 27.7 at 40 of 100 to 1,000 of D 256.
constexpr double kWarpRowsPerSm = 2.5;
constexpr int kMinCtaPages = 4;
int row_cost(int dim, int team) { return team > 1 ? 1024 / dim : dim == 64 ? 6 : 256 / dim; }
constexpr int kJoinFan = 40;

// Row strides in elements: multiples of 8 (16-byte vectors), at least one row wide.
bool stride_ok(int64_t s, int64_t width) { return s >= width && s % 8 == 0; }

// Subgroups that the join of m segments is cut into (1: none). A CTA joins a slot in about 0.1 us, a second level
// costs up to 2 us: one request of 65,536 tokens and one KV head (D 128, 256 segments) took 24.7 us with one
// level and 11.0 with two; 8 x 8,192 tokens (32 segments each) 9.7 with one and 9.85 with two, of 4 KV heads 17.3 and 18.7.
int join_subgroups(int m) {
  if (m <= kJoinFan) return 1;
  int size = 1;
  while (size * size < m) ++size;
  return (m + size - 1) / size;
}

// What a worker's time is made of, in microseconds (rough, from timelines of the kernel): its pages, each started
// segment, and each partial that it writes or joins.
struct Times {
  double page, segment, partial;
};
Times worker_times(int dim, int group, int team) {
  const double unit = (dim == 256 ? 1.2 : 0.9) * (group > 8 ? 1.3 : 1.0);      // 8 KB by one warp
  return {unit * (2.0 * kPage * dim / 8192) / team, team == 1 ? 1.0 : 2.5, team == 1 ? 2.5 : 3.0};
}

// Rows kept whole, consecutive rows to a worker: the least makespan for `workers`, by bisection, and its ranges.
double whole_rows(const std::vector<int32_t>& pages, int workers, const Times& t, std::vector<int32_t>& wptr) {
  auto fill = [&](double budget, int32_t* ptr) {
    size_t i = 0;
    for (int w = 0; w < workers; ++w) {
      if (ptr) ptr[w] = static_cast<int32_t>(i);
      double sum = 0.0;
      while (i < pages.size() && (sum += pages[i] * t.page + t.segment) <= budget) ++i;
    }
    if (ptr) ptr[workers] = static_cast<int32_t>(i);
    return i == pages.size();
  };
  double longest = 0.0, mean = 0.0;
  for (int32_t p : pages) {
    longest = std::max(longest, p * t.page + t.segment);
    mean += p * t.page + t.segment;
  }
  mean /= workers;
  // filled up to the mean and the longest row, a worker holds more than the mean, so every row finds a place
  double lo = std::max(longest, mean), hi = (mean + longest) * 1.000001;
  for (int i = 0; i < 12 && hi > lo * 1.01; ++i) {
    const double mid = 0.5 * (lo + hi);
    if (fill(mid, nullptr)) hi = mid; else lo = mid;
  }
  wptr.resize(workers + 1);
  fill(hi, wptr.data());
  return hi;
}

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
  if (n_tokens == 0) return QKVP_OK;       // of empty arrays, which may have no addresses
  if ((q_pe != nullptr) != (q != nullptr) || (q_pe != nullptr) != (num_heads > 0)) return QKVP_E_INVALID;
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
  if (n_tokens > INT32_MAX || max_positions > INT32_MAX) return QKVP_E_UNSUPPORTED;
  if (n_tokens == 0) return QKVP_OK;       // of empty arrays, which may have no addresses
  if ((q != nullptr) != (q_out != nullptr) || (q != nullptr) != (num_heads > 0)) return QKVP_E_INVALID;
  if (batch == 0) return QKVP_OK;
  if (!k || !v || !tok_indptr || !kv_len || !kv_indptr || (!kv_indices && nnz > 0) || !kv_data || !kv_scale) return QKVP_E_INVALID;
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

  // Workers are CTAs where there are few rows: their four warps share a row and join at its end. With many rows, or
  // as many as SMs but short ones, they are single warps, which need no barrier.
  const int64_t units = row_pages * (kPage * head_dim / 4096);
  const int team = rows >= static_cast<int64_t>(kWarpRowsPerSm * num_sms) || (rows >= num_sms && units <= 8 * rows) ? 1 : 4;
  const int per_cta = 4 / team, min_pages = team == 1 ? 1 : kMinCtaPages;
  const int64_t useful = std::max<int64_t>(1, (row_pages + min_pages - 1) / min_pages);
  int workers = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(num_sms) * gqa_ctas_per_sm(head_dim, group) * per_cta, useful));
  workers = (workers + per_cta - 1) / per_cta * per_cta;
  const int cost = row_cost(head_dim, team);
  SplitInfo info;
  info.num_segments = rows + workers;      // each worker's end cuts one row at most; asked-for splits are counted first
  if (min_splits > 0) split_pages(indptr.data(), len.data(), static_cast<int>(rows), workers, min_splits, SplitOut{}, info, cost);
  std::vector<Segment> cut(static_cast<size_t>(std::max<int64_t>(1, info.num_segments)));
  std::vector<int32_t> wptr(workers + 1), rptr(rows + 1), wide(std::max<int64_t>(1, rows));
  SplitOut out{cut.data(), info.num_segments, wptr.data(), rptr.data(), wide.data()};
  if (!split_pages(indptr.data(), len.data(), static_cast<int>(rows), workers, min_splits, out, info, cost))
    return QKVP_E_INVALID;
  // Whole rows instead, where that does not take longer: the bandwidth is shared, so a worker with less than the
  // others costs nothing while the others keep the memory busy, and partials do cost. (128 x 2,048 tokens of 8 KV
  // heads, D 128: 81 us whole, 88 split evenly.)
  if (min_splits == 0 && info.partials > 0) {
    const Times times = worker_times(head_dim, group, team);
    double split_us = 0.0;
    for (int w = 0; w < workers; ++w) {
      double sum = 0.0;
      for (int32_t i = wptr[w]; i < wptr[w + 1]; ++i)
        sum += cut[i].num_pages * times.page + times.segment + (cut[i].partial >= 0 ? times.partial : 0.0);
      split_us = std::max(split_us, sum);
    }
    const double memory_us = static_cast<double>(row_pages) * 2 * kPage * head_dim / 6.7e6;
    std::vector<int32_t> whole;
    std::vector<int32_t> row_len(rows);
    for (int64_t i = 0; i < rows; ++i) row_len[i] = len[i] / kPage;
    if (whole_rows(row_len, workers, times, whole) <= std::max(split_us, 0.8 * memory_us)) {
      cut.clear();
      info.num_segments = info.partials = info.split_reqs = info.max_req_segs = 0;
      info.max_pages = 0;
      info.min_pages = INT32_MAX;
      for (int w = 0; w < workers; ++w) {
        wptr[w] = static_cast<int32_t>(cut.size());
        int32_t held = 0;
        for (int32_t i = whole[w]; i < whole[w + 1]; ++i) {
          if (len[i] == 0) continue;
          Segment g{};
          g.req = i;
          g.page_begin = indptr[i];
          g.num_pages = row_len[i];
          g.partial = -1;
          held += row_len[i];
          cut.push_back(g);
        }
        info.max_pages = std::max(info.max_pages, held);
        info.min_pages = std::min(info.min_pages, held);
      }
      info.num_segments = static_cast<int64_t>(cut.size());
      info.max_req_segs = 1;
      wptr[workers] = static_cast<int32_t>(cut.size());
      int32_t at = 0;
      for (int64_t i = 0; i < rows; ++i) {
        rptr[i] = at;
        at += len[i] > 0;
      }
      rptr[rows] = at;
    }
  }
  // rows without a visible page get a segment of no pages, which writes zeros: appended to the workers in turn
  const int64_t empty = info.empty_reqs;
  const int64_t total = info.num_segments + empty;
  // the joins: their counters, and the slots of the subgroups behind those of the segments
  int64_t counters = 0, slots = info.partials;
  for (int64_t i = 0; i < rows; ++i) {
    const int m = rptr[i + 1] - rptr[i];
    if (m < 2) continue;
    const int subs = join_subgroups(m);
    counters += subs > 1 ? subs + 1 : 1;
    if (subs > 1) slots += subs;
  }
  if (slots > INT32_MAX || total > INT32_MAX) return QKVP_E_UNSUPPORTED;
  const GqaTable t = gqa_table(total, workers, counters);

  plan->batch = batch;
  plan->num_heads = num_heads;
  plan->num_kv_heads = num_kv_heads;
  plan->head_dim = head_dim;
  plan->page_size = page_size;
  plan->cache_dtype = cache_dtype;
  plan->window = window;
  plan->sinks = sinks;
  plan->num_workers = workers;
  plan->warps_per_worker = team;
  plan->num_segments = static_cast<int32_t>(total);
  plan->num_split_groups = info.split_reqs;
  plan->max_group_segments = info.max_req_segs;
  plan->num_partials = static_cast<int32_t>(slots);
  plan->max_worker_pages = info.max_pages;
  plan->min_worker_pages = info.min_pages;
  plan->table_entries = batch > 0 ? kv_indptr_host[batch] : 0;
  plan->total_pages = pages;
  plan->total_tokens = tokens;
  plan->table_bytes = t.bytes;
  plan->status_offset = t.status;
  plan->partial_o_offset = t.bytes;
  plan->partial_lse_offset = t.bytes + align_up(static_cast<uint64_t>(slots) * kGqaPassHeads * head_dim * 4);
  plan->workspace_bytes = plan->partial_lse_offset + align_up(static_cast<uint64_t>(slots) * kGqaPassHeads * 4);
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
  GqaWorker* work = reinterpret_cast<GqaWorker*>(blob.data() + t.workers);
  std::vector<int32_t> counter(rows, 0), sub_slot(rows, 0);
  int32_t next_counter = 0, next_slot = info.partials;
  for (int64_t i = 0; i < rows; ++i) {
    const int m = rptr[i + 1] - rptr[i];
    if (m < 2) continue;
    const int subs = join_subgroups(m);
    counter[i] = next_counter;
    sub_slot[i] = next_slot;
    next_counter += subs > 1 ? subs + 1 : 1;
    if (subs > 1) next_slot += subs;
  }
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
    g.top_counter = -1;
  };
  int64_t n = 0, next_empty = 0, given = 0;
  for (int w = 0; w < workers; ++w) {
    work[w].begin = static_cast<int32_t>(n);
    for (int32_t i = wptr[w]; i < wptr[w + 1]; ++i) {
      const Segment& s = cut[i];
      GqaSegment& g = segs[n++];
      fill(g, s.req);
      g.page_begin = s.page_begin - indptr[s.req];
      g.num_pages = s.num_pages;
      g.partial = s.partial;
      if (s.partial >= 0) {
        // segment `at` of the row's m; subgroups of `size` consecutive segments where there are many
        const int m = rptr[s.req + 1] - rptr[s.req], at = i - rptr[s.req], subs = join_subgroups(m);
        const int size = (m + subs - 1) / subs, sub = at / size, first = cut[rptr[s.req]].partial;
        g.group_first = first + sub * size;
        g.group_count = std::min(size, m - sub * size);
        g.counter = counter[s.req] + sub;
        if (subs > 1) {
          g.top_first = sub_slot[s.req];
          g.top_count = subs;
          g.top_counter = counter[s.req] + subs;
          g.sub_slot = sub_slot[s.req] + sub;
        }
      }
    }
    for (const int64_t share = empty * (w + 1) / workers; given < share; ++given) {
      while (len[next_empty] > 0) ++next_empty;
      fill(segs[n++], next_empty++);
    }
    work[w].end = static_cast<int32_t>(n);
    if (work[w].begin < work[w].end) work[w].first = segs[work[w].begin];
  }
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
  const GqaTable t = gqa_table(plan->num_segments, plan->num_workers, 0);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  GqaDecodeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.kv = static_cast<const uint8_t*>(kv_data);
  a.kv_scale = kv_scale;
  a.num_pages = num_pages;
  a.kv_indices = kv_indices;
  a.segs = reinterpret_cast<const GqaSegment*>(ws + t.segs);
  a.workers = reinterpret_cast<const GqaWorker*>(ws + t.workers);
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
  a.team = plan->warps_per_worker;
  a.scale_log2 = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
  return launch_gqa_decode(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? QKVP_OK : QKVP_E_CUDA;
}

}  // extern "C"
