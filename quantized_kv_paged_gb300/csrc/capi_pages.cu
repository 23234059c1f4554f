// C entry points of the pages of a cache: copy, fork, grow, free and compact. Argument checks and dispatch.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/qkvp.h"
#include "qkvp_internal.h"

using namespace qkvp;

namespace {

struct WorkLayout {
  uint64_t claim, marks, src, dst, rank, bytes;
};
WorkLayout work_layout(int64_t num_pages, int64_t rows, int64_t n) {
  const uint64_t most = static_cast<uint64_t>(std::max(n, num_pages));
  WorkLayout w;
  w.claim = kTableAlign;
  w.marks = w.claim + align_up(static_cast<uint64_t>(rows) * 4);
  w.src = w.marks + align_up(static_cast<uint64_t>((num_pages + 31) / 32) * 4);
  w.dst = w.src + align_up(most * 4);
  w.rank = w.dst + align_up(most * 4);
  w.bytes = w.rank + align_up(static_cast<uint64_t>(num_pages) * 4);
  return w;
}

int take_pools(const qkvp_pool* pools, int32_t count, int64_t num_pages, PagePools& p) {
  if (count < 0 || (count > 0 && !pools)) return QKVP_E_INVALID;
  if (count > kMaxPools) return QKVP_E_UNSUPPORTED;
  p = PagePools{};
  int64_t units = 0;
  for (int i = 0; i < count; ++i) {
    const int64_t bytes = pools[i].page_bytes;
    if (!pools[i].data || bytes <= 0 || bytes % 4 || !aligned(pools[i].data, 4)) return QKVP_E_INVALID;
    if (num_pages > 0 && bytes > INT64_MAX / num_pages) return QKVP_E_INVALID;
    if (bytes > (1 << 30)) return QKVP_E_UNSUPPORTED;
    p.base[i] = static_cast<uint8_t*>(pools[i].data);
    p.bytes[i] = static_cast<uint32_t>(bytes);
    p.first_unit[i] = static_cast<uint32_t>(units);
    units += (bytes + kCopyUnit - 1) / kCopyUnit;
  }
  p.units = static_cast<uint32_t>(units);
  p.count = count;
  return QKVP_OK;
}

int take_state(const qkvp_page_state* s, int64_t n, void* workspace, uint64_t workspace_bytes, PageState& t, PageWork& ws) {
  if (!s || s->rows < 0 || s->row_pages < 0 || s->num_pages < 0 || n < 0) return QKVP_E_INVALID;
  if (s->num_pages > INT32_MAX) return QKVP_E_UNSUPPORTED;
  if ((s->rows > 0 && (!s->held || !s->lens || (s->row_pages > 0 && !s->table))) || !s->free_count ||
      (s->num_pages > 0 && (!s->refs || !s->free_list)))
    return QKVP_E_INVALID;
  if (!aligned(s->table, 4) || !aligned(s->held, 4) || !aligned(s->lens, 4) || !aligned(s->refs, 4) || !aligned(s->free_list, 4) ||
      !aligned(s->free_count, 4))
    return QKVP_E_INVALID;
  const WorkLayout w = work_layout(s->num_pages, s->rows, n);
  if (!workspace || workspace_bytes < w.bytes || !aligned(workspace, kTableAlign)) return QKVP_E_WORKSPACE;
  t = PageState{s->table, s->held, s->lens, s->refs, s->free_list, s->free_count, s->rows, s->row_pages, s->num_pages};
  uint8_t* at = static_cast<uint8_t*>(workspace);
  ws.arrived = reinterpret_cast<int32_t*>(at);
  ws.moves = ws.arrived + 1;
  ws.claim = reinterpret_cast<int32_t*>(at + w.claim);
  ws.marks = reinterpret_cast<uint32_t*>(at + w.marks);
  ws.src = reinterpret_cast<int32_t*>(at + w.src);
  ws.dst = reinterpret_cast<int32_t*>(at + w.dst);
  ws.rank = reinterpret_cast<int32_t*>(at + w.rank);
  return QKVP_OK;
}

bool list_ok(const void* p) { return p && aligned(p, 4); }
int status_of(cudaError_t e) { return e == cudaSuccess ? QKVP_OK : QKVP_E_CUDA; }

}  // namespace

extern "C" {

int kv_pages_workspace(int64_t num_pages, int32_t rows, int32_t n, uint64_t* bytes) {
  if (!bytes || num_pages < 0 || rows < 0 || n < 0) return QKVP_E_INVALID;
  if (num_pages > INT32_MAX) return QKVP_E_UNSUPPORTED;
  *bytes = work_layout(num_pages, rows, n).bytes;
  return QKVP_OK;
}

int kv_pages_copy(const qkvp_pool* pools, int32_t num_pools, const int32_t* src, const int32_t* dst, int64_t n, int64_t num_pages,
                  qkvp_stream_t stream) {
  if (n < 0 || num_pages < 0) return QKVP_E_INVALID;
  if (num_pages > INT32_MAX) return QKVP_E_UNSUPPORTED;
  PagePools p;
  const int st = take_pools(pools, num_pools, num_pages, p);
  if (st != QKVP_OK) return st;
  if (n == 0 || num_pools == 0) return QKVP_OK;
  if (!list_ok(src) || !list_ok(dst)) return QKVP_E_INVALID;
  if (n > INT64_MAX / p.units) return QKVP_E_UNSUPPORTED;
  const int sms = query_sms();
  if (sms <= 0) return QKVP_E_CUDA;
  return status_of(launch_pages_copy(p, src, dst, n, num_pages, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int kv_pages_fork(const qkvp_pool* pools, int32_t num_pools, const qkvp_page_state* state, const int32_t* parents, const int32_t* children,
                  int32_t n, int32_t* status, void* workspace, uint64_t workspace_bytes, qkvp_stream_t stream) {
  PageState t;
  PageWork ws;
  PagePools p;
  int st = take_state(state, n, workspace, workspace_bytes, t, ws);
  if (st == QKVP_OK) st = take_pools(pools, num_pools, t.num_pages, p);
  if (st != QKVP_OK) return st;
  if (n == 0) return QKVP_OK;
  if (!list_ok(parents) || !list_ok(children) || !list_ok(status)) return QKVP_E_INVALID;
  const int sms = query_sms();
  if (sms <= 0) return QKVP_E_CUDA;
  return status_of(launch_pages_fork(p, t, parents, children, n, status, ws, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int kv_pages_grow(const qkvp_page_state* state, const int32_t* list, const int32_t* tokens, int32_t n, int32_t* status, void* workspace,
                  uint64_t workspace_bytes, qkvp_stream_t stream) {
  PageState t;
  PageWork ws;
  const int st = take_state(state, n, workspace, workspace_bytes, t, ws);
  if (st != QKVP_OK || n == 0) return st;
  if (!list_ok(list) || !list_ok(tokens) || !list_ok(status)) return QKVP_E_INVALID;
  return status_of(launch_pages_grow(t, list, tokens, n, status, ws, reinterpret_cast<cudaStream_t>(stream)));
}

int kv_pages_free(const qkvp_page_state* state, const int32_t* list, int32_t n, void* workspace, uint64_t workspace_bytes, qkvp_stream_t stream) {
  PageState t;
  PageWork ws;
  const int st = take_state(state, n, workspace, workspace_bytes, t, ws);
  if (st != QKVP_OK || n == 0) return st;
  if (!list_ok(list)) return QKVP_E_INVALID;
  return status_of(launch_pages_free(t, list, n, ws, reinterpret_cast<cudaStream_t>(stream)));
}

int kv_pages_compact(const qkvp_pool* pools, int32_t num_pools, const qkvp_page_state* state, void* workspace, uint64_t workspace_bytes,
                     qkvp_stream_t stream) {
  PageState t;
  PageWork ws;
  PagePools p;
  int st = take_state(state, 0, workspace, workspace_bytes, t, ws);
  if (st == QKVP_OK) st = take_pools(pools, num_pools, t.num_pages, p);
  if (st != QKVP_OK || t.num_pages == 0) return st;
  const int sms = query_sms();
  if (sms <= 0) return QKVP_E_CUDA;
  return status_of(launch_pages_compact(p, t, ws, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
