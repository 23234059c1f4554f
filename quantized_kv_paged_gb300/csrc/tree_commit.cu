// The end of a verified step: the accepted drafted tokens of each request move to the slots right behind its cached
// tokens, in every layer of a head pool.
//
// A warp has one (request, layer, K or V, head), whose blocks nobody else touches: the blocks that take tokens are walked in
// order, so a block's scale changes only after the blocks before it have read from it, and within a block the tokens go in
// order of the path, each no later than where it comes from, a batch of them in registers between the loads and
// the stores. A token from another block is requantized; the amax of those decides how far the block's scale grows.
// What bounds it is the chain path -> page id -> scale -> codes, four dependent reads, and the number of 64 to 256 byte rows.
#include <cstdint>

#include "qkvp_device.cuh"
#include "qkvp_internal.h"

namespace qkvp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;

template <bool E4M3>
__device__ __forceinline__ float value_of(uint32_t byte) {
  return E4M3 ? dev::e4m3_to_float(byte) : static_cast<float>(static_cast<int8_t>(byte));
}
template <bool E4M3>
__device__ __forceinline__ uint32_t code_of(float x) {
  if (E4M3) return dev::encode_e4m3(x);
  if (x != x) return 0;
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(x), -127.0f), 127.0f))) & 0xFFu;
}

// Every byte of the 16 through f.
template <class F>
__device__ __forceinline__ uint4 each_byte(uint4 v, F f) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) r |= f(w[i] >> (8 * b) & 0xFFu) << (8 * b);
    w[i] = r;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) tree_commit_kernel(const __grid_constant__ TreeCommitArgs a) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;      // lanes of a token's row, rows at a time
  constexpr int kU = 4, kBatch = kU * kRows;               // tokens between loads and stores
  dev::wait_for_previous();
  dev::allow_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int per = 2 * a.kv_heads;
  if (job >= static_cast<int64_t>(a.batch) * a.layers * per) return;
  const int r = static_cast<int>(job / (static_cast<int64_t>(a.layers) * per));
  const int rest = static_cast<int>(job % (static_cast<int64_t>(a.layers) * per)), layer = rest / per, block = rest % per;
  const int n = a.path_len[r];
  if (n <= 0 || n > a.max_path) return;
  const int32_t* path = a.path + static_cast<int64_t>(r) * a.max_path;
  const int64_t held = a.kv_len[r], first = a.kv_indptr[r], last = min(static_cast<int64_t>(a.kv_indptr[r + 1]), a.nnz);
  // the page of a token of the request, or -1
  auto page_of = [&](int64_t pos) -> int64_t {
    const int64_t e = first + pos / kPage;
    if (pos < 0 || first < 0 || e >= last) return -1;
    const int64_t page = a.kv_indices[e];
    return page < a.num_pages ? page : -1;
  };
  // a path that does not ascend, or leaves the request's pages, changes nothing; one that stays in its place neither
  bool bad = held < 0, moves = false;
  for (int k = lane; k < n; k += 32) {
    const int p = path[k];
    bad |= p < k || (k > 0 && p <= path[k - 1]) || page_of(held + p) < 0 || page_of(held + k) < 0;
    moves |= p != k;
  }
  if (__any_sync(kFull, bad) || !__any_sync(kFull, moves)) return;

  uint8_t* codes = a.kv[layer] + static_cast<int64_t>(block) * kPage * D;
  float* scales = a.scale[layer] + block;
  const int64_t page_codes = static_cast<int64_t>(per) * kPage * D;
  const int sub = lane / kLanes, part = lane % kLanes;
  for (int k0 = 0; k0 < n;) {
    const int64_t to = page_of(held + k0);
    const int at0 = static_cast<int>((held + k0) % kPage), count = min(n - k0, kPage - at0);
    uint8_t* dst = codes + to * page_codes;
    const float old = scales[to * per];
    uint4 v[kU];
    float s[kU];                 // scale of the block that a token comes from; -1: from the block itself
    auto load = [&](int base) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int k = base + u * kRows + sub;
        v[u] = make_uint4(0, 0, 0, 0);
        s[u] = -1.0f;
        if (k < k0 + count) {
          const int64_t pos = held + path[k], from = page_of(pos);
          v[u] = *reinterpret_cast<const uint4*>(codes + from * page_codes + (pos % kPage) * D + 16 * part);
          if (from != to) s[u] = scales[from * per];
        }
      }
    };
    // the largest finite |x| that comes from other blocks
    float amax = 0.0f;
    for (int base = k0; base < k0 + count; base += kBatch) {
      load(base);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (s[u] >= 0.0f)
          each_byte(v[u], [&](uint32_t c) {
            const float x = fabsf(__fmul_rn(value_of<E4M3>(c), s[u]));
            if (x <= 3.402823466e38f) amax = fmaxf(amax, x);
            return 0u;
          });
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const float need = __fdiv_rn(amax, E4M3 ? 448.0f : 127.0f);
    int j = 0;
    float scale = old;
    if (old == 0.0f) {
      scale = need;
    } else if (need > old) {
      int e_need, e_old;
      const float m_need = frexpf(need, &e_need), m_old = frexpf(old, &e_old);
      j = e_need - e_old + (m_need > m_old ? 1 : 0);
      scale = ldexpf(old, j);
    }
    auto shrink = [&](uint4 x) {
      return each_byte(x, [&](uint32_t c) { return code_of<E4M3>(ldexpf(value_of<E4M3>(c), -j)); });
    };
    if (j > 0)
      for (int o = sub; o < at0; o += kRows) {
        uint4* at = reinterpret_cast<uint4*>(dst + o * D + 16 * part);
        *at = shrink(*at);
      }
    for (int base = k0; base < k0 + count; base += kBatch) {
      if (count > kBatch) load(base);            // otherwise they are there
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int k = base + u * kRows + sub;
        if (k >= k0 + count) continue;
        uint4 x = v[u];
        if (s[u] >= 0.0f)
          x = each_byte(x, [&](uint32_t c) {
            const float y = __fmul_rn(value_of<E4M3>(c), s[u]);
            return code_of<E4M3>(scale > 0.0f ? __fdiv_rn(y, scale) : y);
          });
        else if (j > 0) x = shrink(x);
        *reinterpret_cast<uint4*>(dst + (at0 + k - k0) * D + 16 * part) = x;
      }
      __syncwarp();
    }
    if (lane == 0 && scale != old) scales[to * per] = scale;
    k0 += count;
  }
}

template <int D>
cudaError_t launch_dim(const TreeCommitArgs& a, unsigned grid, cudaStream_t s) {
  return a.cache_dtype == QKVP_CACHE_E4M3 ? launch_overlapped(tree_commit_kernel<D, true>, grid, 32 * kWarps, 0, s, a)
                                          : launch_overlapped(tree_commit_kernel<D, false>, grid, 32 * kWarps, 0, s, a);
}

}  // namespace

cudaError_t launch_tree_commit(const TreeCommitArgs& a, cudaStream_t s) {
  const int64_t jobs = static_cast<int64_t>(a.batch) * a.layers * 2 * a.kv_heads;
  const int64_t grid = (jobs + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  switch (a.dim) {
    case 64: return launch_dim<64>(a, static_cast<unsigned>(grid), s);
    case 128: return launch_dim<128>(a, static_cast<unsigned>(grid), s);
    case 256: return launch_dim<256>(a, static_cast<unsigned>(grid), s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qkvp
