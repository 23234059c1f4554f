// Decode attention over a paged 8-bit cache of K and V heads, one scale per (page, K or V, head).
//
// Per query head with its KV head's codes kc, vc and block scales sk, sv, over the visible tokens t:
//   z_t = sm_scale * sk (q . kc_t),  out = sum_t softmax(z)_t sv vc_t,  lse = log sum_t exp z_t.
// One pass over the pages with a running maximum m: l = sum 2^(z' - m), o = sum 2^(z' - m) sv vc, z' = z
// log2(e). A CTA walks the segments of its worker; its warps take tokens of a segment in turn and join
// their (m, l, o) at the end. A group (request, KV head) that is cut into segments leaves normalised FP32
// partials, and the last of its CTAs to arrive joins them by log-sum-exp in segment order.
//
// This form computes on the FP32 units: a warp per page, a lane per D / 32 dims, one token at a time.
#include <cstdint>

#include "qkvp_device.cuh"
#include "qkvp_internal.h"

namespace qkvp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kH = kGqaPassHeads;
constexpr unsigned kFull = 0xffffffffu;

template <bool E4M3>
__device__ __forceinline__ float value8(uint32_t c) {
  if constexpr (E4M3) return dev::e4m3_to_float(c);
  return static_cast<float>(static_cast<int8_t>(c & 0xFFu));
}

__device__ __forceinline__ bool visible(const GqaSegment& s, int64_t t) {
  return t < s.len && (t >= s.win_begin || t < s.sink_end);
}

// First token of visible page v of the segment's request, and its entry of the page table.
__device__ __forceinline__ int64_t page_of(const GqaSegment& s, int v) {
  return v < s.sink_pages ? v : s.win_page + (v - s.sink_pages);
}

// Hands on a segment's normalised output o [heads][D] and base-2 log-sum-exp L [heads] (shared memory):
// to out and lse, or to its partial slot, where the group's last CTA joins all slots in order.
template <int D>
__device__ void finish(const GqaDecodeArgs& a, const GqaSegment& s, const float* o, const float* L, int* flag) {
  const int tid = threadIdx.x;
  const int64_t row0 = static_cast<int64_t>(s.req) * a.heads + s.head0;
  if (s.partial < 0) {
    for (int i = tid; i < s.heads * D / 2; i += kThreads)
      reinterpret_cast<uint32_t*>(a.out + row0 * D)[i] = dev::pack_bf16x2(o[2 * i], o[2 * i + 1]);
    if (a.lse)
      for (int h = tid; h < s.heads; h += kThreads) a.lse[row0 + h] = L[h] * 0.69314718055994531f;
    return;
  }
  float* po = a.part_o + static_cast<int64_t>(s.partial) * kH * D;
  for (int i = tid; i < s.heads * D; i += kThreads) po[i] = o[i];
  for (int h = tid; h < s.heads; h += kThreads) a.part_lse[static_cast<int64_t>(s.partial) * kH + h] = L[h];
  __threadfence();
  __syncthreads();
  if (tid == 0) *flag = atomicAdd(a.counters + s.counter, 1u) == static_cast<unsigned>(s.group_count - 1);
  __syncthreads();
  if (*flag == 0) return;
  __threadfence();
  if (tid == 0) a.counters[s.counter] = 0;      // ready for the next run
  const float* gl = a.part_lse + static_cast<int64_t>(s.group_first) * kH;
  const float* go = a.part_o + static_cast<int64_t>(s.group_first) * kH * D;
  for (int i = tid; i < s.heads * D / 2; i += kThreads) {
    const int h = 2 * i / D;
    float m = -INFINITY;
    for (int k = 0; k < s.group_count; ++k) m = dev::max_nan(m, __ldcg(gl + k * kH + h));
    float w = 0.0f, x = 0.0f, y = 0.0f;
    if (m > -INFINITY) {
      for (int k = 0; k < s.group_count; ++k) {
        const float c = exp2f(__ldcg(gl + k * kH + h) - m);
        const float2 p = __ldcg(reinterpret_cast<const float2*>(go + static_cast<int64_t>(k) * kH * D) + i);
        w += c;
        if (c > 0.0f) {
          x += c * p.x;
          y += c * p.y;
        }
      }
    } else {
      w = m == -INFINITY ? 0.0f : m;               // NaN stays NaN
    }
    const float inv = w == 0.0f ? 0.0f : 1.0f / w;
    reinterpret_cast<uint32_t*>(a.out + row0 * D)[i] = dev::pack_bf16x2(x * inv, y * inv);
    if (a.lse && 2 * i % D == 0) a.lse[row0 + h] = w == 0.0f ? -INFINITY : (m + log2f(w)) * 0.69314718055994531f;
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) gqa_decode_kernel(const GqaDecodeArgs a) {
  constexpr int kE = D / 32;                       // dims of a lane
  extern __shared__ float sm[];
  float* sq = sm;                                  // [kH][D]
  float* so = sq + kH * D;                         // [kWarps][kH][D]
  float* sL = so + kWarps * kH * D;                // [kWarps][kH], then the segment's L [kH]
  int* flag = reinterpret_cast<int*>(sL + kWarps * kH + kH);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  for (int si = a.worker_ptr[blockIdx.x]; si < a.worker_ptr[blockIdx.x + 1]; ++si) {
    const GqaSegment s = a.segs[si];
    __syncthreads();
    for (int i = tid; i < kH * D; i += kThreads) {
      const int h = i / D;
      sq[i] = h < s.heads ? __uint_as_float(static_cast<uint32_t>(a.q[(static_cast<int64_t>(s.req) * a.heads + s.head0 + h) * D + i % D]) << 16) * a.scale_log2 : 0.0f;
    }
    __syncthreads();
    float m[kH], l[kH], acc[kH][kE];
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.0f;
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[h][e] = 0.0f;
    }
    for (int p = warp; p < s.num_pages; p += kWarps) {
      const int64_t local = page_of(s, s.page_begin + p);
      const int64_t page = a.kv_indices[s.page0 + local];
      if (page < 0 || page >= a.num_pages) continue;
      const int64_t kb = page * 2 * a.kv_heads + s.kv_head, vb = kb + a.kv_heads;
      const float sk = a.kv_scale[kb], sv = a.kv_scale[vb];
      const uint8_t* kp = a.kv + kb * kPage * D + lane * kE;
      const uint8_t* vp = a.kv + vb * kPage * D + lane * kE;
      for (int t = 0; t < kPage; ++t) {
        if (!visible(s, local * kPage + t)) continue;
        float k[kE], v[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          k[e] = value8<E4M3>(kp[t * D + e]);
          v[e] = value8<E4M3>(vp[t * D + e]) * sv;
        }
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          if (h >= s.heads) break;
          float z = 0.0f;
#pragma unroll
          for (int e = 0; e < kE; ++e) z += sq[h * D + lane * kE + e] * k[e];
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
          z *= sk;
          const float mn = dev::max_nan(m[h], z);
          const float c = mn == -INFINITY ? 1.0f : exp2f(m[h] - mn);
          const float w = mn == -INFINITY ? 0.0f : exp2f(z - mn);
          m[h] = mn;
          l[h] = l[h] * c + w;
#pragma unroll
          for (int e = 0; e < kE; ++e) acc[h][e] = acc[h][e] * c + w * v[e];
        }
      }
    }
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      const float inv = l[h] == 0.0f ? 0.0f : 1.0f / l[h];
#pragma unroll
      for (int e = 0; e < kE; ++e) so[(warp * kH + h) * D + lane * kE + e] = acc[h][e] * inv;
      if (lane == 0) sL[warp * kH + h] = l[h] == 0.0f ? -INFINITY : m[h] + log2f(l[h]);
    }
    __syncthreads();
    // join the warps: the result replaces warp 0's part
    for (int i = tid; i < s.heads * D; i += kThreads) {
      const int h = i / D;
      float M = -INFINITY, w = 0.0f, x = 0.0f;
      for (int k = 0; k < kWarps; ++k) M = dev::max_nan(M, sL[k * kH + h]);
      for (int k = 0; k < kWarps; ++k) {
        const float c = M == -INFINITY ? 0.0f : exp2f(sL[k * kH + h] - M);
        w += c;
        if (c > 0.0f || c != c) x += c * so[(k * kH + h) * D + i % D];
      }
      so[i] = w == 0.0f ? 0.0f : x / w;
      if (i % D == 0) sL[kWarps * kH + h] = w == 0.0f ? -INFINITY : M + log2f(w);
    }
    __syncthreads();
    finish<D>(a, s, so, sL + kWarps * kH, flag);
  }
}

template <int D>
cudaError_t launch(const GqaDecodeArgs& a, cudaStream_t st) {
  const int bytes = (kH * D * (1 + kWarps) + kWarps * kH + kH + 1) * 4;
  auto kernel = a.cache_dtype == QKVP_CACHE_E4M3 ? gqa_decode_kernel<D, true> : gqa_decode_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<a.num_workers, kThreads, bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gqa_decode(const GqaDecodeArgs& a, cudaStream_t st) {
  switch (a.dim) {
    case 64: return launch<64>(a, st);
    case 128: return launch<128>(a, st);
    default: return launch<256>(a, st);
  }
}

}  // namespace qkvp
