// Appends that apply the rotary position embedding on the way into a quantized cache.
//
// Rotation of pair i at position p: (a, b) -> (a c - b s, b c + a s) with c = cos_sin[p][i] and
// s = cos_sin[p][r/2 + i]; the table is the caller's, so no angle is computed here and positions far out
// cost no precision. Every product and sum is one FP32 rounding (no contraction), which makes the codes
// reproducible bit for bit by any other implementation of the same formula.
//
// Both kernels are streams: BF16 in, 8-bit codes (and BF16 queries) out, each byte once. A lane holds 16
// bytes = 8 dims of a head; where a pair's halves lie r/2 dims apart its partner's 8 dims come from the
// lane r/16 further on by shuffle, so no element is loaded twice.
#include <algorithm>
#include <cstdint>

#include "qkvp_device.cuh"
#include "qkvp_internal.h"

namespace qkvp {
namespace {

constexpr int kRope = kLatent - kDv;    // 64 rope dims of the latent
constexpr int kBlocks = kLatent / 16;   // 36 blocks of 16 elements per latent row
constexpr int kFull = 0xffffffff;

__device__ __forceinline__ float rot_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rot_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

__device__ __forceinline__ uint4 shfl4(uint4 v, int src) {
  return make_uint4(__shfl_sync(kFull, v.x, src), __shfl_sync(kFull, v.y, src), __shfl_sync(kFull, v.z, src),
                    __shfl_sync(kFull, v.w, src));
}

// cos and sin of the pairs that 8 consecutive dims (chunk c8 of a head, dims 8 c8 ..) belong to. PAIRS:
// four pairs, HALVES: eight.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(Turn& t, const float* row, int rot, int c8, int style) {
  if (style == QKVP_ROPE_PAIRS) {
    const float4 c = *reinterpret_cast<const float4*>(row + 4 * c8), s = *reinterpret_cast<const float4*>(row + rot / 2 + 4 * c8);
    t.c[0] = c.x; t.c[1] = c.y; t.c[2] = c.z; t.c[3] = c.w;
    t.s[0] = s.x; t.s[1] = s.y; t.s[2] = s.z; t.s[3] = s.w;
  } else {
    const int i = 8 * c8 < rot / 2 ? 8 * c8 : 8 * c8 - rot / 2;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 c = *reinterpret_cast<const float4*>(row + i + 4 * k), s = *reinterpret_cast<const float4*>(row + rot / 2 + i + 4 * k);
      t.c[4 * k] = c.x; t.c[4 * k + 1] = c.y; t.c[4 * k + 2] = c.z; t.c[4 * k + 3] = c.w;
      t.s[4 * k] = s.x; t.s[4 * k + 1] = s.y; t.s[4 * k + 2] = s.z; t.s[4 * k + 3] = s.w;
    }
  }
}

// Rotates the 8 dims x of chunk c8; `other` holds the partner chunk's 8 dims (HALVES only).
__device__ __forceinline__ void turn8(float (&x)[8], const float (&other)[8], const Turn& t, int rot, int c8, int style) {
  if (style == QKVP_ROPE_PAIRS) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = rot_a(a, b, t.c[i], t.s[i]);
      x[2 * i + 1] = rot_b(a, b, t.c[i], t.s[i]);
    }
  } else if (8 * c8 < rot / 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = rot_a(x[i], other[i], t.c[i], t.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = rot_b(other[i], x[i], t.c[i], t.s[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(dev::pack_bf16x2(x[0], x[1]), dev::pack_bf16x2(x[2], x[3]), dev::pack_bf16x2(x[4], x[5]),
                    dev::pack_bf16x2(x[6], x[7]));
}

// ------------------------------------------------------------------------------------------------
// Latent rows. One warp per token, or per (token, 16 query heads): a decode step of 44 tokens and 128
// heads is 44 + 352 warps, enough to reach every SM; with a warp for all 128 heads it was 44 + 44.
// ------------------------------------------------------------------------------------------------
constexpr int kLatentThreads = 128;
constexpr int kQHeads = 16;             // query heads per warp
constexpr int kRopeLanes = kRope / 8;   // 8 lanes hold one head's 64 dims

__global__ void __launch_bounds__(kLatentThreads) mla_append_rope_kernel(const MlaAppendArgs a) {
  const int64_t job = (static_cast<int64_t>(blockIdx.x) * kLatentThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int head_jobs = (a.heads + kQHeads - 1) / kQHeads;
  if (job >= a.n * (1 + head_jobs)) return;       // the whole warp
  if (job >= a.n) {
    // query heads h0 .. h0 + 15 of one token, four at a time, 8 lanes each
    const int64_t tok = (job - a.n) / head_jobs;
    const int h0 = static_cast<int>((job - a.n) % head_jobs) * kQHeads;
    const int64_t pos = a.positions[tok];
    if (pos < 0 || pos >= a.max_pos) return;
    const int c8 = lane % kRopeLanes, hl = lane / kRopeLanes;
    const uint16_t* src = a.q_pe + tok * a.q_pe_tok + c8 * 8;
    uint4 raw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int h = h0 + 4 * k + hl;
      raw[k] = h < a.heads ? *reinterpret_cast<const uint4*>(src + h * a.q_pe_head) : make_uint4(0, 0, 0, 0);
    }
    Turn t;
    load_turn(t, a.cos_sin + pos * kRope, kRope, c8, a.style);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int h = h0 + 4 * k + hl;
      const uint4 far = shfl4(raw[k], lane ^ (kRopeLanes / 2));
      float x[8], o[8];
      dev::bf16x8_to_float(raw[k], x);
      dev::bf16x8_to_float(far, o);
      turn8(x, o, t, kRope, c8, a.style);
      if (h < a.heads) *reinterpret_cast<uint4*>(a.q + (tok * a.heads + h) * kLatent + kDv + c8 * 8) = pack8(x);
    }
    return;
  }
  // the latent row: lane l quantizes block l of c_kv, lanes 0..3 also the rotated blocks 32..35
  const int64_t tok = job;
  const int64_t slot = a.slots[tok], pos = a.positions[tok];
  if (slot < 0 || slot >= a.num_slots || pos < 0 || pos >= a.max_pos) return;
  constexpr int kExtra = kBlocks - 32;
  float x0[16], x1[16];
  {
    const uint4* p = reinterpret_cast<const uint4*>(a.c_kv + tok * a.c_kv_stride + lane * 16);
    dev::bf16x8_to_float(p[0], x0);
    dev::bf16x8_to_float(p[1], x0 + 8);
  }
  uint4 pe[2] = {};
  if (lane < kExtra) {
    const uint4* p = reinterpret_cast<const uint4*>(a.k_pe + tok * a.k_pe_stride + lane * 16);
    pe[0] = p[0];
    pe[1] = p[1];
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 far = shfl4(pe[k], lane ^ (kExtra / 2));      // 32 dims further
    if (lane < kExtra) {
      const int c8 = 2 * lane + k;
      float x[8], o[8];
      Turn t;
      load_turn(t, a.cos_sin + pos * kRope, kRope, c8, a.style);
      dev::bf16x8_to_float(pe[k], x);
      dev::bf16x8_to_float(far, o);
      turn8(x, o, t, kRope, c8, a.style);
#pragma unroll
      for (int i = 0; i < 8; ++i) x1[8 * k + i] = x[i];
    }
  }
  if (a.kv_dtype == KV_NVFP4) {
    uint32_t s8;
    const uint2 w = dev::encode_nvfp4_block(x0, a.g, s8);
    *reinterpret_cast<uint2*>(a.kv + slot * kPacked + lane * 8) = w;
    a.kv_scale[slot * kScales + lane] = static_cast<uint8_t>(s8);
    if (lane < kExtra) {
      const uint2 w1 = dev::encode_nvfp4_block(x1, a.g, s8);
      *reinterpret_cast<uint2*>(a.kv + slot * kPacked + (32 + lane) * 8) = w1;
      a.kv_scale[slot * kScales + 32 + lane] = static_cast<uint8_t>(s8);
    }
  } else if (a.kv_dtype == KV_FP8) {
    uint8_t* row = a.kv + slot * kLatent;
    *reinterpret_cast<uint4*>(row + lane * 16) = dev::encode_e4m3_plain(x0);
    if (lane < kExtra) *reinterpret_cast<uint4*>(row + (32 + lane) * 16) = dev::encode_e4m3_plain(x1);
  } else {
    float amax = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      nan |= (x0[i] != x0[i]);
      amax = fmaxf(amax, fabsf(x0[i]));
      if (lane < kExtra) {
        nan |= (x1[i] != x1[i]);
        amax = fmaxf(amax, fabsf(x1[i]));
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const float sc = __any_sync(kFull, nan) ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 448.0f);
    uint8_t* page = a.kv + (slot / kPage) * kPtPageBytes;
    uint8_t* row = page + (slot % kPage) * kLatent;
    *reinterpret_cast<uint4*>(row + lane * 16) = dev::encode_e4m3_scaled(x0, sc);
    if (lane < kExtra) *reinterpret_cast<uint4*>(row + (32 + lane) * 16) = dev::encode_e4m3_scaled(x1, sc);
    if (lane == 0) *reinterpret_cast<float*>(page + kPtScaleOff + (slot % kPage) * 4) = sc;
  }
}

// ------------------------------------------------------------------------------------------------
// K and V heads. One CTA per (page that the call writes, K or V, head): the block's scale needs the
// amax of all the page's new tokens, and its older codes change with it, so a block has one owner and
// no atomics. The CTA keeps the new elements in registers between the amax and the codes.
//
// Which pages are written is known on the device only. The launch has, for request r, floor(n_r / 64) + 2
// candidates, the most pages that n_r tokens can touch: job c belongs to the last request with
// tok_indptr[r] / 64 + 2 r <= c. With few tokens there is a job per token instead, and the first token of
// each page does the work. Idle jobs leave after the search.
// ------------------------------------------------------------------------------------------------
constexpr int kHeadThreads = 256;

// The largest r in [0, batch) with f(r) <= c for a non-decreasing f with f(0) <= c (0 if there is none):
// 32 probes at a time, so two dependent loads for up to 1,024 requests.
template <class F>
__device__ __forceinline__ int last_at_most(int batch, int64_t c, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int off = lane * step;
    const unsigned hit = __ballot_sync(kFull, off < n && f(lo + off) <= c);
    const int k = max(__popc(hit) - 1, 0) * step;
    lo += k;
    n = min(step, n - k);
  }
  return lo;
}

struct Place {
  int64_t page;        // pool page, -1: none
  int64_t tok, pos;    // source row and cache position of the token at offset `first`
  int first, last;     // the page's new tokens are the offsets [first, last)
};

// The clipped token range of request r.
__device__ __forceinline__ void request_tokens(const GqaAppendArgs& a, int r, int64_t& t0, int64_t& t1) {
  t0 = min(max(static_cast<int64_t>(a.tok_indptr[r]), int64_t(0)), a.n);
  t1 = min(max(static_cast<int64_t>(a.tok_indptr[r + 1]), t0), a.n);
}

__device__ __forceinline__ Place find_place(const GqaAppendArgs& a, int64_t job) {
  Place p{-1, 0, 0, 0, 0};
  const int32_t* tp = a.tok_indptr;
  const int r = a.per_token ? last_at_most(a.batch, job, [tp](int i) { return static_cast<int64_t>(tp[i]); })
                            : last_at_most(a.batch, job, [tp](int i) { return static_cast<int64_t>(tp[i] / kPage) + 2ll * i; });
  int64_t t0, t1;
  request_tokens(a, r, t0, t1);
  const int64_t held = a.kv_len[r];
  const int64_t p0 = a.kv_indptr[r], p1 = a.kv_indptr[r + 1];
  if (held < 0 || t0 >= t1) return p;
  int64_t local;                         // page of the request
  if (a.per_token) {
    if (job < t0 || job >= t1) return p;
    const int64_t pos = held + job - t0;
    if (job != t0 && pos % kPage != 0) return p;
    local = pos / kPage;
  } else {
    local = held / kPage + (job - (static_cast<int64_t>(tp[r] / kPage) + 2ll * r));
  }
  const int64_t lo = max(held, local * kPage), hi = min(held + t1 - t0, (local + 1) * kPage);
  const int64_t e = p0 + local;
  if (lo >= hi || p0 < 0 || e < p0 || e >= p1 || e >= a.nnz) return p;
  const int64_t page = a.kv_indices[e];
  if (page < 0 || page >= a.num_pages) return p;
  p.page = page;
  p.tok = t0 + lo - held;
  p.pos = lo;
  p.first = static_cast<int>(lo - local * kPage);
  p.last = static_cast<int>(hi - local * kPage);
  return p;
}

template <bool E4M3>
__device__ __forceinline__ uint32_t encode8(float x) {
  if constexpr (E4M3) return dev::encode_e4m3(x);
  const float c = fminf(fmaxf(rintf(x), -127.0f), 127.0f);
  return x != x ? 0u : static_cast<uint32_t>(static_cast<int>(c)) & 0xFFu;
}
template <bool E4M3>
__device__ __forceinline__ float decode8(uint32_t c) {
  if constexpr (E4M3) return dev::e4m3_to_float(c);
  return static_cast<float>(static_cast<int8_t>(c & 0xFFu));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kHeadThreads) gqa_append_rope_kernel(const GqaAppendArgs a) {
  constexpr int kLanes = D / 8;                    // lanes of one token's head
  constexpr int kTok = kHeadThreads / kLanes;      // tokens of one pass over the CTA
  constexpr int kPasses = kPage / kTok;
  const int lane = threadIdx.x & 31, c8 = threadIdx.x % kLanes;
  const int partner = (lane & ~(kLanes - 1)) | ((c8 + (8 * c8 < a.rot / 2 ? a.rot / 16 : -(a.rot / 16))) & (kLanes - 1));
  const bool turned = 8 * c8 < a.rot;
  if (blockIdx.x >= a.kv_ctas) {
    // query heads: a warp per (token, 4 passes of heads)
    constexpr int kH = 32 / kLanes;                // heads of one pass over the warp
    const int64_t job = ((static_cast<int64_t>(blockIdx.x) - a.kv_ctas) * kHeadThreads + threadIdx.x) >> 5;
    const int head_jobs = (a.heads + 4 * kH - 1) / (4 * kH);
    if (job >= a.n * head_jobs) return;
    const int64_t tok = job / head_jobs;
    const int h0 = static_cast<int>(job % head_jobs) * 4 * kH + lane / kLanes;
    const int32_t* tp = a.tok_indptr;
    const int r = last_at_most(a.batch, tok, [tp](int i) { return static_cast<int64_t>(tp[i]); });
    int64_t t0, t1;
    request_tokens(a, r, t0, t1);
    if (tok < t0 || tok >= t1) return;             // padding
    const int64_t pos = a.positions ? a.positions[tok] : a.kv_len[r] + tok - t0;
    if (a.rot > 0 && (pos < 0 || pos >= a.max_pos)) return;
    uint4 raw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int h = h0 + k * kH;
      raw[k] = h < a.heads ? *reinterpret_cast<const uint4*>(a.q + tok * a.q_stride + h * D + c8 * 8) : make_uint4(0, 0, 0, 0);
    }
    Turn t;
    if (turned) load_turn(t, a.cos_sin + pos * a.rot, a.rot, c8, a.style);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int h = h0 + k * kH;
      const uint4 far = shfl4(raw[k], partner);
      uint4 res = raw[k];
      if (turned) {
        float x[8], o[8];
        dev::bf16x8_to_float(raw[k], x);
        dev::bf16x8_to_float(far, o);
        turn8(x, o, t, a.rot, c8, a.style);
        res = pack8(x);
      }
      if (h < a.heads) *reinterpret_cast<uint4*>(a.q_out + (tok * a.heads + h) * D + c8 * 8) = res;
    }
    return;
  }
  const int blocks = 2 * a.kv_heads;
  const int blk = static_cast<int>(blockIdx.x % blocks);       // K heads, then V heads
  const bool is_k = blk < a.kv_heads;
  const int h = is_k ? blk : blk - a.kv_heads;
  const Place p = find_place(a, blockIdx.x / blocks);
  if (p.page < 0) return;                                      // the whole CTA
  const uint16_t* src = (is_k ? a.k + p.tok * a.k_stride : a.v + p.tok * a.v_stride) + h * D + c8 * 8;
  const int64_t stride = is_k ? a.k_stride : a.v_stride;
  const bool rotate = is_k && a.rot > 0;
  uint4 raw[kPasses];
  bool mine[kPasses];
  int64_t pos[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int o = k * kTok + threadIdx.x / kLanes;
    mine[k] = o >= p.first && o < p.last;
    raw[k] = mine[k] ? *reinterpret_cast<const uint4*>(src + (o - p.first) * stride) : make_uint4(0, 0, 0, 0);
    pos[k] = 0;
    if (a.rot > 0 && mine[k]) {
      pos[k] = a.positions ? a.positions[p.tok + o - p.first] : p.pos + o - p.first;
      mine[k] = pos[k] >= 0 && pos[k] < a.max_pos;
    }
  }
  float x[kPasses][8];
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    dev::bf16x8_to_float(raw[k], x[k]);
    if (rotate) {
      const uint4 far = shfl4(raw[k], partner);
      if (turned && mine[k]) {
        float o[8];
        Turn t;
        dev::bf16x8_to_float(far, o);
        load_turn(t, a.cos_sin + pos[k] * a.rot, a.rot, c8, a.style);
        turn8(x[k], o, t, a.rot, c8, a.style);
      }
    }
    if (mine[k]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = fabsf(x[k][i]);
        if (m <= 3.402823466e38f) amax = fmaxf(amax, m);       // finite: not NaN, not inf
      }
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  __shared__ float part[kHeadThreads / 32];
  if (lane == 0) part[threadIdx.x / 32] = amax;
  const int64_t block = p.page * blocks + blk;
  const float old = a.kv_scale[block];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHeadThreads / 32; ++i) amax = fmaxf(amax, part[i]);
  const float need = __fdiv_rn(amax, E4M3 ? 448.0f : 127.0f);
  float scale = old, shrink = 1.0f;
  if (p.first == 0 || !(old > 0.0f)) {
    scale = need;
  } else {
    while (scale < need) {             // doubling is exact; ends at the latest when scale is infinite
      scale *= 2.0f;
      shrink *= 0.5f;
    }
  }
  uint8_t* dst = a.kv + block * (kPage * D);
  if (shrink != 1.0f) {
    // older codes, 4 at a time
    uint32_t* w = reinterpret_cast<uint32_t*>(dst);
    for (int i = threadIdx.x; i < p.first * D / 4; i += kHeadThreads) {
      const uint32_t c = w[i];
      uint32_t n = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) n |= encode8<E4M3>(__fmul_rn(decode8<E4M3>(c >> (8 * b)), shrink)) << (8 * b);
      w[i] = n;
    }
  }
  if (threadIdx.x == 0 && scale != old) a.kv_scale[block] = scale;
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    if (!mine[k]) continue;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i / 4] |= encode8<E4M3>(scale == 0.0f ? x[k][i] : __fdiv_rn(x[k][i], scale)) << (8 * (i % 4));
    *reinterpret_cast<uint2*>(dst + (k * kTok + threadIdx.x / kLanes) * D + c8 * 8) = make_uint2(w[0], w[1]);
  }
}

template <int D>
cudaError_t launch_heads(const GqaAppendArgs& a, int64_t ctas, cudaStream_t s) {
  if (a.cache_dtype == QKVP_CACHE_E4M3) gqa_append_rope_kernel<D, true><<<static_cast<unsigned>(ctas), kHeadThreads, 0, s>>>(a);
  else gqa_append_rope_kernel<D, false><<<static_cast<unsigned>(ctas), kHeadThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mla_append_rope(const MlaAppendArgs& a, cudaStream_t s) {
  const int64_t jobs = a.n * (1 + (a.heads + kQHeads - 1) / kQHeads);
  const int64_t ctas = (jobs * 32 + kLatentThreads - 1) / kLatentThreads;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  mla_append_rope_kernel<<<static_cast<unsigned>(ctas), kLatentThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_gqa_append_rope(GqaAppendArgs a, cudaStream_t s) {
  const int64_t by_page = a.n / kPage + 2ll * a.batch;
  a.per_token = a.n <= by_page ? 1 : 0;
  const int64_t jobs = std::min(a.n, by_page);
  const int64_t kv_ctas = jobs * 2 * a.kv_heads;
  const int heads_per_warp = 4 * 32 / (a.dim / 8);
  const int64_t q_jobs = a.heads > 0 ? a.n * ((a.heads + heads_per_warp - 1) / heads_per_warp) : 0;
  const int64_t ctas = kv_ctas + (q_jobs * 32 + kHeadThreads - 1) / kHeadThreads;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  if (ctas == 0) return cudaSuccess;
  a.kv_ctas = static_cast<uint32_t>(kv_ctas);
  switch (a.dim) {
    case 64: return launch_heads<64>(a, ctas, s);
    case 128: return launch_heads<128>(a, ctas, s);
    default: return launch_heads<256>(a, ctas, s);
  }
}

}  // namespace qkvp
