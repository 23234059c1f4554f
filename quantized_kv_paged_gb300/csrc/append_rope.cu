// Appends that apply the rotary position embedding on the way into a quantized cache.
//
// Rotation of pair i at position p: (a, b) -> (a c - b s, b c + a s) with c = cos_sin[p][i] and
// s = cos_sin[p][r/2 + i]; the table is the caller's, so no angle is computed here and positions far out
// cost no precision. Every product and sum is one FP32 rounding (no contraction), which makes the codes
// reproducible bit for bit by any other implementation of the same formula.
//
// Both kernels are streams: BF16 in, 8-bit codes (and BF16 queries) out, each byte once, so memory bounds them
// where there are many tokens and a chain of dependent reads where there are few. A lane holds 8 dims of a
// head as two quads that rotate together: dims 4 l .. and r/2 + 4 l .. (HALVES), or 8 l .. and 8 l + 4 ..
// (PAIRS and what is not rotated). Either way it needs 4 cosines and 4 sines and nothing from another lane.
// Measured on GB300, kernel time: 20,011 latent rows with 16 query heads into the per-token pool 23.7 us (122
// MB, 5.1 TB/s; issue slots 48 %, the reads of position, table row and data in line), 4,096 rows with 128
// heads 24.4 us (142 MB, 5.8 TB/s), 44 rows with 128 heads 1.9 us; 12,086 tokens of 8 KV and 32 query heads of
// 128 in eight chunks 46 us (278 MB, 6.1 TB/s), 64 single tokens of the same heads 4.0 us.
#include <algorithm>
#include <cstdint>

#include "qkvp_device.cuh"
#include "qkvp_internal.h"

namespace qkvp {
namespace {

constexpr int kRope = kLatent - kDv;    // 64 rope dims of the latent
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float rot_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rot_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Where the two quads of lane l of a head start. `apart`: not next to one another.
struct Quads {
  int a, b;
  bool turned, apart;
  __device__ Quads(int l, int rot, int style) : turned(8 * l < rot), apart(turned && style == QKVP_ROPE_HALVES) {
    a = apart ? 4 * l : 8 * l;
    b = apart ? rot / 2 + 4 * l : 8 * l + 4;
  }
};

__device__ __forceinline__ uint4 load_quads(const uint16_t* head, const Quads& q) {
  if (!q.apart) return *reinterpret_cast<const uint4*>(head + q.a);
  const uint2 x = *reinterpret_cast<const uint2*>(head + q.a), y = *reinterpret_cast<const uint2*>(head + q.b);
  return make_uint4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ void store_quads(uint16_t* head, const Quads& q, uint4 v) {
  if (!q.apart) {
    *reinterpret_cast<uint4*>(head + q.a) = v;
  } else {
    *reinterpret_cast<uint2*>(head + q.a) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(head + q.b) = make_uint2(v.z, v.w);
  }
}
// The same two quads as codes, one byte each.
__device__ __forceinline__ void store_codes(uint8_t* head, const Quads& q, uint2 v) {
  if (!q.apart) {
    *reinterpret_cast<uint2*>(head + q.a) = v;
  } else {
    *reinterpret_cast<uint32_t*>(head + q.a) = v.x;
    *reinterpret_cast<uint32_t*>(head + q.b) = v.y;
  }
}

// Lane l's cosines and sines from the row of a position, and the rotation of its quads.
struct Turn {
  float4 c, s;
  __device__ void load(const float* row, int rot, int l) {
    c = *reinterpret_cast<const float4*>(row + 4 * l);
    s = *reinterpret_cast<const float4*>(row + rot / 2 + 4 * l);
  }
  __device__ void apply(float (&x)[8], int style) const {
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
    const bool halves = style == QKVP_ROPE_HALVES;       // pair i of the lane: (i, 4 + i), or (2 i, 2 i + 1)
    float ra[4], rb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = halves ? x[i] : x[2 * i], q = halves ? x[4 + i] : x[2 * i + 1];
      ra[i] = rot_a(p, q, cc[i], ss[i]);
      rb[i] = rot_b(p, q, cc[i], ss[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = halves ? ra[i] : i % 2 ? rb[i / 2] : ra[i / 2];
      x[4 + i] = halves ? rb[i] : i % 2 ? rb[2 + i / 2] : ra[2 + i / 2];
    }
  }
};

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(dev::pack_bf16x2(x[0], x[1]), dev::pack_bf16x2(x[2], x[3]), dev::pack_bf16x2(x[4], x[5]),
                    dev::pack_bf16x2(x[6], x[7]));
}

// ------------------------------------------------------------------------------------------------
// x / s for many x and one s, correctly rounded, without a division each: Markstein's correction of a
// quotient by fused multiply-adds (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990). r is 1 / s correctly rounded; q0 = x r is off by at most 2 steps, one
// correction brings it within one, and a correction from there rounds as the division does. The
// remainders are exact when nothing in them underflows: s in [2^-60, 2^60] and finite x, where a quotient
// that does not round to the code 0 comes from an x of 2^-72 and more. The signs are arranged so that -0
// stays -0. Equal to the division on 1.9e10 pairs on GB300, in five operations: with a division per element
// the chunked append of 12,086 tokens (8 KV heads, 32 query heads of 128) was issue-bound, 95 us.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ bool divides_fast(float s) { return s >= 0x1p-60f && s <= 0x1p60f; }
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q0 = __fmul_rn(x, r);
  const float q1 = __fmaf_rn(-__fmaf_rn(q0, s, -x), r, q0);
  return __fmaf_rn(-__fmaf_rn(q1, s, -x), r, q1);
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

// Four and eight FP32 -> E4M3 two at a time: nearest even, saturating, NaN to 0x7F and the sign of a zero kept, the
// same byte as encode_e4m3 for every one of the 2^32 inputs (compared on GB300).
__device__ __forceinline__ uint32_t encode_e4m3x4(const float* y) {
  return dev::f32x2_to_e4m3x2(y[0], y[1]) | dev::f32x2_to_e4m3x2(y[2], y[3]) << 16;
}
__device__ __forceinline__ uint2 encode_e4m3x8(const float (&x)[8]) { return make_uint2(encode_e4m3x4(x), encode_e4m3x4(x + 4)); }

// Codes of 8 values over the scale s: round(x / s), or round(x) where s is 0. fast: every x is finite and
// divides_fast(s), so |x / s| is at most 448 (127) up to its rounding, and the conversions below need no
// care for infinities (the corrected quotient of one is NaN). INT8: adding 1.5 * 2^23 leaves the nearest whole number, ties to even, in the
// low byte.
template <bool E4M3>
__device__ __forceinline__ uint2 encode_scaled(const float (&x)[8], float s, float r, bool fast) {
  uint32_t w[2] = {0, 0};
  if (fast) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = quotient(x[4 * i + k], s, r);
      if constexpr (E4M3) {
        w[i] = encode_e4m3x4(y);
      } else {
        uint32_t b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = __float_as_uint(__fadd_rn(y[k], 12582912.0f));
        w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4] |= encode8<E4M3>(s == 0.0f ? x[i] : __fdiv_rn(x[i], s)) << (8 * (i % 4));
  }
  return make_uint2(w[0], w[1]);
}

// ------------------------------------------------------------------------------------------------
// Latent rows. One warp per token, or per (token, 16 query heads): a decode step of 44 tokens and 128
// heads is 44 + 352 warps, enough to reach every SM. Everything that does not depend on the position is
// loaded before it is known.
// ------------------------------------------------------------------------------------------------
constexpr int kLatentThreads = 128;
constexpr int kQHeads = 16;             // query heads per warp
constexpr int kFusedTokens = 1024;
constexpr int kRopeLanes = kRope / 8;   // 8 lanes hold one head's 64 dims

// NVFP4 codes of 4 values (two bytes) under a block's E4M3 scale: the formulas of kv_append_quant.
__device__ __forceinline__ uint32_t nvfp4_scale(float amax, float g) { return dev::encode_e4m3(__fdiv_rn(amax, __fmul_rn(6.0f, g))); }
__device__ __forceinline__ uint32_t nvfp4_quad(const float* x, uint32_t s8, float g) {
  const float sd = __fmul_rn(dev::e4m3_to_float(s8), g);
  uint32_t w = 0;
  if (sd != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= dev::encode_e2m1(__fdiv_rn(x[i], sd)) << (4 * i);
  }
  return w;
}
__device__ __forceinline__ float amax4(const float* x) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = dev::max_nan(m, fabsf(x[i]));
  return m;
}

// The lane's two quads of the latent row, at dims qa and qb, as NVFP4. Next to one another they are half a block
// of 16 and lane ^ 1 holds the other half; apart each is a quarter of its block, with lanes ^ 1, ^ 2, ^ 3.
__device__ __forceinline__ void store_nvfp4(const MlaAppendArgs& a, int64_t slot, const float (&x)[8], int qa, int qb, bool apart, bool writes) {
  float ma = amax4(x), mb = amax4(x + 4);
  if (!apart) ma = mb = dev::max_nan(ma, mb);
  ma = dev::max_nan(ma, __shfl_xor_sync(kFull, ma, 1));
  mb = dev::max_nan(mb, __shfl_xor_sync(kFull, mb, 1));
  const float ma2 = dev::max_nan(ma, __shfl_xor_sync(kFull, ma, 2)), mb2 = dev::max_nan(mb, __shfl_xor_sync(kFull, mb, 2));
  if (!writes) return;
  const uint32_t sa = nvfp4_scale(apart ? ma2 : ma, a.g), sb = apart ? nvfp4_scale(mb2, a.g) : sa;
  uint8_t* row = a.kv + slot * kPacked;
  *reinterpret_cast<uint16_t*>(row + qa / 2) = static_cast<uint16_t>(nvfp4_quad(x, sa, a.g));
  *reinterpret_cast<uint16_t*>(row + qb / 2) = static_cast<uint16_t>(nvfp4_quad(x + 4, sb, a.g));
  if (qa % 16 == 0) a.kv_scale[slot * kScales + qa / 16] = static_cast<uint8_t>(sa);
  if (apart && qb % 16 == 0) a.kv_scale[slot * kScales + qb / 16] = static_cast<uint8_t>(sb);
}

// FUSED: the warp of a token takes the row and the token's first 16 query heads, with all loads in flight
// together and one look at the position and its table row: for many tokens (20,011 rows 23.7 us, 26.4 apart). Apart,
// a decode step of few tokens reaches twice as many SMs.
template <bool FUSED>
__global__ void __launch_bounds__(kLatentThreads) mla_append_rope_kernel(const MlaAppendArgs a) {
  dev::allow_dependents();
  dev::wait_for_previous();
  const int64_t job = (static_cast<int64_t>(blockIdx.x) * kLatentThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int head_jobs = (a.heads + kQHeads - 1) / kQHeads;
  if (job >= a.n * (FUSED ? head_jobs : 1 + head_jobs)) return;       // the whole warp
  const Quads quads(lane % kRopeLanes, kRope, a.style);
  const bool has_row = job < a.n, has_heads = FUSED || !has_row;
  // job n + i (FUSED: the jobs from n on, and the first n for their own token's first heads)
  const int more = FUSED ? head_jobs - 1 : head_jobs;
  const int64_t tok = has_row ? job : (job - a.n) / more;
  const int chunk = has_row ? 0 : static_cast<int>((job - a.n) % more) + (FUSED ? 1 : 0);
  const int h0 = chunk * kQHeads + lane / kRopeLanes;
  const int64_t pos = a.positions[tok], slot = has_row ? a.slots[tok] : 0;
  // query heads: four at a time, 8 lanes each
  uint4 raw[kQHeads / 4];
#pragma unroll
  for (int k = 0; k < kQHeads / 4; ++k)
    raw[k] = has_heads && h0 + 4 * k < a.heads ? load_quads(a.q_pe + tok * a.q_pe_tok + (h0 + 4 * k) * a.q_pe_head, quads)
                                               : make_uint4(0, 0, 0, 0);
  // the latent row: lane l holds dims 8 l .. and 256 + 8 l .. of c_kv, and lanes 0..7 the rope dims
  const bool rope = lane < kRopeLanes;
  uint4 raw0{}, raw1{}, raw2{};
  if (has_row) {
    raw0 = *reinterpret_cast<const uint4*>(a.c_kv + tok * a.c_kv_stride + 8 * lane);
    raw1 = *reinterpret_cast<const uint4*>(a.c_kv + tok * a.c_kv_stride + 256 + 8 * lane);
    if (rope) raw2 = load_quads(a.k_pe + tok * a.k_pe_stride, quads);
  }
  if (pos < 0 || pos >= a.max_pos) return;
  Turn t;
  t.load(a.cos_sin + pos * kRope, kRope, lane % kRopeLanes);
  if (has_heads) {
#pragma unroll
    for (int k = 0; k < kQHeads / 4; ++k) {
      if (h0 + 4 * k >= a.heads) continue;
      float y[8];
      dev::bf16x8_to_float(raw[k], y);
      t.apply(y, a.style);
      store_quads(a.q + (tok * a.heads + h0 + 4 * k) * kLatent + kDv, quads, pack8(y));
    }
  }
  if (!has_row || slot < 0 || slot >= a.num_slots) return;
  float x[3][8];
  dev::bf16x8_to_float(raw0, x[0]);
  dev::bf16x8_to_float(raw1, x[1]);
  dev::bf16x8_to_float(raw2, x[2]);
  if (rope) t.apply(x[2], a.style);
  if (a.kv_dtype == KV_NVFP4) {
    store_nvfp4(a, slot, x[0], 8 * lane, 8 * lane + 4, false, true);
    store_nvfp4(a, slot, x[1], 256 + 8 * lane, 256 + 8 * lane + 4, false, true);
    store_nvfp4(a, slot, x[2], kDv + quads.a, kDv + quads.b, quads.apart, rope);
    return;
  }
  if (a.kv_dtype == KV_FP8) {
    uint8_t* row = a.kv + slot * kLatent;
    *reinterpret_cast<uint2*>(row + 8 * lane) = encode_e4m3x8(x[0]);
    *reinterpret_cast<uint2*>(row + 256 + 8 * lane) = encode_e4m3x8(x[1]);
    if (rope) store_codes(row + kDv, quads, encode_e4m3x8(x[2]));
    return;
  }
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = dev::max_nan(amax, fabsf(x[k][i]));
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) amax = dev::max_nan(amax, __shfl_xor_sync(kFull, amax, o));
  uint8_t* page = a.kv + (slot / kPage) * kPtPageBytes;
  uint8_t* row = page + (slot % kPage) * kLatent;
  // a token holding a NaN gets the scale 0x7FC00000 (one fixed NaN pattern for the stored bytes)
  const float sc = amax != amax ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 448.0f);
  const bool fast = divides_fast(sc) && amax <= 3.402823466e38f;
  const float inv = __frcp_rn(sc);
  if (lane == 0) *reinterpret_cast<float*>(page + kPtScaleOff + (slot % kPage) * 4) = sc;
  *reinterpret_cast<uint2*>(row + 8 * lane) = encode_scaled<true>(x[0], sc, inv, fast);
  *reinterpret_cast<uint2*>(row + 256 + 8 * lane) = encode_scaled<true>(x[1], sc, inv, fast);
  if (rope) store_codes(row + kDv, quads, encode_scaled<true>(x[2], sc, inv, fast));
}

// ------------------------------------------------------------------------------------------------
// K and V heads. A CTA has one page that the call writes, of K or of V, and walks some of its heads: the
// block's scale needs the amax of all the page's new tokens, and its older codes change with it, so a
// block has one owner and no atomics. The new elements stay in registers between the amax and the codes.
// To find the page takes four dependent reads (request, its length, page table, page id), some 4 us cold:
// a CTA of many heads pays that once and loads each head's elements while it works on the one before.
//
// Which pages are written is known on the device only. The launch has, for request r, floor(n_r / 64) + 2
// candidates, the most pages that n_r tokens can touch: job c belongs to the last request with
// tok_indptr[r] / 64 + 2 r <= c. With few tokens there is a job per token instead, and the first token of
// each page does the work, in smaller CTAs of one head that keep the first few tokens only (the others are
// read again for their codes): 128 single tokens of 8 KV heads took 11 us at the 205 registers that 64 tokens ask
// for. Idle jobs leave after the search.
// ------------------------------------------------------------------------------------------------

// 8 passes of query heads to a warp: eight chunks (above) 46 us; 4 passes 54, 2 passes 67, 16 passes 58 (too few warps).
constexpr int kQueryPasses = 8;
// CTAs that the heads of the pages are shared out to, two per SM: eight chunks 46 us, 100 requests of 3 to 300 tokens
// (8 KV heads of 64) 17.5; with 512 CTAs 48 and 19.4, with 1,024 50 and 23.7, with one head each 58 and 33.
constexpr int kFillCtas = 300;

// The largest r in [0, batch) with f(r) <= c for a non-decreasing f with f(0) <= c (0 if there is none):
// 256 probes at a time, one round of loads for up to 256 requests.
template <class F>
__device__ __forceinline__ int last_at_most(int batch, int64_t c, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n + 255) / 256;
    int hits = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int off = (lane + 32 * j) * step;
      if (32 * j * step < n) hits += __popc(__ballot_sync(kFull, off < n && f(lo + off) <= c));
    }
    const int k = max(hits - 1, 0) * step;
    lo += k;
    n = min(step, n - k);
  }
  return lo;
}

// The new tokens of one page: offsets [first, last) of it, from source row tok, cache position pos on.
// entry: of the page table, -1: nothing to do.
struct Place {
  int64_t entry, tok, pos;
  int first, last;
};

// The token range of request r, cut to the rows that there are.
__device__ __forceinline__ void request_tokens(const GqaAppendArgs& a, int r, int64_t& t0, int64_t& t1) {
  t0 = min(max(static_cast<int64_t>(a.tok_indptr[r]), int64_t(0)), a.n);
  t1 = min(max(static_cast<int64_t>(a.tok_indptr[r + 1]), t0), a.n);
}

template <bool PER_TOKEN>
__device__ __forceinline__ Place find_place(const GqaAppendArgs& a, int64_t job) {
  Place p{-1, 0, 0, 0, 0};
  const int32_t* tp = a.tok_indptr;
  const int r = PER_TOKEN ? last_at_most(a.batch, job, [tp](int i) { return static_cast<int64_t>(tp[i]); })
                          : last_at_most(a.batch, job, [tp](int i) { return static_cast<int64_t>(tp[i] / kPage) + 2ll * i; });
  int64_t t0, t1;
  request_tokens(a, r, t0, t1);
  const int64_t held = a.kv_len[r];
  const int64_t p0 = a.kv_indptr[r], p1 = a.kv_indptr[r + 1];
  if (held < 0 || t0 >= t1) return p;
  int64_t local;                         // page of the request
  if (PER_TOKEN) {
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
  p.entry = e;
  p.tok = t0 + lo - held;
  p.pos = lo;
  p.first = static_cast<int>(lo - local * kPage);
  p.last = static_cast<int>(hi - local * kPage);
  return p;
}

// A warp's query heads: some passes over 32 / (D / 8) heads of one token.
template <int D>
__device__ __forceinline__ void rotate_queries(const GqaAppendArgs& a, int64_t job) {
  constexpr int kLanes = D / 8, kH = 32 / kLanes, kPasses = kQueryPasses;
  const int lane = threadIdx.x & 31;
  const int head_jobs = (a.heads + kPasses * kH - 1) / (kPasses * kH);
  if (job >= a.n * head_jobs) return;
  const int64_t tok = job / head_jobs;
  const int h0 = static_cast<int>(job % head_jobs) * kPasses * kH + lane / kLanes;
  const Quads quads(lane % kLanes, a.rot, a.style);
  uint4 raw[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k)
    raw[k] = h0 + k * kH < a.heads ? load_quads(a.q + tok * a.q_stride + (h0 + k * kH) * D, quads) : make_uint4(0, 0, 0, 0);
  const int32_t* tp = a.tok_indptr;
  const int r = last_at_most(a.batch, tok, [tp](int i) { return static_cast<int64_t>(tp[i]); });
  int64_t t0, t1;
  request_tokens(a, r, t0, t1);
  const int64_t pos = a.positions ? a.positions[tok] : a.kv_len[r] + tok - t0;
  if (tok < t0 || tok >= t1) return;             // padding
  if (a.rot > 0 && (pos < 0 || pos >= a.max_pos)) return;
  Turn t;
  if (quads.turned) t.load(a.cos_sin + pos * a.rot, a.rot, lane % kLanes);
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    if (h0 + k * kH >= a.heads) continue;
    uint4 res = raw[k];
    if (quads.turned) {
      float x[8];
      dev::bf16x8_to_float(raw[k], x);
      t.apply(x, a.style);
      res = pack8(x);
    }
    store_quads(a.q_out + (tok * a.heads + h0 + k * kH) * D, quads, res);
  }
}

template <int D, bool E4M3, bool PER_TOKEN, int THREADS>
__global__ void __launch_bounds__(THREADS) gqa_append_rope_kernel(const GqaAppendArgs a) {
  constexpr int kLanes = D / 8;                    // lanes of one token's head
  constexpr int kTok = THREADS / kLanes;           // tokens of one pass over the CTA
  constexpr int kPasses = kPage / kTok;
  constexpr int kHold = PER_TOKEN ? 1 : kPasses;   // passes whose elements stay in registers
  dev::allow_dependents();
  dev::wait_for_previous();
  if (blockIdx.x >= a.kv_ctas) {
    rotate_queries<D>(a, ((static_cast<int64_t>(blockIdx.x) - a.kv_ctas) * THREADS + threadIdx.x) >> 5);
    return;
  }
  const int lane = threadIdx.x & 31, l = threadIdx.x % kLanes, mine0 = threadIdx.x / kLanes;
  const int parts = 2 * a.head_parts;              // of a page: K's heads in head_parts parts, then V's
  const int part = static_cast<int>(blockIdx.x % parts);
  const bool is_k = part < a.head_parts;
  const int per_part = (a.kv_heads + a.head_parts - 1) / a.head_parts;
  const int h0 = (is_k ? part : part - a.head_parts) * per_part, h1 = min(h0 + per_part, a.kv_heads);
  const Place p = find_place<PER_TOKEN>(a, blockIdx.x / parts);
  if (p.entry < 0 || h0 >= h1) return;                         // the whole CTA
  const int64_t page = a.kv_indices[p.entry];
  const int count = p.last - p.first;
  const Quads quads(l, is_k ? a.rot : 0, a.style);
  const int64_t stride = is_k ? a.k_stride : a.v_stride;
  const uint16_t* src = (is_k ? a.k : a.v) + p.tok * stride;
  // the page's i-th new token: its elements of head h as stored, and its position (-1: skipped, or none)
  auto stored = [&](int i, int h) { return i < count ? load_quads(src + i * stride + h * D, quads) : make_uint4(0, 0, 0, 0); };
  auto position = [&](int i) -> int64_t {
    if (i >= count) return -1;
    if (a.rot == 0) return 0;
    const int64_t at = a.positions ? a.positions[p.tok + i] : p.pos + i;
    return at < a.max_pos ? max(at, int64_t(-1)) : -1;
  };
  auto turned = [&](float (&x)[8], uint4 raw, int64_t at) {
    dev::bf16x8_to_float(raw, x);
    if (quads.turned && at >= 0) {
      Turn t;
      t.load(a.cos_sin + at * a.rot, a.rot, l);
      t.apply(x, a.style);
    }
  };
  uint4 raw[kHold];
  int at[kHold];
#pragma unroll
  for (int k = 0; k < kHold; ++k) raw[k] = stored(k * kTok + mine0, h0);
#pragma unroll
  for (int k = 0; k < kHold; ++k) at[k] = static_cast<int>(position(k * kTok + mine0));
  if (page < 0 || page >= a.num_pages) return;
  const int64_t block0 = page * 2 * a.kv_heads + (is_k ? 0 : a.kv_heads);
  float old = a.kv_scale[block0 + h0];
  __shared__ float shared_max[3][THREADS / 32];
  auto over_cta = [&](float v, int buf) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = dev::max_nan(v, __shfl_xor_sync(kFull, v, o));
    if (lane == 0) shared_max[buf][threadIdx.x / 32] = v;
    __syncthreads();
    v = shared_max[buf][0];
#pragma unroll
    for (int i = 1; i < THREADS / 32; ++i) v = dev::max_nan(v, shared_max[buf][i]);
    return v;
  };
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    float x[kHold][8];
#pragma unroll
    for (int k = 0; k < kHold; ++k) turned(x[k], raw[k], at[k]);
    float next_old = 0.0f;
    if (h + 1 < h1) {
#pragma unroll
      for (int k = 0; k < kHold; ++k) raw[k] = stored(k * kTok + mine0, h + 1);
      next_old = a.kv_scale[block0 + h + 1];
    }
    // calls f(x, offset of the page) for every new token that is not skipped
    auto each = [&](auto f) {
#pragma unroll
      for (int k = 0; k < kHold; ++k)
        if (at[k] >= 0) f(x[k], k * kTok + mine0);
      if constexpr (kHold < kPasses) {
#pragma unroll 1
        for (int i = kTok + mine0; i < count; i += kTok) {
          const int64_t pos = position(i);
          if (pos < 0) continue;
          float y[8];
          turned(y, stored(i, h), pos);
          f(y, i);
        }
      }
    };
    float amax = 0.0f;
    each([&](const float (&v)[8], int) {
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = dev::max_nan(amax, fabsf(v[i]));
    });
    amax = over_cta(amax, (h - h0) & 1);
    const bool finite = amax <= 3.402823466e38f;
    if (!finite) {
      // a NaN or an infinity among the new elements: the largest of the others
      amax = 0.0f;
      each([&](const float (&v)[8], int) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (fabsf(v[i]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(v[i]));
      });
      amax = over_cta(amax, 2);
    }
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
    const int64_t block = block0 + h;
    uint8_t* dst = a.kv + block * (kPage * D);
    if (shrink != 1.0f) {
      // older codes, 4 at a time
      uint32_t* w = reinterpret_cast<uint32_t*>(dst);
      for (int i = threadIdx.x; i < p.first * D / 4; i += THREADS) {
        const uint32_t c = w[i];
        uint32_t n = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) n |= encode8<E4M3>(__fmul_rn(decode8<E4M3>(c >> (8 * b)), shrink)) << (8 * b);
        w[i] = n;
      }
    }
    if (threadIdx.x == 0 && scale != old) a.kv_scale[block] = scale;
    const bool fast = finite && divides_fast(scale);
    const float inv = __frcp_rn(scale);
    each([&](const float (&v)[8], int i) { store_codes(dst + (p.first + i) * D, quads, encode_scaled<E4M3>(v, scale, inv, fast)); });
    old = next_old;
  }
}

template <int D, bool E4M3>
cudaError_t launch_heads(GqaAppendArgs a, cudaStream_t s) {
  constexpr int kPageThreads = 256, kTokenThreads = D == 256 ? 128 : 64;
  const int64_t by_page = a.n / kPage + 2ll * a.batch;
  // a job per token up to 4 tokens a request: 33 requests of 1 to 5 tokens 3.2 us, as pages 4.6
  const bool per_token = a.n <= std::max<int64_t>(by_page, 4ll * a.batch);
  const int threads = per_token ? kTokenThreads : kPageThreads;
  const int64_t jobs = per_token ? a.n : by_page;
  // heads to a CTA: as many as leave kFillCtas CTAs that have work
  const int64_t busy = per_token ? a.n : a.n / kPage + a.batch;
  int64_t per_cta = per_token ? 1 : std::max<int64_t>(1, std::min<int64_t>(a.kv_heads, busy * 2 * a.kv_heads / kFillCtas));
  a.head_parts = static_cast<int>((a.kv_heads + per_cta - 1) / per_cta);
  const int64_t kv_ctas = jobs * 2 * a.head_parts;
  constexpr int kHeadsPerWarp = kQueryPasses * 32 / (D / 8);
  const int64_t q_jobs = a.heads > 0 ? a.n * ((a.heads + kHeadsPerWarp - 1) / kHeadsPerWarp) : 0;
  const int64_t ctas = kv_ctas + (q_jobs * 32 + threads - 1) / threads;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  a.kv_ctas = static_cast<uint32_t>(kv_ctas);
  auto kernel = per_token ? gqa_append_rope_kernel<D, E4M3, true, kTokenThreads> : gqa_append_rope_kernel<D, E4M3, false, kPageThreads>;
  return launch_overlapped(kernel, static_cast<unsigned>(ctas), threads, 0, s, a);
}

}  // namespace

cudaError_t launch_mla_append_rope(const MlaAppendArgs& a, cudaStream_t s) {
  const int head_jobs = (a.heads + kQHeads - 1) / kQHeads;
  const bool fused = a.n >= kFusedTokens && head_jobs > 0;
  const int64_t jobs = a.n * (fused ? head_jobs : 1 + head_jobs);
  const int64_t ctas = (jobs * 32 + kLatentThreads - 1) / kLatentThreads;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return launch_overlapped(fused ? mla_append_rope_kernel<true> : mla_append_rope_kernel<false>, static_cast<unsigned>(ctas), kLatentThreads, 0, s, a);
}

cudaError_t launch_gqa_append_rope(const GqaAppendArgs& a, cudaStream_t s) {
  const bool e4m3 = a.cache_dtype == QKVP_CACHE_E4M3;
  switch (a.dim) {
    case 64: return e4m3 ? launch_heads<64, true>(a, s) : launch_heads<64, false>(a, s);
    case 128: return e4m3 ? launch_heads<128, true>(a, s) : launch_heads<128, false>(a, s);
    default: return e4m3 ? launch_heads<256, true>(a, s) : launch_heads<256, false>(a, s);
  }
}

}  // namespace qkvp
