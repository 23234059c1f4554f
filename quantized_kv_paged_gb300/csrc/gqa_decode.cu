// Decode attention over a paged 8-bit cache of K and V heads, one scale per (page, K or V, head).
//
// Per query head with its KV head's codes kc, vc and block scales sk, sv, over the visible tokens t:
//   z_t = sm_scale * sk (q . kc_t),  out = sum_t softmax(z)_t sv vc_t,  lse = log sum_t exp z_t.
// Reading the pages once is the floor (2 G operations per byte, G query heads per KV head: far below the
// tensor rate), so the kernel is a stream with the arithmetic kept out of its way.
//
// Work. A CTA of four warps walks the segments of its worker; each warp takes every fourth unit of 4 KB of
// K and 4 KB of V (64 / 32 / 16 tokens at D = 64 / 128 / 256) and runs a pipeline of its own: a ring of
// units that its lane 0 fills by TMA, one mbarrier per unit, no barrier with other warps until the segment
// ends. Two CTAs per SM keep up to 192 KB of loads in flight, several times what the latency asks for. The
// four warps join their sums at a segment's end; a group (request, KV head) cut into segments leaves
// normalised FP32 partials, joined by the last of its CTAs to arrive, in segment order.
//
// Products. Heads are the columns (N = 8) of both products, so that G <= 8 wastes no rows:
//   S^T [tokens x heads] = K Q^T,  O^T [dims x heads] += V^T P^T,  mma m16n8k16, FP16 in, FP32 sums.
// E4M3 codes and INT8 codes are exact in FP16, Q is exact after a power of two per head. Both operands from
// the cache come straight from the bytes: which 16 dims make up a k-step, and which dim is which row of
// O^T, is free as long as Q and the output agree, so a lane takes 16 bytes of one token at a time and no
// byte moves between lanes. V^T needs two tokens of one dim in a register: two byte permutes of two
// tokens' words, then the conversion. The tokens of an 8-token block are taken in the order `tok8`, which
// makes every 16-byte (D = 64: 8-byte) shared-memory read free of bank conflicts under the TMA's 128-byte
// swizzle. P^T is S^T's accumulator layout transposed: one 8x8 transpose per 8 tokens.
//
// Softmax. One running reference m per head. It moves only when a logit passes it by 2^8 (a vote instead
// of a reduction per unit); P = 2^(z - m + 6) <= 2^14 is in FP16's normal range down to 2^-28 of the
// largest weight. l is summed from the unrounded FP32 values. The V scale sv = f 2^k of a page multiplies
// P: f (in [1, 2)) on the value, k in the exponent, less the first page's k; l takes 2^-k back. So pages
// with scales far apart keep their precision, whichever comes first.
#include <atomic>
#include <cstdint>
#include <cstring>

#include <cuda.h>

#include "decode_common.cuh"
#include "qkvp_device.cuh"
#include "qkvp_internal.h"

namespace qkvp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kH = kGqaPassHeads;
constexpr int kHalf = 4096;              // bytes of K (and of V) in a unit
constexpr int kUnit = 2 * kHalf;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kSlack = 8.0f;           // how far (log2) a logit may pass the reference
constexpr float kLift = 6.0f;            // P is held as 2^(z - m + kLift)
constexpr float kNone = -3e38f;          // reference before the first unit

template <int D, int NT>
struct Shape {
  static constexpr int kTokens = kHalf / D;            // tokens of a unit
  static constexpr int kUnits = kPage / kTokens;       // units of a page
  static constexpr int kStages = D == 256 && NT == 2 ? 2 : 3;
  static constexpr int kTiles = D / 16;                // 16-dim row tiles of O^T
  static constexpr int kPart = kTiles * NT * 32 * 16;  // bytes of one warp's O^T
  // shared memory: rings, the join's buffer, the units' scales, barriers, per-warp lse, flags
  static constexpr int kJoin = kWarps * kStages * kUnit;
  static constexpr int kScale = kJoin + 2 * kPart;
  static constexpr int kBars = kScale + kWarps * kStages * 8;
  static constexpr int kLse = kBars + kWarps * kStages * 8;
  static constexpr int kFlags = kLse + kWarps * kH * 4;
  static constexpr int kBytes = kFlags + 16;
};

// The token of an 8-token block that row n of its tile holds.
template <int D>
__device__ __forceinline__ int tok8(int n) {
  const int t = n >> 1, odd = n & 1;
  if constexpr (D == 64) return ((t & 1) + ((t >> 1) << 2)) ^ (odd ? 3 : 0);
  if constexpr (D == 128) return odd ? (2 * t + 5) & 7 : 2 * t;
  return odd ? 4 + (t ^ 2) : t;
}

__device__ __forceinline__ int page_of(const GqaSegment& s, int v) {
  return v < s.sink_pages ? v : s.win_page + (v - s.sink_pages);
}

// Where the visible tokens of a unit lie: token i of it is visible if i < lim and (i >= win or i < sink).
struct Range {
  int lim, win, sink;
  __device__ Range(const GqaSegment& s, int t0) : lim(s.len - t0), win(s.win_begin - t0), sink(s.sink_end - t0) {}
  __device__ bool sees(int i) const { return i < lim && (i >= win || i < sink); }
  __device__ bool any(int n) const { return lim > 0 && (sink > 0 || win < min(lim, n)); }
  __device__ bool all(int n) const { return lim >= n && (win <= 0 || sink >= n); }
};

__device__ __forceinline__ GqaSegment load_segment(const GqaSegment* p) {
  GqaSegment s;
  const int4* src = reinterpret_cast<const int4*>(p);
  int4* dst = reinterpret_cast<int4*>(&s);
#pragma unroll
  for (int i = 0; i < 4; ++i) dst[i] = __ldg(src + i);
  return s;
}

// Walks the units that one warp will take, ahead of their use; the page id of the unit it stands on is
// loaded when it gets there, one unit before it is needed.
template <int U>
struct Feed {
  const GqaDecodeArgs& a;
  int si, se, u, t0, sub;
  int32_t page;
  GqaSegment s;
  __device__ Feed(const GqaDecodeArgs& args, int s0, int s1, int warp) : a(args), si(s0), se(s1), u(warp - kWarps), t0(0), sub(0), page(-1) {
    if (si < se) s = load_segment(a.segs + si);
    next(warp);
  }
  __device__ void next(int warp) {
    if (si >= se) return;
    u += kWarps;
    while (u >= s.num_pages * U) {
      if (++si >= se) return;
      s = load_segment(a.segs + si);
      u = warp;
    }
    const int local = page_of(s, s.page_begin + u / U);
    sub = u % U;
    page = __ldg(a.kv_indices + s.page0 + local);
    t0 = local * kPage + sub * (kPage / U);
  }
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, int x, int y, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
  const uint2 v = lds64(addr);
  return make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The four codes of a word -> FP16 pairs (bytes 0, 1) and (bytes 2, 3), exact. INT8: the biased byte
// under the exponent of 1024 is 1024 + 128 + c; the subtraction is exact.
template <bool E4M3>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  } else {
    const uint32_t b = w ^ 0x80808080u;
    const uint32_t l = __byte_perm(b, 0x64646464u, 0x4140), h = __byte_perm(b, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(l), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(h), "r"(0x64806480u));
  }
}

// O^T and softmax state of one warp; column e of tile nt is head 8 nt + 2 (lane % 4) + e.
template <int D, int NT>
struct State {
  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2];
  __device__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][n][k] = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = kNone;
        l[n][e] = 0.0f;
      }
  }
};

// Q^T as the B operand of K Q^T: [64-dim group][k-step][register][head tile].
template <int D, int NT>
struct Query {
  uint32_t q[D / 64][4][2][NT];
  float scale[NT][2];       // logit factor of the lane's columns: sm_scale log2(e) / (the head's power of two)
};

template <int D, int NT>
__device__ __forceinline__ void load_query(Query<D, NT>& Q, const GqaDecodeArgs& a, const GqaSegment& s, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = 8 * n + g;
    uint4 raw[D / 64][2];
    const uint16_t* row = a.q + (static_cast<int64_t>(s.req) * a.heads + s.head0 + h) * D + 16 * t;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        raw[c][k] = h < s.heads ? __ldg(reinterpret_cast<const uint4*>(row + 64 * c + 8 * k)) : make_uint4(0, 0, 0, 0);
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x[8];
        dev::bf16x8_to_float(raw[c][k], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
      }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    // 2^e that brings the largest |q| to [2^14, 2^15), where FP16 holds 8 bits down to 2^-29 of it
    const int ex = static_cast<int>(__float_as_uint(amax) >> 23);
    const int e = amax == 0.0f ? 0 : min(126, 14 + 127 - ex);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23), down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t w[4] = {raw[c][k].x, raw[c][k].y, raw[c][k].z, raw[c][k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) Q.q[c][2 * k + i / 2][i % 2][n] = dev::bf16x2_to_f16x2(w[i], up);
      }
    const float f = a.scale_log2 * down;
#pragma unroll
    for (int e2 = 0; e2 < 2; ++e2) Q.scale[n][e2] = __shfl_sync(kFull, f, 4 * (2 * t + e2));
  }
}

// One unit: S^T, the running softmax, O^T. PARTIAL: some of its tokens are not visible.
template <int D, bool E4M3, int NT, bool PARTIAL>
__device__ __forceinline__ void take_unit(State<D, NT>& st, const Query<D, NT>& Q, uint32_t kbase, uint32_t scale_addr,
                                          const Range& range, int& kref, int lane) {
  constexpr int MT = kHalf / D / 16;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t vbase = kbase + kHalf;
  const float2 sc = lds_f2(scale_addr);
  float s[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[m][n][k] = 0.0f;
  const int tg = tok8<D>(g);
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const uint32_t off = tg * D + c * 64 + t * 16;
    const uint32_t at = kbase + (off ^ (((off >> 7) & 7) << 4));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      // at D = 64 the odd 8-token block of a tile is 4 rows of 128 bytes further: its swizzle differs in bit 6
      const uint4 x = lds128(at + 16 * m * D);
      const uint4 y = lds128((D == 64 ? at ^ 64 : at) + (16 * m + 8) * D);
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a0, a1, a2, a3;
        codes_to_f16<E4M3>(xw[j], a0, a2);
        codes_to_f16<E4M3>(yw[j], a1, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n) dev::mma_f16(s[m][n], a0, a1, a2, a3, Q.q[c][j][0][n], Q.q[c][j][1][n]);
      }
    }
  }

  // V's scale f 2^k, k relative to the warp's first page of the segment
  const uint32_t vs = __float_as_uint(sc.y);
  const bool zero = sc.y == 0.0f;
  const int vk = min(max(static_cast<int>((vs >> 23) & 0xFF), 1) - 127, 126);
  if (kref == INT32_MIN && !zero) kref = vk;
  const int k = zero ? 0 : max(-90, min(90, vk - kref));       // the bound keeps l finite
  const float f = zero ? 0.0f : sc.y * __uint_as_float(static_cast<uint32_t>(127 - vk) << 23);
  const float back = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);

  float top[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float f0 = Q.scale[n][0] * sc.x, f1 = Q.scale[n][1] * sc.x;
    top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool off = PARTIAL && !range.sees(16 * m + 8 * r + tg);
        float& z0 = s[m][n][2 * r];
        float& z1 = s[m][n][2 * r + 1];
        z0 = off ? -INFINITY : z0 * f0;
        z1 = off ? -INFINITY : z1 * f1;
        top[n][0] = fmaxf(top[n][0], z0);
        top[n][1] = fmaxf(top[n][1], z1);
      }
    }
  }
  bool move = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) move |= top[n][e] + k > st.m[n][e] + kSlack;
  if (__any_sync(kFull, move)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float c[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = top[n][e] + k;
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
        x = fmaxf(fminf(x, 3e38f), st.m[n][e]);
        c[e] = dev::fast_exp2(st.m[n][e] - x);
        st.m[n][e] = x;
        st.l[n][e] *= c[e];
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        st.o[i][n][0] *= c[0];
        st.o[i][n][1] *= c[1];
        st.o[i][n][2] *= c[0];
        st.o[i][n][3] *= c[1];
      }
    }
  }
  uint32_t p[MT][NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float sum[2] = {0.0f, 0.0f};
    const float b0 = static_cast<float>(k) - st.m[n][0] + kLift, b1 = static_cast<float>(k) - st.m[n][1] + kLift;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = dev::fast_exp2(s[m][n][2 * r] + b0), p1 = dev::fast_exp2(s[m][n][2 * r + 1] + b1);
        sum[0] += p0;
        sum[1] += p1;
        p[m][n][r] = transpose8(dev::pack_f16x2(p0 * f, p1 * f));
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) st.l[n][e] += sum[e] * back;
  }

  const int ta = tok8<D>(2 * t), tb = tok8<D>(2 * t + 1);
#pragma unroll
  for (int h = 0; h < (D + 127) / 128; ++h) {
    const int width = D == 64 ? 8 : 16;                // bytes of a lane's piece of a token
    const uint32_t oa = ta * D + h * 128 + g * width, ob = tb * D + h * 128 + g * width;
    const uint32_t va = vbase + (oa ^ (((oa >> 7) & 7) << 4)), vb = vbase + (ob ^ (((ob >> 7) & 7) << 4));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      constexpr int W = D == 64 ? 2 : 4;
      uint32_t w[4][W];                                // tokens ta, tb, ta + 8, tb + 8 of the tile
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint32_t at = r & 1 ? vb : va;
        if (D == 64 && r >= 2) at ^= 64;
        at += (16 * m + (r >= 2 ? 8 : 0)) * D;
        if constexpr (D == 64) {
          const uint2 v = lds64(at);
          w[r][0] = v.x;
          w[r][1] = v.y;
        } else {
          const uint4 v = lds128(at);
          w[r][0] = v.x;
          w[r][1] = v.y;
          w[r][2] = v.z;
          w[r][3] = v.w;
        }
        // what stands behind a token that is not visible may be NaN, and 0 * NaN is not 0
        if (PARTIAL && !range.sees(16 * m + (r >= 2 ? 8 : 0) + (r & 1 ? tb : ta))) {
#pragma unroll
          for (int i = 0; i < W; ++i) w[r][i] = 0;
        }
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {                  // dims 4 i + 2 q (row g) and 4 i + 2 q + 1 (row g + 8)
          uint32_t a0, a1, a2, a3;
          codes_to_f16<E4M3>(__byte_perm(w[0][i], w[1][i], q ? 0x7362 : 0x5140), a0, a1);
          codes_to_f16<E4M3>(__byte_perm(w[2][i], w[3][i], q ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) dev::mma_f16(st.o[8 * h + 2 * i + q][n], a0, a1, a2, a3, p[m][n][0], p[m][n][1]);
        }
      }
    }
  }
}

// Sums the O^T of the four warps into warp 0's, in a fixed order, through two warps' worth of buffer.
template <int D, int NT>
__device__ __forceinline__ void sum_warps(float (&o)[D / 16][NT][4], float4* buf, int warp, int lane) {
  constexpr int kVec = D / 16 * NT * 32;
#pragma unroll
  for (int step = kWarps / 2; step >= 1; step /= 2) {
    if (warp >= step && warp < 2 * step) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          buf[(warp - step) * kVec + (i * NT + n) * 32 + lane] = make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
    }
    __syncthreads();
    if (warp < step) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 v = buf[warp * kVec + (i * NT + n) * 32 + lane];
          o[i][n][0] += v.x;
          o[i][n][1] += v.y;
          o[i][n][2] += v.z;
          o[i][n][3] += v.w;
        }
    }
    if (step > 1) __syncthreads();
  }
}

// Warp 0's finished O^T (normalised) and base-2 lse of a segment's heads to out and lse.
template <int D, int NT>
__device__ __forceinline__ void write_out(const GqaDecodeArgs& a, const GqaSegment& s, const float (&o)[D / 16][NT][4],
                                          const float (&L)[NT][2], int lane) {
  const int g = lane >> 2, t = lane & 3;
  const int64_t row0 = static_cast<int64_t>(s.req) * a.heads + s.head0;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = 8 * n + 2 * t + e;
      if (h >= s.heads) continue;
      uint16_t* dst = a.out + (row0 + h) * D;
      if constexpr (D == 64) {
        *reinterpret_cast<uint4*>(dst + 8 * g) =
            make_uint4(dev::pack_bf16x2(o[0][n][e], o[0][n][2 + e]), dev::pack_bf16x2(o[1][n][e], o[1][n][2 + e]),
                       dev::pack_bf16x2(o[2][n][e], o[2][n][2 + e]), dev::pack_bf16x2(o[3][n][e], o[3][n][2 + e]));
      } else {
#pragma unroll
        for (int i = 0; i < D / 16; i += 4)
          *reinterpret_cast<uint4*>(dst + 128 * (i / 8) + 16 * g + 2 * (i % 8)) =
              make_uint4(dev::pack_bf16x2(o[i][n][e], o[i][n][2 + e]), dev::pack_bf16x2(o[i + 1][n][e], o[i + 1][n][2 + e]),
                         dev::pack_bf16x2(o[i + 2][n][e], o[i + 2][n][2 + e]), dev::pack_bf16x2(o[i + 3][n][e], o[i + 3][n][2 + e]));
      }
      if (a.lse && g == 0) a.lse[row0 + h] = L[n][e] * 0.69314718055994531f;
    }
}

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads, 2) gqa_decode_kernel(const GqaDecodeArgs a, const __grid_constant__ CUtensorMap map) {
  using P = Shape<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = dev::smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t ring = base + warp * P::kStages * kUnit;
  const uint32_t scales = base + P::kScale + warp * P::kStages * 8;
  const uint32_t bars = base + P::kBars + warp * P::kStages * 8;
  float4* join = reinterpret_cast<float4*>(smem + P::kJoin);
  float* wl = reinterpret_cast<float*>(smem + P::kLse);          // [kWarps][kH] lse of each warp
  int* flag = reinterpret_cast<int*>(smem + P::kFlags);
  if (lane < P::kStages) tc::mbar_init(bars + 8 * lane, 2);
  tc::fence_mbar_init();
  __syncwarp();

  const int s0 = a.worker_ptr[blockIdx.x], s1 = a.worker_ptr[blockIdx.x + 1];
  bool dead = (base & 1023) != 0;          // the swizzle needs the ring aligned; never expected
  if (dead && threadIdx.x == 0) atomicOr(a.status, 2);
  Feed<P::kUnits> feed(a, s0, s1, warp);
  uint32_t loaded = 0, parity = 0;         // bit i: stage i holds a unit to take / parity of its barrier
  auto fill = [&](int stage) {
    const bool ok = feed.si < feed.se && !dead && feed.page >= 0 && feed.page < a.num_pages && Range(feed.s, feed.t0).any(P::kTokens);
    loaded = (loaded & ~(1u << stage)) | (ok ? 1u << stage : 0u);
    if (ok && lane == 0) {
      const int64_t kb = static_cast<int64_t>(feed.page) * 2 * a.kv_heads + feed.s.kv_head, vb = kb + a.kv_heads;
      const uint32_t bar = bars + 8 * stage, dst = ring + stage * kUnit;
      cp_async4(scales + 8 * stage, a.kv_scale + kb);
      cp_async4(scales + 8 * stage + 4, a.kv_scale + vb);
      cp_async_arrive(bar);
      tc::mbar_arrive_expect_tx(bar, kUnit);
      tma_load_2d(dst, &map, 0, static_cast<int>(kb * (kPage * D / 128) + feed.sub * (kHalf / 128)), bar);
      tma_load_2d(dst + kHalf, &map, 0, static_cast<int>(vb * (kPage * D / 128) + feed.sub * (kHalf / 128)), bar);
    }
    feed.next(warp);
  };
#pragma unroll 1
  for (int i = 0; i < P::kStages; ++i) fill(i);

  State<D, NT> st;
  Query<D, NT> Q;
  int stage = 0;
  const int t = lane & 3, g = lane >> 2;
#pragma unroll 1
  for (int si = s0; si < s1; ++si) {
    const GqaSegment s = load_segment(a.segs + si);
    load_query<D, NT>(Q, a, s, lane);
    st.clear();
    int kref = INT32_MIN;
#pragma unroll 1
    for (int u = warp; u < s.num_pages * P::kUnits; u += kWarps) {
      if (loaded >> stage & 1) {
        if (!dead && !tc::mbar_wait(bars + 8 * stage, parity >> stage & 1)) {
          dead = true;
          if (lane == 0) atomicOr(a.status, 1);
        }
        dead = __any_sync(kFull, dead);
        parity ^= 1u << stage;
        const Range range(s, page_of(s, s.page_begin + u / P::kUnits) * kPage + u % P::kUnits * P::kTokens);
        if (range.all(P::kTokens)) take_unit<D, E4M3, NT, false>(st, Q, ring + stage * kUnit, scales + 8 * stage, range, kref, lane);
        else take_unit<D, E4M3, NT, true>(st, Q, ring + stage * kUnit, scales + 8 * stage, range, kref, lane);
        __syncwarp();
      }
      fill(stage);
      stage = stage + 1 == P::kStages ? 0 : stage + 1;
    }
    // this warp's l over its lanes, its lse, and the four warps' weights
    const float vref = kref == INT32_MIN ? 0.0f : __uint_as_float(static_cast<uint32_t>(max(127 + kref, 1)) << 23);
    float L[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = st.l[n][e];
        l += __shfl_xor_sync(kFull, l, 4);
        l += __shfl_xor_sync(kFull, l, 8);
        l += __shfl_xor_sync(kFull, l, 16);
        st.l[n][e] = l;
        if (g == 0) wl[warp * kH + 8 * n + 2 * t + e] = l == 0.0f ? -INFINITY : st.m[n][e] - kLift + log2f(l);
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float lw[kWarps], M = -INFINITY, W = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          lw[w] = wl[w * kH + 8 * n + 2 * t + e];
          M = dev::max_nan(M, lw[w]);
        }
        float mine = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float c = M == -INFINITY ? 0.0f : exp2f(lw[w] - M);
          W += c;
          if (w == warp) mine = c;
        }
        L[n][e] = M == -INFINITY ? -INFINITY : M + log2f(W);
        const float c = mine == 0.0f ? 0.0f : mine / W * vref / st.l[n][e];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          st.o[i][n][e] *= c;
          st.o[i][n][2 + e] *= c;
        }
      }
    sum_warps<D, NT>(st.o, join, warp, lane);
    if (s.partial < 0) {
      if (warp == 0) write_out<D, NT>(a, s, st.o, L, lane);
      continue;
    }
    if (warp == 0) {
      float4* po = reinterpret_cast<float4*>(a.part_o + static_cast<int64_t>(s.partial) * kH * D);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) __stcg(po + (i * NT + n) * 32 + lane, make_float4(st.o[i][n][0], st.o[i][n][1], st.o[i][n][2], st.o[i][n][3]));
      if (g == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          __stcg(reinterpret_cast<float2*>(a.part_lse + static_cast<int64_t>(s.partial) * kH + 8 * n + 2 * t), make_float2(L[n][0], L[n][1]));
      }
      __threadfence();
      __syncwarp();
      if (lane == 0) *flag = atomicAdd(a.counters + s.counter, 1u) == static_cast<unsigned>(s.group_count - 1);
    }
    __syncthreads();
    if (*flag == 0) continue;
    // the group's last CTA: every partial is written. Warp w takes slots w, w + 4, ...
    __threadfence();
    if (threadIdx.x == 0) a.counters[s.counter] = 0;      // ready for the next run
    const float* gl = a.part_lse + static_cast<int64_t>(s.group_first) * kH;
    const float4* go = reinterpret_cast<const float4*>(a.part_o + static_cast<int64_t>(s.group_first) * kH * D);
    float M[NT][2], W[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float m0 = -INFINITY, m1 = -INFINITY;
      for (int k = g; k < s.group_count; k += 8) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(gl + k * kH + 8 * n + 2 * t));
        m0 = dev::max_nan(m0, x.x);
        m1 = dev::max_nan(m1, x.y);
      }
#pragma unroll
      for (int d = 4; d <= 16; d *= 2) {
        m0 = dev::max_nan(m0, __shfl_xor_sync(kFull, m0, d));
        m1 = dev::max_nan(m1, __shfl_xor_sync(kFull, m1, d));
      }
      float w0 = 0.0f, w1 = 0.0f;
      for (int k = g; k < s.group_count; k += 8) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(gl + k * kH + 8 * n + 2 * t));
        w0 += m0 == -INFINITY ? 0.0f : exp2f(x.x - m0);
        w1 += m1 == -INFINITY ? 0.0f : exp2f(x.y - m1);
      }
#pragma unroll
      for (int d = 4; d <= 16; d *= 2) {
        w0 += __shfl_xor_sync(kFull, w0, d);
        w1 += __shfl_xor_sync(kFull, w1, d);
      }
      M[n][0] = m0;
      M[n][1] = m1;
      W[n][0] = w0;
      W[n][1] = w1;
    }
    st.clear();
    for (int k = warp; k < s.group_count; k += kWarps) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(gl + k * kH + 8 * n + 2 * t));
        const float c0 = M[n][0] == -INFINITY ? 0.0f : exp2f(x.x - M[n][0]) / W[n][0];
        const float c1 = M[n][1] == -INFINITY ? 0.0f : exp2f(x.y - M[n][1]) / W[n][1];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const float4 v = __ldcg(go + static_cast<int64_t>(k) * (kH * D / 4) + (i * NT + n) * 32 + lane);
          st.o[i][n][0] += c0 * v.x;
          st.o[i][n][1] += c1 * v.y;
          st.o[i][n][2] += c0 * v.z;
          st.o[i][n][3] += c1 * v.w;
        }
      }
    }
    sum_warps<D, NT>(st.o, join, warp, lane);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) L[n][e] = M[n][e] == -INFINITY ? -INFINITY : M[n][e] + log2f(W[n][e]);
    if (warp == 0) write_out<D, NT>(a, s, st.o, L, lane);
  }
  if (dead) {
    // copies may still be on their way into this CTA's shared memory: let them land before it is given up
    const long long c0 = clock64();
    while (clock64() - c0 < (1ll << 28)) {}
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// The pool as rows of 128 bytes: a unit's K or V is 32 consecutive rows whatever the head size, and the
// 128-byte swizzle is a function of the linear offset in it alone.
cudaError_t pool_map(const GqaDecodeArgs& a, CUtensorMap* map) {
  const EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t rows = static_cast<cuuint64_t>(a.num_pages) * 2 * a.kv_heads * kPage * a.dim / 128;
  const cuuint64_t dims[2] = {128, rows}, strides[1] = {128};
  const cuuint32_t box[2] = {128, kHalf / 128}, estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.kv), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, bool E4M3, int NT>
cudaError_t launch(const GqaDecodeArgs& a, const CUtensorMap& map, cudaStream_t st) {
  // once per device: the attribute belongs to the device's copy of the kernel
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit) || bit == 0) {
    e = cudaFuncSetAttribute(gqa_decode_kernel<D, E4M3, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D, NT>::kBytes);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  gqa_decode_kernel<D, E4M3, NT><<<a.num_workers, kThreads, Shape<D, NT>::kBytes, st>>>(a, map);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_dim(const GqaDecodeArgs& a, const CUtensorMap& map, cudaStream_t st) {
  const bool wide = a.heads / a.kv_heads > 8;
  if (a.cache_dtype == QKVP_CACHE_E4M3) return wide ? launch<D, true, 2>(a, map, st) : launch<D, true, 1>(a, map, st);
  return wide ? launch<D, false, 2>(a, map, st) : launch<D, false, 1>(a, map, st);
}

}  // namespace

cudaError_t launch_gqa_decode(const GqaDecodeArgs& a, cudaStream_t st) {
  CUtensorMap map;
  std::memset(&map, 0, sizeof(map));
  if (a.kv != nullptr && a.num_pages > 0) {
    const cudaError_t e = pool_map(a, &map);
    if (e != cudaSuccess) return e;
  }
  switch (a.dim) {
    case 64: return launch_dim<64>(a, map, st);
    case 128: return launch_dim<128>(a, map, st);
    default: return launch_dim<256>(a, map, st);
  }
}

}  // namespace qkvp
