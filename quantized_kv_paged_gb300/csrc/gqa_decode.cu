// Decode attention over a paged 8-bit cache of K and V heads, one scale per (page, K or V, head).
//
// Per query head with its KV head's codes kc, vc and block scales sk, sv, over the visible tokens t:
//   z_t = sm_scale * sk (q . kc_t),  out = sum_t softmax(z)_t sv vc_t,  lse = log sum_t exp z_t.
// Reading the pages once is the floor (2 G operations per byte, G query heads per KV head: far below the
// tensor rate), so the kernel is a stream with the arithmetic kept out of its way.
//
// Work. A worker, a CTA's four warps (TEAM 4) or one warp (TEAM 1), walks its segments in units of 4 KB of K and
// 4 KB of V (64 / 32 / 16 tokens at D = 64 / 128 / 256). Each warp takes its units through a pipeline of its
// own: a ring of two that its lane 0 fills by TMA, one mbarrier per unit, no barrier with other warps until
// the segment ends. Two units, not three: 8 warps with 128 KB in flight per SM ran 44 x 32,768 tokens (8 KV
// heads of 128) in 428 us, 192 KB in 446, and 12 warps with 192 KB in 455; D = 64 takes 12 warps all the
// same, its units take more time each (128 x 1,024 tokens 24 against 26 us). The warps of a CTA join their
// sums at a segment's end; a group (request, KV head) cut into segments leaves normalised FP32 partials,
// joined by the last to arrive, in segment order, in two levels where there are many.
//
// Products. Heads are the columns (N = 8) of both products, so that G <= 8 wastes no rows:
//   S^T [tokens x heads] = K Q^T,  O^T [dims x heads] += V^T P^T,  mma m16n8k16, FP16 in, FP32 sums.
// E4M3 codes and INT8 codes are exact in FP16, Q is exact after a power of two per head. Both operands from
// the cache come straight from the bytes: which 16 dims make up a k-step, and which dim is which row of
// O^T, is free as long as Q and the output agree, so a lane takes 16 bytes of one token at a time and no
// byte moves between lanes. V^T needs two tokens of one dim in a register: two byte permutes of two
// tokens' words, then the conversion. The tokens of an 8-token block are taken in the order `tok8`, which
// makes every 16-byte (D = 64: 8-byte) shared-memory read free of bank conflicts under the TMA's 128-byte
// swizzle. P^T is S^T's accumulator layout transposed: one 8x8 transpose per 8 tokens. Computing S^T of the
// next unit along with the softmax of this one (rings of three) was 1 to 5 % slower: two warps per scheduler are
// short of issue slots, not of independent work (INT8, 16 heads: some 860 instructions a unit, 350 of them conversions).
//
// Softmax. One running reference m per head. It moves only when a logit passes it by 2^8 (a vote instead
// of a reduction per unit); P = 2^(z - m + 6) <= 2^14 is in FP16's normal range down to 2^-28 of the
// largest weight. l is summed from the unrounded FP32 values. The V scale sv = f 2^k of a page multiplies
// P: f (in [1, 2)) on the value, k in the exponent, less that of the warp's first page of the segment; l takes 2^-k
// back. That serves scales within 2^24 of the first. A segment with one further away is left for the worker's end, where
// it is taken in a second form, in which l has exponentials of its own, relative to the largest logit, while m bounds
// logit + k: what a page adds to l and what it adds to O^T may then be any powers of two apart, in any order. Every
// finite scale is taken. (The second form in the usual loop took 47.7 us instead of 42.8 for 4,096 rows of 128 tokens of
// D 128 with 16 heads. What is left of its cost, against a kernel without it: these 42.1, 16 x 4,096 tokens of D 256 with
// 10 heads 33.9 instead of 34.4.)
//
// Measured on GB300, kernel time: 44 x 32,768 tokens (8 KV heads of 128, 64 query heads, E4M3) 429 us, 2.96 GB at
// 6.9 TB/s, 103 % of the measured copy rate (DRAM busy 88 %, issue 33 %, tensor pipe 19 %); 1 x 1,048,576 (4
// heads) 163 us; 64 ragged requests (4 KV heads, 16 query heads each, INT8) 80 us. What is short is bound by its
// start and end: 2.5 to 3 us from the launch to the first unit (the worker's record, its page id and the page
// are three reads in line, cold), 1 us a unit, 1 us for a partial to be written and counted, 1 to 3 us to join.
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
// how far (log2) a logit may pass the reference; with 0 the 64 ragged INT8 requests take 83.1 us instead of 80.0
constexpr float kSlack = 8.0f;
constexpr float kLift = 6.0f;            // P is held as 2^(z - m + kLift)
constexpr float kNone = -3e38f;          // reference before the first unit
// How far (log2) V's scale may be from the first page's for l to be summed from P: the token of the largest logit has a P
// of at least 2^(kLift - 2 kReach) then, far from where FP32 flushes. The scale that a page of zeros counts as, below the
// first: beside such a page weights down to 2^-80 of its own are normal numbers in FP16. And the least first scale: O^T's
// last factor, weight / l 2^first, is not flushed for weights of a warp in its team of 2^-70 and more.
constexpr int kReach = 24, kZeros = 60, kLowest = -30;
constexpr int kFarApart = 1 << 20;       // in the place of the first scale's exponent

// At D = 256 and 16 heads Q^T would take 64 of the 255 registers next to 128 of O^T: it is kept in shared memory (16 x
// 4,096 tokens, 4 KV heads, 10 query heads each: 34 us, and 44 with it in registers, which spill).
constexpr bool query_in_smem(int dim, int nt) { return dim == 256 && nt == 2; }

template <int D, int NT, int TEAM>
struct Shape {
  static constexpr int kTokens = kHalf / D;            // tokens of a unit
  static constexpr int kUnits = kPage / kTokens;       // units of a page
  static constexpr int kCtas = gqa_ctas_per_sm(D, 8 * NT);
  static constexpr int kStages = 2;                    // units of a warp's ring
  static constexpr int kTiles = D / 16;                // 16-dim row tiles of O^T
  static constexpr int kPart = kTiles * NT * 32 * 16;  // bytes of one warp's O^T
  // shared memory: rings, the join's buffer, Q^T where it is kept there, the units' scales, barriers, per-warp lse,
  // per-warp references of l, the warps' flags of scales far apart, the join's flag
  static constexpr int kJoin = kWarps * kStages * kUnit;
  static constexpr int kQ = kJoin + (TEAM > 1 ? 2 * kPart : 0);
  static constexpr int kQBytes = query_in_smem(D, NT) ? D / 16 * 32 * 8 * NT : 0;   // of one worker
  static constexpr int kScale = kQ + kWarps / TEAM * kQBytes;
  static constexpr int kBars = kScale + kWarps * kStages * 8;
  static constexpr int kLse = kBars + kWarps * kStages * 8;
  static constexpr int kRefs = kLse + kWarps * kH * 4;
  static constexpr int kFar = kRefs + kWarps * kH * 4;
  static constexpr int kFlags = kFar + kWarps * 4;
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
  // any of the tokens [i, i + n) / all of the tokens [0, n)
  __device__ bool any(int i, int n) const { return i < min(sink, lim) || max(win, i) < min(lim, i + n); }
  __device__ bool all(int n) const { return lim >= n && (win <= 0 || sink >= n); }
};

// What the kernel before this one may have written while this one was already there is read by ordinary loads: the
// read-only path is for memory that does not change during a kernel's life.
template <class T>
__device__ __forceinline__ T load_record(const T* p) {
  static_assert(sizeof(T) % 16 == 0, "records are read 16 bytes at a time");
  T s;
  const int4* src = reinterpret_cast<const int4*>(p);
  int4* dst = reinterpret_cast<int4*>(&s);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 16); ++i) dst[i] = src[i];
  return s;
}

// Walks the units that one warp will take, ahead of their use; the page id of the unit it stands on is
// loaded when it gets there, one unit before it is needed.
template <int U, int TEAM>
struct Feed {
  const GqaDecodeArgs& a;
  int si, se, u, t0, sub;
  int32_t page;
  GqaSegment s;
  __device__ Feed(const GqaDecodeArgs& args, const GqaWorker& w, int member) : a(args), si(w.begin), se(w.end), u(member - TEAM), t0(0), sub(0), page(-1), s(w.first) {
    next(member);
  }
  __device__ void next(int member) {
    if (si >= se) return;
    u += TEAM;
    while (u >= s.num_pages * U) {
      if (++si >= se) return;
      s = load_record(a.segs + si);
      u = member;
    }
    const int local = page_of(s, s.page_begin + u / U);
    sub = u % U;
    page = a.kv_indices[s.page0 + local];
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
__device__ __forceinline__ float lds_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
  const uint2 v = lds64(addr);
  return make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
}

__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The pool to the TMA: boxes of a unit's K or V, and of a quarter of it.
struct PoolMaps {
  CUtensorMap unit, piece;
};

// Whether a unit, from token t0 of the request on, is in the pool and has visible tokens.
template <int D>
__device__ __forceinline__ bool seen(const GqaDecodeArgs& a, const GqaSegment& s, int32_t page, int t0) {
  return page >= 0 && page < a.num_pages && Range(s, t0).any(0, kHalf / D);
}

// One lane: the copies of a unit's K, V and scales, which complete a phase of the barrier.
template <int D>
__device__ __forceinline__ void load_unit(const GqaDecodeArgs& a, const PoolMaps& maps, const GqaSegment& s, int32_t page, int t0, int sub,
                                          uint32_t dst, uint32_t scale, uint32_t bar) {
  constexpr int kTokens = kHalf / D;
  const int64_t kb = static_cast<int64_t>(page) * 2 * a.kv_heads + s.kv_head, vb = kb + a.kv_heads;
  cp_async4(scale, a.kv_scale + kb);
  cp_async4(scale + 4, a.kv_scale + vb);
  cp_async_arrive(bar);
  const int krow = static_cast<int>(kb * (kPage * D / 128)) + sub * (kHalf / 128);
  const int vrow = static_cast<int>(vb * (kPage * D / 128)) + sub * (kHalf / 128);
  const Range range(s, t0);
  if (range.all(kTokens)) {
    tc::mbar_arrive_expect_tx(bar, kUnit);
    tma_load_2d(dst, &maps.unit, 0, krow, bar);
    tma_load_2d(dst + kHalf, &maps.unit, 0, vrow, bar);
  } else {
    // of a unit at an edge only the quarters that hold a visible token; what is left in the others is masked
    constexpr int kPiece = kTokens / 4;
    uint32_t bytes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) bytes += range.any(i * kPiece, kPiece) ? 2 * kHalf / 4 : 0;
    tc::mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!range.any(i * kPiece, kPiece)) continue;
      tma_load_2d(dst + i * (kHalf / 4), &maps.piece, 0, krow + i * (kHalf / 4 / 128), bar);
      tma_load_2d(dst + kHalf + i * (kHalf / 4), &maps.piece, 0, vrow + i * (kHalf / 4 / 128), bar);
    }
  }
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
  static constexpr bool kShared = query_in_smem(D, NT);
  uint32_t q[kShared ? 1 : D / 64][4][2][NT];
  uint32_t addr;            // of the worker's copy in shared memory: 16 bytes per lane and k-step
  float scale[NT][2];       // logit factor of the lane's columns: sm_scale log2(e) / (the head's power of two)
};

// The lane's share of a segment's queries as stored: 16 dims of GROUPS 64-dim groups, from group c0 on, of heads g
// and 8 + g. A team that keeps Q^T in shared memory splits the groups among its warps.
template <int D, int NT, int TEAM>
struct RawQuery {
  static constexpr bool kSplit = Query<D, NT>::kShared && TEAM > 1;
  static constexpr int kGroups = kSplit ? 1 : D / 64;
  static_assert(!kSplit || D / 64 == TEAM, "a 64-dim group per warp");
  uint4 v[NT][kGroups][2];
  __device__ void load(const GqaDecodeArgs& a, const GqaSegment& s, int member, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = 8 * n + g;
      const uint16_t* row = a.q + (static_cast<int64_t>(s.req) * a.heads + s.head0 + h) * D + (kSplit ? 64 * member : 0) + 16 * t;
#pragma unroll
      for (int c = 0; c < kGroups; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          v[n][c][k] = h < s.heads ? *reinterpret_cast<const uint4*>(row + 64 * c + 8 * k) : make_uint4(0, 0, 0, 0);
    }
  }
};

// `top`: shared memory [kWarps][kH] for the largest |q| of each warp's groups, where the groups are split.
template <int D, int NT, int TEAM>
__device__ __forceinline__ void convert_query(Query<D, NT>& Q, const RawQuery<D, NT, TEAM>& raw, float scale_log2, float* top, int member, int lane) {
  using R = RawQuery<D, NT, TEAM>;
  const int g = lane >> 2, t = lane & 3;
  float amax[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    amax[n] = 0.0f;
#pragma unroll
    for (int c = 0; c < R::kGroups; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x[8];
        dev::bf16x8_to_float(raw.v[n][c][k], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax[n] = fmaxf(amax[n], fabsf(x[i]));
      }
    amax[n] = fmaxf(amax[n], __shfl_xor_sync(kFull, amax[n], 1));
    amax[n] = fmaxf(amax[n], __shfl_xor_sync(kFull, amax[n], 2));
    if (R::kSplit && t == 0) top[member * kH + 8 * n + g] = amax[n];
  }
  if constexpr (R::kSplit) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) amax[n] = fmaxf(amax[n], top[w * kH + 8 * n + g]);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // 2^e that brings the largest |q| to [2^14, 2^15), where FP16 holds 8 bits down to 2^-29 of it
    const int ex = static_cast<int>(__float_as_uint(amax[n]) >> 23);
    const int e = amax[n] == 0.0f ? 0 : min(126, 14 + 127 - ex);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23), down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int c = 0; c < R::kGroups; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t w[4] = {raw.v[n][c][k].x, raw.v[n][c][k].y, raw.v[n][c][k].z, raw.v[n][c][k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = dev::bf16x2_to_f16x2(w[i], up);
          if constexpr (Query<D, NT>::kShared) tc::sts_u32(Q.addr + (((R::kSplit ? member : c) * 4 + 2 * k + i / 2) * 32 + lane) * 16 + (i % 2) * 8 + n * 4, x);
          else Q.q[c][2 * k + i / 2][i % 2][n] = x;
        }
      }
    const float f = scale_log2 * down;
#pragma unroll
    for (int e2 = 0; e2 < 2; ++e2) Q.scale[n][e2] = __shfl_sync(kFull, f, 4 * (2 * t + e2));
  }
  if constexpr (R::kSplit) __syncthreads();
  else if constexpr (Query<D, NT>::kShared) __syncwarp();
}

// The exponent of a scale, at most 127; that of FP32's smallest normal number where it is below that.
__device__ __forceinline__ int exponent_of(float scale) {
  return min(max(static_cast<int>(__float_as_uint(scale) >> 23 & 0xFF), 1), 254) - 127;
}

// Whether a V scale is out of reach of the warp's first one of the segment that is not 0, whose exponent is `first`
// (INT32_MIN: none yet, then it is this one).
__device__ __forceinline__ bool out_of_reach(float scale, int& first) {
  const int vk = exponent_of(scale);
  if (scale == 0.0f) return false;
  if (first == INT32_MIN) first = vk;
  return abs(vk - first) > kReach || first < kLowest || vk == 127;
}

// One unit: S^T, the running softmax, O^T. PARTIAL: some of its tokens may be not visible. first: the exponent of the
// warp's first V scale of the segment that is not 0 (INT32_MIN: none yet). A unit whose scale is out of reach of it makes it
// kFarApart; the state is worth nothing from there on. APART: no scale is; l is relative to the references at `ref` in
// shared memory (for the lane's columns), and both references are renewed at every unit.
template <int D, bool E4M3, int NT, int TEAM, bool PARTIAL, bool APART>
__device__ __forceinline__ void take_unit(State<D, NT>& st, const Query<D, NT>& Q, uint32_t kbase, uint32_t scale_addr,
                                          const Range& range, int& first, uint32_t ref, int lane) {
  constexpr int MT = kHalf / D / 16;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t vbase = kbase + kHalf;
  const float2 sc = lds_f2(scale_addr);
  // one sum of products: two, of the even and of the odd 64-dim groups, are as fast (9 shapes of D
  // 256, where one is a chain of 16: within 1 %, 4,096 rows of 32 to 256 tokens 53.9 us, 54.5 with two)
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
        uint32_t b[2][NT];
        if constexpr (Query<D, NT>::kShared) {
          const uint4 x = lds128(Q.addr + ((c * 4 + j) * 32 + lane) * 16);
          b[0][0] = x.x;
          b[0][NT - 1] = x.y;
          b[1][0] = x.z;
          b[1][NT - 1] = x.w;
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            b[0][n] = Q.q[c][j][0][n];
            b[1][n] = Q.q[c][j][1][n];
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) dev::mma_f16(s[m][n], a0, a1, a2, a3, b[0][n], b[1][n]);
      }
    }
  }

  // V's bytes are loaded ahead of the softmax, so that they wait for it and not it for them: 4,096 rows of 512 tokens of
  // D 256 with 16 heads take 195 us, and 204 with the loads behind it. With fewer registers left, at D 128 with 16
  // heads and at D 256 in a team, they come behind it: 4,096 rows of 128 tokens of D 128 42.8 us, 46.8 ahead of it;
  // 16 x 4,096 tokens of D 256 34.7 us, 34.9. D 64 and up to 8 heads do not tell the two apart.
  constexpr bool kEarlyV = NT == 1 || D == 64 || (D == 256 && TEAM == 1);
  const int ta = tok8<D>(2 * t), tb = tok8<D>(2 * t + 1);
  constexpr int kSides = (D + 127) / 128;              // 128-dim halves of a token
  constexpr int W = D == 64 ? 2 : 4;                   // words of a lane's piece of a token
  uint32_t v[kSides][MT][4][W];                        // tokens ta, tb, ta + 8, tb + 8 of each tile
  auto load_v = [&](int h, int m) {
    const uint32_t oa = ta * D + h * 128 + g * 4 * W, ob = tb * D + h * 128 + g * 4 * W;
    const uint32_t va = vbase + (oa ^ (((oa >> 7) & 7) << 4)), vb = vbase + (ob ^ (((ob >> 7) & 7) << 4));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      uint32_t at = r & 1 ? vb : va;
      if (D == 64 && r >= 2) at ^= 64;
      at += (16 * m + (r >= 2 ? 8 : 0)) * D;
      if constexpr (D == 64) {
        const uint2 x = lds64(at);
        v[h][m][r][0] = x.x;
        v[h][m][r][1] = x.y;
      } else {
        const uint4 x = lds128(at);
        v[h][m][r][0] = x.x;
        v[h][m][r][1] = x.y;
        v[h][m][r][2] = x.z;
        v[h][m][r][3] = x.w;
      }
      // what stands behind a token that is not visible may be NaN, and 0 * NaN is not 0
      if (PARTIAL && !range.sees(16 * m + (r >= 2 ? 8 : 0) + (r & 1 ? tb : ta))) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[h][m][r][i] = 0;
      }
    }
  };
  if constexpr (kEarlyV) {
#pragma unroll
    for (int h = 0; h < kSides; ++h)
#pragma unroll
      for (int m = 0; m < MT; ++m) load_v(h, m);
  }

  // V's scale f 2^vk, k relative to the first. A page of zeros adds to l alone.
  const bool out = out_of_reach(sc.y, first), zero = sc.y == 0.0f;
  const int vk = exponent_of(sc.y), k = zero ? -kZeros : vk - first;
  if (!APART && out) first = kFarApart;
  // (an f of 4 times a P of 2^14 would be past FP16's largest number)
  const float f = sc.y * __uint_as_float(static_cast<uint32_t>(127 - (APART ? min(vk, 126) : vk)) << 23) * (APART && vk == 127 ? 0.5f : 1.0f);
  const float kz = APART && zero ? -INFINITY : static_cast<float>(k);

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
  bool move = APART;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) move |= top[n][e] + kz > st.m[n][e] + kSlack;
  if (__any_sync(kFull, move)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float c[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = top[n][e];
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
        if constexpr (APART) {
          // the lanes of a column write one value, once all have read the last
          const uint32_t at = ref + 32 * n + 4 * e;
          const float was = lds_f1(at), y = fmaxf(fminf(x, 3e38f), was);
          __syncwarp();
          tc::sts_u32(at, __float_as_uint(y));
          float l = st.l[n][e] * dev::fast_exp2(was - y);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) l += dev::fast_exp2(s[m][n][2 * r + e] - y + kLift);
          st.l[n][e] = l;
        }
        x = fmaxf(fminf(x + kz, 3e38f), st.m[n][e]);
        c[e] = dev::fast_exp2(st.m[n][e] - x);
        if constexpr (!APART) st.l[n][e] *= c[e];
        st.m[n][e] = x;
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
  const float back = __uint_as_float(static_cast<uint32_t>(APART ? 0 : 127 - k) << 23);
  uint32_t p[MT][NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float sum[2] = {0.0f, 0.0f};
    const float b0 = kz - st.m[n][0] + kLift, b1 = kz - st.m[n][1] + kLift;
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
    for (int e = 0; e < 2; ++e) {
      if constexpr (!APART) st.l[n][e] += sum[e] * back;
    }
  }

#pragma unroll
  for (int h = 0; h < kSides; ++h) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (!kEarlyV) load_v(h, m);
#pragma unroll
      for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {                  // dims 4 i + 2 q (row g) and 4 i + 2 q + 1 (row g + 8)
          uint32_t a0, a1, a2, a3;
          codes_to_f16<E4M3>(__byte_perm(v[h][m][0][i], v[h][m][1][i], q ? 0x7362 : 0x5140), a0, a1);
          codes_to_f16<E4M3>(__byte_perm(v[h][m][2][i], v[h][m][3][i], q ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) dev::mma_f16(st.o[8 * h + 2 * i + q][n], a0, a1, a2, a3, p[m][n][0], p[m][n][1]);
        }
      }
    }
  }
}

// Sums the four warps' O^T so that warp w is left with the sum of its quarter of the tiles, w D / 64 .., in the
// first elements of o: halves first (with warp ^ 2), then quarters (with warp ^ 1), (o0 + o2) + (o1 + o3) for
// every tile. Between the two exchanges a warp writes where only it has read.
template <int D, int NT>
__device__ __forceinline__ void scatter_sum(float (&o)[D / 16][NT][4], float4* buf, int warp, int lane) {
  constexpr int kHalfTiles = D / 32, kQuarter = D / 64, kVec = kHalfTiles * NT * 32;
#pragma unroll
  for (int i = 0; i < kHalfTiles; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float4 out;
      float* v = &out.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = warp & 2 ? o[i][n][k] : o[kHalfTiles + i][n][k];
        o[i][n][k] = warp & 2 ? o[kHalfTiles + i][n][k] : o[i][n][k];
      }
      buf[warp * kVec + (i * NT + n) * 32 + lane] = out;
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHalfTiles; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float4 v = buf[(warp ^ 2) * kVec + (i * NT + n) * 32 + lane];
      o[i][n][0] += v.x;
      o[i][n][1] += v.y;
      o[i][n][2] += v.z;
      o[i][n][3] += v.w;
    }
#pragma unroll
  for (int i = 0; i < kQuarter; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float4 out;
      float* v = &out.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = warp & 1 ? o[i][n][k] : o[kQuarter + i][n][k];
        o[i][n][k] = warp & 1 ? o[kQuarter + i][n][k] : o[i][n][k];
      }
      buf[(warp ^ 2) * kVec + (i * NT + n) * 32 + lane] = out;
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQuarter; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float4 v = buf[(warp ^ 3) * kVec + (i * NT + n) * 32 + lane];
      o[i][n][0] += v.x;
      o[i][n][1] += v.y;
      o[i][n][2] += v.z;
      o[i][n][3] += v.w;
    }
}

// 2^(top - M) / sum_w 2^(lse_w - M) over the four warps' lse at stride kH, M their maximum: what a sum that
// a warp holds relative to 2^top counts in the whole. `joined` becomes the whole's lse.
__device__ __forceinline__ float weigh(const float* lse, float top, float& joined) {
  float x[kWarps], M = -INFINITY, W = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    x[w] = lse[w * kH];
    M = dev::max_nan(M, x[w]);
  }
  if (M == -INFINITY) {
    joined = -INFINITY;
    return 0.0f;
  }
#pragma unroll
  for (int w = 0; w < kWarps; ++w) W += dev::fast_exp2(x[w] - M);
  const float mine = __fdividef(dev::fast_exp2(top - M), W);
  joined = M + lg2(W);
  return mine;
}

// The first TILES tiles of o (normalised), which are O^T's tiles tile0 .., and the base-2 lse of a segment's heads, to
// out and lse. A lane holds 2 TILES consecutive dims of each of its heads.
template <int D, int NT, int TILES>
__device__ __forceinline__ void write_out(const GqaDecodeArgs& a, const GqaSegment& s, const float (&o)[D / 16][NT][4], int tile0,
                                          const float (&L)[NT][2], int lane) {
  const int g = lane >> 2, t = lane & 3;
  const int64_t row0 = static_cast<int64_t>(s.req) * a.heads + s.head0;
  // tile i of a 128-dim half: dims 16 g + 2 i, 16 g + 2 i + 1 of it (D = 64: 8 g + ...)
  const int dim0 = D == 64 ? 8 * g + 2 * tile0 : 128 * (tile0 / 8) + 16 * g + 2 * (tile0 % 8);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = 8 * n + 2 * t + e;
      if (h >= s.heads) continue;
      uint16_t* dst = a.out + (row0 + h) * D + dim0;
      uint32_t w[TILES];
#pragma unroll
      for (int i = 0; i < TILES; ++i) w[i] = dev::pack_bf16x2(o[i][n][e], o[i][n][2 + e]);
      if constexpr (TILES == 1) {
        *reinterpret_cast<uint32_t*>(dst) = w[0];
      } else if constexpr (TILES == 2) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int i = 0; i < TILES; i += 4)
          *reinterpret_cast<uint4*>(dst + 128 * (i / 8) + 2 * (i % 8)) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
      }
      if (a.lse && g == 0 && tile0 == 0) a.lse[row0 + h] = L[n][e] * 0.69314718055994531f;
    }
}

// The end of a segment: the warp's sums become outputs, or a partial that the last of its group joins. first: the exponent
// that O^T is relative to. Where one of the warps met scales far apart nothing is done, and false returned.
template <int D, int NT, int TEAM>
__device__ __forceinline__ bool finish_segment(const GqaDecodeArgs& a, const GqaSegment& s, State<D, NT>& st, int first, uint8_t* smem, int warp,
                                               int lane) {
  using P = Shape<D, NT, TEAM>;
  const int member = TEAM == 1 ? 0 : warp, t = lane & 3, g = lane >> 2;
  float4* join = reinterpret_cast<float4*>(smem + P::kJoin);
  float* wl = reinterpret_cast<float*>(smem + P::kLse);          // [kWarps][kH] lse of each warp
  int* flag = reinterpret_cast<int*>(smem + P::kFlags);
  if (TEAM == 1 && __builtin_expect(first == kFarApart, 0)) return false;
  // this warp's l over its lanes, and its lse
  const float vref = first == INT32_MIN ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 + first) << 23);
  float L[NT][2], weight[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = st.l[n][e];
      l += __shfl_xor_sync(kFull, l, 4);
      l += __shfl_xor_sync(kFull, l, 8);
      l += __shfl_xor_sync(kFull, l, 16);
      st.l[n][e] = l;
      L[n][e] = l == 0.0f ? -INFINITY : st.m[n][e] - kLift + lg2(l);
      weight[n][e] = 1.0f;
      if (TEAM > 1 && g == 0) wl[warp * kH + 8 * n + 2 * t + e] = L[n][e];
    }
  if constexpr (TEAM > 1) {
    int* far = reinterpret_cast<int*>(smem + P::kFar);
    if (lane == 0) far[warp] = first == kFarApart;
    __syncthreads();
    const int4 x = *reinterpret_cast<const int4*>(far);
    if (__builtin_expect((x.x | x.y | x.z | x.w) != 0, 0)) {
      __syncthreads();                     // all have read it before the next segment writes it
      return false;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) weight[n][e] = weigh(wl + 8 * n + 2 * t + e, L[n][e], L[n][e]);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float c = st.l[n][e] == 0.0f || weight[n][e] == 0.0f ? 0.0f : __fdividef(weight[n][e], st.l[n][e]) * vref;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        st.o[i][n][e] *= c;
        st.o[i][n][2 + e] *= c;
      }
    }
  // from here on a warp of a team owns a quarter of the tiles, the first kOwn of st.o
  constexpr int kOwn = D / 16 / TEAM;
  const int tile0 = member * kOwn;
  if constexpr (TEAM > 1) scatter_sum<D, NT>(st.o, join, warp, lane);
  if (s.partial < 0) {
    write_out<D, NT, kOwn>(a, s, st.o, tile0, L, lane);
    return true;
  }
  int slot = s.partial, from = s.group_first, count = s.group_count, counter = s.counter;
  bool top = s.top_counter < 0;
#pragma unroll 1
  while (true) {
    float4* po = reinterpret_cast<float4*>(a.part_o + static_cast<int64_t>(slot) * kH * D) + tile0 * NT * 32 + lane;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) __stcg(po + (i * NT + n) * 32, make_float4(st.o[i][n][0], st.o[i][n][1], st.o[i][n][2], st.o[i][n][3]));
    if (member == 0 && g == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        __stcg(reinterpret_cast<float2*>(a.part_lse + static_cast<int64_t>(slot) * kH + 8 * n + 2 * t), make_float2(L[n][0], L[n][1]));
    }
    // arrive once all of the slot is written
    __threadfence();
    int last = 0;
    if constexpr (TEAM > 1) {
      __syncthreads();
      if (threadIdx.x == 0) *flag = atomicAdd(a.counters + counter, 1u) == static_cast<unsigned>(count - 1);
      __syncthreads();
      last = *flag;
    } else {
      __syncwarp();
      if (lane == 0) last = atomicAdd(a.counters + counter, 1u) == static_cast<unsigned>(count - 1);
      last = __shfl_sync(kFull, last, 0);
    }
    if (last == 0) break;
    // The last arrival: every slot is written. Each warp joins its tiles of all slots, in their order, a few
    // slots at a time with their lse, under a running maximum.
    __threadfence();
    if (member == 0 && lane == 0) a.counters[counter] = 0;        // ready for the next run
    const float* gl = a.part_lse + static_cast<int64_t>(from) * kH + 2 * t;
    const float4* go = reinterpret_cast<const float4*>(a.part_o + static_cast<int64_t>(from) * kH * D) + tile0 * NT * 32 + lane;
    float M[NT][2], W[NT][2];
    st.clear();
#pragma unroll
    for (int n = 0; n < NT; ++n) M[n][0] = M[n][1] = -INFINITY, W[n][0] = W[n][1] = 0.0f;
    constexpr int kVecs = P::kCtas == 3 ? 16 : 32;                // 16-byte loads in flight of a lane
    constexpr int kBatch = kOwn * NT >= kVecs ? 1 : kVecs / (kOwn * NT) > 8 ? 8 : kVecs / (kOwn * NT);
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += kBatch) {
      float4 v[kBatch][kOwn][NT];
      float2 x[kBatch][NT];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int k = k0 + j;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          x[j][n] = k < count ? __ldcg(reinterpret_cast<const float2*>(gl + k * kH + 8 * n)) : make_float2(-INFINITY, -INFINITY);
#pragma unroll
          for (int i = 0; i < kOwn; ++i)
            v[j][i][n] = k < count ? __ldcg(go + static_cast<int64_t>(k) * (kH * D / 4) + (i * NT + n) * 32) : make_float4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = M[n][e];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) m = dev::max_nan(m, e ? x[j][n].y : x[j][n].x);
          const float c = m == -INFINITY ? 1.0f : dev::fast_exp2(M[n][e] - m);
          W[n][e] *= c;
          M[n][e] = m;
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            st.o[i][n][e] *= c;
            st.o[i][n][2 + e] *= c;
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const float z = m == -INFINITY ? 0.0f : dev::fast_exp2((e ? x[j][n].y : x[j][n].x) - m);
            W[n][e] += z;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
              st.o[i][n][e] += z * (e ? v[j][i][n].y : v[j][i][n].x);
              st.o[i][n][2 + e] += z * (e ? v[j][i][n].w : v[j][i][n].z);
            }
          }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float c = W[n][e] == 0.0f ? 0.0f : __fdividef(1.0f, W[n][e]);
        L[n][e] = W[n][e] == 0.0f ? -INFINITY : M[n][e] + lg2(W[n][e]);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          st.o[i][n][e] *= c;
          st.o[i][n][2 + e] *= c;
        }
      }
    if (top) {
      write_out<D, NT, kOwn>(a, s, st.o, tile0, L, lane);
      break;
    }
    slot = s.sub_slot;
    from = s.top_first;
    count = s.top_count;
    counter = s.top_counter;
    top = true;
  }
  return true;
}

// Whether a warp's part of a segment was left: the units in their order, by their V scales alone.
template <int D, int TEAM>
__device__ bool was_left(const GqaDecodeArgs& a, const GqaSegment& s, int member) {
  constexpr int kTokens = kHalf / D, kUnits = kPage / kTokens;
  int first = INT32_MIN;
#pragma unroll 1
  for (int u = member; u < s.num_pages * kUnits; u += TEAM) {
    const int local = page_of(s, s.page_begin + u / kUnits);
    const int32_t page = a.kv_indices[s.page0 + local];
    if (!seen<D>(a, s, page, local * kPage + u % kUnits * kTokens)) continue;
    if (out_of_reach(a.kv_scale[(static_cast<int64_t>(page) * 2 + 1) * a.kv_heads + s.kv_head], first)) return true;
  }
  return false;
}

// A worker's segments whose V scales are far apart, after all others, with nothing else alive: the usual form loses
// registers to this one in its own loop. The units come one after the other through the first stage of the warp's ring,
// whose barrier's parity is given. O^T is normalised here, so that the segment's end finds an l of 1 and values relative
// to 2^0. Returns whether a wait ran out.
template <int D, bool E4M3, int NT, int TEAM>
__device__ __forceinline__ bool take_apart(const GqaDecodeArgs& a, const PoolMaps& maps, unsigned parity, bool dead) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const GqaWorker* w = a.workers + (TEAM == 1 ? blockIdx.x * kWarps + warp : blockIdx.x);
  const int begin = w->begin, end = w->end;          // read again, not kept
  using P = Shape<D, NT, TEAM>;
  const int member = TEAM == 1 ? 0 : warp;
  volatile int* far = reinterpret_cast<volatile int*>(smem + P::kFar);
  float* wl = reinterpret_cast<float*>(smem + P::kLse);
  const uint32_t base = dev::smem_u32(smem), ref = base + P::kRefs + warp * kH * 4 + 8 * (lane & 3);
  const uint32_t ring = base + warp * P::kStages * kUnit, scale = base + P::kScale + warp * P::kStages * 8, bar = base + P::kBars + warp * P::kStages * 8;
  Query<D, NT> Q;
  Q.addr = base + P::kQ + (TEAM == 1 ? warp : 0) * P::kQBytes;
#pragma unroll 1
  for (int si = begin; si < end; ++si) {
    const GqaSegment s = load_record(a.segs + si);
    bool mine = was_left<D, TEAM>(a, s, member);
    if constexpr (TEAM > 1) {
      if (lane == 0) far[warp] = mine;
      __syncthreads();
      mine = (far[0] | far[1] | far[2] | far[3]) != 0;
      __syncthreads();                     // all have read it before it is written again
    }
    if (!mine) continue;
    RawQuery<D, NT, TEAM> raw;
    raw.load(a, s, member, lane);
    convert_query<D, NT, TEAM>(Q, raw, a.scale_log2, wl, member, lane);
    State<D, NT> st;
    st.clear();
    int first = INT32_MIN;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) tc::sts_u32(ref + 32 * n + 4 * e, __float_as_uint(kNone));
#pragma unroll 1
    for (int u = member; u < s.num_pages * P::kUnits; u += TEAM) {
      const int local = page_of(s, s.page_begin + u / P::kUnits), t0 = local * kPage + u % P::kUnits * P::kTokens;
      const int32_t page = a.kv_indices[s.page0 + local];
      if (dead || !seen<D>(a, s, page, t0)) continue;
      if (lane == 0) load_unit<D>(a, maps, s, page, t0, u % P::kUnits, ring, scale, bar);
      if (!tc::mbar_wait(bar, parity)) {
        dead = true;
        if (lane == 0) atomicOr(a.status, 1);
      }
      dead = __any_sync(kFull, dead);
      parity ^= 1u;
      take_unit<D, E4M3, NT, TEAM, true, true>(st, Q, ring, scale, Range(s, t0), first, ref, lane);
      __syncwarp();
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = st.l[n][e];
        l += __shfl_xor_sync(kFull, l, 4);
        l += __shfl_xor_sync(kFull, l, 8);
        l += __shfl_xor_sync(kFull, l, 16);
        // sum 2^z V = O^T 2^(first + m - kLift), of a whole of 2^lse: in two factors, neither of which is flushed
        const float lse = lds_f1(ref + 32 * n + 4 * e) - kLift + lg2(l);
        const float x = first == INT32_MIN || l == 0.0f ? -600.0f : static_cast<float>(first) + (st.m[n][e] - lse) - kLift;
        const float half = floorf(0.5f * x), c0 = dev::fast_exp2(half), c1 = dev::fast_exp2(x - half);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          st.o[i][n][e] = st.o[i][n][e] * c0 * c1;
          st.o[i][n][2 + e] = st.o[i][n][2 + e] * c0 * c1;
        }
        st.l[n][e] = l != 0.0f && lane < 4 ? 1.0f : 0.0f;          // one lane of the eight that share a column
        st.m[n][e] = lse + kLift;
      }
    finish_segment<D, NT, TEAM>(a, s, st, 0, smem, warp, lane);
  }
  return dead;
}

// TEAM warps share a worker's segments: 4 (the CTA) or 1 (each warp a worker of its own, no barrier at all).
template <int D, bool E4M3, int NT, int TEAM>
__global__ void __launch_bounds__(kThreads, Shape<D, NT, TEAM>::kCtas) gqa_decode_kernel(const __grid_constant__ GqaDecodeArgs a, const __grid_constant__ PoolMaps maps) {
  using P = Shape<D, NT, TEAM>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = dev::smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int member = TEAM == 1 ? 0 : warp;
  const uint32_t ring = base + warp * P::kStages * kUnit;
  const uint32_t scales = base + P::kScale + warp * P::kStages * 8;
  const uint32_t bars = base + P::kBars + warp * P::kStages * 8;
  float* wl = reinterpret_cast<float*>(smem + P::kLse);
  if (lane < P::kStages) tc::mbar_init(bars + 8 * lane, 2);
  tc::fence_mbar_init();
  __syncwarp();

  // the launch may overlap the end of the kernel before it in the stream (launch_overlapped)
  dev::allow_dependents();
  dev::wait_for_previous();
  const GqaWorker w = load_record(a.workers + (TEAM == 1 ? blockIdx.x * kWarps + warp : blockIdx.x));
  bool dead = (base & 1023) != 0;          // the swizzle needs the ring aligned; never expected
  if (dead && threadIdx.x == 0) atomicOr(a.status, 2);
  // a segment's queries are loaded before what precedes its first unit: the first fills, the join of the last segment
  RawQuery<D, NT, TEAM> raw;
  GqaSegment s = w.first;
  if (w.begin < w.end) raw.load(a, s, member, lane);
  Feed<P::kUnits, TEAM> feed(a, w, member);
  uint32_t loaded = 0, parity = 0;         // bit i: stage i holds a unit to take / parity of its barrier
  auto fill = [&](int stage) {
    const bool ok = feed.si < feed.se && !dead && seen<D>(a, feed.s, feed.page, feed.t0);
    loaded = (loaded & ~(1u << stage)) | (ok ? 1u << stage : 0u);
    if (ok && lane == 0) load_unit<D>(a, maps, feed.s, feed.page, feed.t0, feed.sub, ring + stage * kUnit, scales + 8 * stage, bars + 8 * stage);
    feed.next(member);
  };
#pragma unroll 1
  for (int i = 0; i < P::kStages; ++i) fill(i);

  State<D, NT> st;
  Query<D, NT> Q;
  Q.addr = base + P::kQ + (TEAM == 1 ? warp : 0) * P::kQBytes;
  int stage = 0;
  bool left = false;                       // segments whose V scales are far apart are left for later
#pragma unroll 1
  for (int si = w.begin; si < w.end;) {
    // no warp still reads the last segment's Q^T in shared memory: that segment ended at a barrier
    convert_query<D, NT, TEAM>(Q, raw, a.scale_log2, wl, member, lane);
    st.clear();
    int vfirst = INT32_MIN;
#pragma unroll 1
    for (int u = member; u < s.num_pages * P::kUnits; u += TEAM) {
      if (loaded >> stage & 1) {
        if (!dead && !tc::mbar_wait(bars + 8 * stage, parity >> stage & 1)) {
          dead = true;
          if (lane == 0) atomicOr(a.status, 1);
        }
        dead = __any_sync(kFull, dead);
        parity ^= 1u << stage;
        const Range range(s, page_of(s, s.page_begin + u / P::kUnits) * kPage + u % P::kUnits * P::kTokens);
        if (range.all(P::kTokens)) take_unit<D, E4M3, NT, TEAM, false, false>(st, Q, ring + stage * kUnit, scales + 8 * stage, range, vfirst, 0, lane);
        else take_unit<D, E4M3, NT, TEAM, true, false>(st, Q, ring + stage * kUnit, scales + 8 * stage, range, vfirst, 0, lane);
        __syncwarp();
      }
      fill(stage);
      stage = stage + 1 == P::kStages ? 0 : stage + 1;
    }
    GqaSegment next = s;
    if (++si < w.end) {
      next = load_record(a.segs + si);
      raw.load(a, next, member, lane);
    }
    if (!finish_segment<D, NT, TEAM>(a, s, st, vfirst, smem, warp, lane)) left = true;
    s = next;
  }
  if (__builtin_expect(left, 0)) dead = take_apart<D, E4M3, NT, TEAM>(a, maps, parity & 1u, dead);
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
cudaError_t pool_map(const GqaDecodeArgs& a, cuuint32_t box_rows, CUtensorMap* map) {
  const EncodeTiledFn fn = encode_tiled();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t rows = static_cast<cuuint64_t>(a.num_pages) * 2 * a.kv_heads * kPage * a.dim / 128;
  const cuuint64_t dims[2] = {128, rows}, strides[1] = {128};
  const cuuint32_t box[2] = {128, box_rows}, estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.kv), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, bool E4M3, int NT, int TEAM>
cudaError_t launch(const GqaDecodeArgs& a, const PoolMaps& maps, cudaStream_t st) {
  constexpr int bytes = Shape<D, NT, TEAM>::kBytes;
  auto kernel = gqa_decode_kernel<D, E4M3, NT, TEAM>;
  // once per device: the attribute belongs to the device's copy of the kernel
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_overlapped(kernel, a.num_workers * TEAM / kWarps, kThreads, bytes, st, a, maps);
}

template <int D, bool E4M3>
cudaError_t launch_dim(const GqaDecodeArgs& a, const PoolMaps& maps, cudaStream_t st) {
  if (a.heads / a.kv_heads > 8) return a.team == 1 ? launch<D, E4M3, 2, 1>(a, maps, st) : launch<D, E4M3, 2, 4>(a, maps, st);
  return a.team == 1 ? launch<D, E4M3, 1, 1>(a, maps, st) : launch<D, E4M3, 1, 4>(a, maps, st);
}

}  // namespace

cudaError_t launch_gqa_decode(const GqaDecodeArgs& a, cudaStream_t st) {
  PoolMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (a.kv != nullptr && a.num_pages > 0) {
    cudaError_t e = pool_map(a, kHalf / 128, &maps.unit);
    if (e == cudaSuccess) e = pool_map(a, kHalf / 4 / 128, &maps.piece);
    if (e != cudaSuccess) return e;
  }
  const bool e4m3 = a.cache_dtype == QKVP_CACHE_E4M3;
  switch (a.dim) {
    case 64: return e4m3 ? launch_dim<64, true>(a, maps, st) : launch_dim<64, false>(a, maps, st);
    case 128: return e4m3 ? launch_dim<128, true>(a, maps, st) : launch_dim<128, false>(a, maps, st);
    default: return e4m3 ? launch_dim<256, true>(a, maps, st) : launch_dim<256, false>(a, maps, st);
  }
}

}  // namespace qkvp
