// Attention of drafted tokens over a paged 8-bit cache of K and V heads, one scale per (page, K or V, head), on the
// 5th-generation tensor cores.
//
// Row (i, a) is drafted token i of a request and query head a; with the KV head's codes kc, vc and block scales sk, sv,
// over the tokens t that i sees (cached ones, and drafted ones of its path):
//   z_t = sm_scale * sk (q . kc_t),  out = sum_t softmax(z)_t sv vc_t,  lse = log sum_t exp z_t.
// A page's 64 tokens of one KV head are 128 D bytes and 256 D T G operations (T drafted tokens, G query heads a KV head):
// reading bounds it up to T G ~ 140 rows, the matrix products above.
//
// Work. A (request, KV head) has T G rows, cut into blocks of 128 (one tile) or 256 (two tiles), and a worker (a CTA) walks
// segments, each a run of the pages that a block sees. Two CTAs of one tile share an SM, so that one's start and end
// hide behind the other; two tiles share a page's conversion and take turns on the tensor cores.
//
// Roles, per CTA:
//   softmax warps (4 a tile, one row a thread): at a segment's start the row of Q, to FP16 times a power of two, into tensor
//     memory; per page the row's 64 logits from there, running maximum, P back into their place as FP16; at the
//     segment's end O / l.
//   dequant warps: one thread keeps a ring of raw K and V blocks (64 D bytes each, contiguous in the pool) filled by bulk
//     copies; all turn the codes into FP16, exactly, in 128-byte-swizzled tiles of 64-dim atoms.
//   one thread a tile issues S = Q K^T (M 128, N 64; Q from tensor memory), another O += P V (M 128, N D; P from tensor
//     memory). The same tile layout is K^T's K-major operand and V's MN-major one.
// Q and P from tensor memory leave shared memory the raw bytes, the tiles and one operand's reads.
//
// Softmax. m is the row's largest logit so far, l the sum of 2^(z - m) in FP32. What a page adds to O is p sv code, and
// V's scales may be far apart, so O has a reference r of its own: P = p F, F = sv 2^(m - r + 6), r renewed (and O
// rescaled) only when the largest z + log2 sv of a page passes it by 2^8. P <= 2^14 stays in FP16's normal range down to
// 2^-28 of the largest contribution.
//
// Masks. Only pages that hold drafted tokens or an edge of a row's window are masked by row: 64 bits from the row's mask
// words. V codes that are NaN there count as zero in the product (0 times NaN would reach rows that do not see the token),
// and the rows that do see one are found at the segment's end.
#include <cstdint>

#include "decode_common.cuh"
#include "qkvp_device.cuh"
#include "qkvp_internal.h"
#include "tc_ptx.cuh"

namespace qkvp {
namespace {

using kern::Sync;
using kern::sts128_relaxed;

constexpr float kSlack = 8.0f;     // how far (log2) a contribution may pass the reference
constexpr float kLift = 6.0f;      // P is held as 2^(... + kLift)
constexpr float kNoRef = -1e30f;   // reference before the first page that contributes

template <int D, int NT>
struct Cfg {
  static constexpr int kCtas = tree_ctas_per_sm(D, NT);
  static constexpr int kDqWarps = D == 256 ? 8 : 4;
  static constexpr int kDQ = 32 * kDqWarps;
  static constexpr int kSmWarps = 4 * NT;
  static constexpr int kQkWarp = kSmWarps + kDqWarps, kPvWarp = kQkWarp + NT;
  static constexpr int kThreads = 32 * (kPvWarp + NT);
  static constexpr int kAtoms = D / 64;
  static constexpr uint32_t kRaw = kPage * D;            // bytes of a raw K or V block
  static constexpr uint32_t kAtom = kPage * 128;         // 64 tokens x 64 FP16
  static constexpr uint32_t kTile = kAtoms * kAtom;      // a converted block
  static constexpr int kKS = D == 256 ? 2 : D == 128 && NT == 1 ? 2 : 3, kVS = kKS;
  static constexpr int kRS = D == 256 || (D == 128 && NT == 1) ? 5 : 8;   // raw blocks in the ring
  static constexpr int kSB = D == 128 ? 1 : 2;           // logit buffers of a tile
  // tensor memory columns
  static constexpr uint32_t TM_S = NT * D, TM_Q = TM_S + NT * kSB * 64, kCols = TM_Q + NT * D / 2 <= 256 ? 256 : 512;
  static_assert(TM_Q + NT * D / 2 <= 512 && kCols * kCtas <= 512, "tensor memory");
  // shared memory
  static constexpr uint32_t OFF_K = 0, OFF_V = OFF_K + kKS * kTile, OFF_RAW = OFF_V + kVS * kTile, OFF_BAR = OFF_RAW + kRS * kRaw;
  // barriers
  static constexpr uint32_t B_RAW_FULL = 0, B_RAW_EMPTY = B_RAW_FULL + kRS, B_K_FULL = B_RAW_EMPTY + kRS, B_K_EMPTY = B_K_FULL + kKS,
                            B_V_FULL = B_K_EMPTY + kKS, B_V_EMPTY = B_V_FULL + kVS, B_S_FULL = B_V_EMPTY + kVS,
                            B_P_FULL = B_S_FULL + NT * kSB, B_O_DONE = B_P_FULL + NT * kSB, B_Q_FULL = B_O_DONE + NT * kSB,
                            B_FINAL = B_Q_FULL + NT, kBars = B_FINAL + 1;
  static constexpr uint32_t OFF_TSLOT = OFF_BAR + 8 * kBars, OFF_ABORT = OFF_TSLOT + 4, OFF_NAN = OFF_ABORT + 4;
  static constexpr uint32_t kSmem = OFF_NAN + 8 + 1024;  // slack to align the base to 1024 bytes
  static_assert((kSmem + 1024) * kCtas <= 233472, "shared memory of an SM");
};

__device__ __forceinline__ TreeSegment load_segment(const TreeSegment* p) {
  TreeSegment s;
  const int4* src = reinterpret_cast<const int4*>(p);
  int4* dst = reinterpret_cast<int4*>(&s);
#pragma unroll
  for (int i = 0; i < 3; ++i) dst[i] = src[i];
  return s;
}

// Walks a worker's pages, segment by segment; every segment has a page at least.
struct Walk {
  int si, se, j;
  TreeSegment s;
  __device__ Walk(const TreeArgs& a, int b, int e) : si(b), se(e), j(0) {
    if (si < se) s = load_segment(a.segs + si);
  }
  __device__ bool done() const { return si >= se; }
  __device__ void next(const TreeArgs& a) {
    if (++j < s.num_pages) return;
    j = 0;
    if (++si < se) s = load_segment(a.segs + si);
  }
  __device__ int local() const {
    const int v = s.page_begin + j;
    return v < s.sink_pages ? v : s.win_page + (v - s.sink_pages);
  }
  __device__ int32_t page(const TreeArgs& a) const { return a.kv_indices[s.page0 + local()]; }
};

__device__ __forceinline__ bool in_pool(const TreeArgs& a, int32_t page) { return page >= 0 && page < a.num_pages; }

// Whether the rows of a segment may see different tokens of the page that starts at position p0.
__device__ __forceinline__ bool by_row(const TreeArgs& a, const TreeSegment& s, int p0) {
  if (p0 + kPage > s.cached) return true;
  // rows' windows begin at cached - window + (0 .. drafted); below that only the sinks are visible
  if (a.window == 0 || p0 >= s.cached - a.window + (s.len - s.cached)) return false;
  return p0 + kPage > a.sinks;
}

__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// What one row sees.
struct RowMask {
  const uint32_t* words;   // its mask, or null: the first `chain` drafted tokens
  int chain, win_begin;
  __device__ void init(const TreeArgs& a, const TreeSegment& s, int t) {
    const int drafted = s.len - s.cached;
    words = a.mask ? a.mask + static_cast<int64_t>(s.tok0 + t) * a.words : nullptr;
    chain = t + 1;
    win_begin = 0;
    if (a.window > 0) {
      int n = chain;
      if (words) {
        n = 0;
        for (int w = 0; 32 * w < drafted && w < a.words; ++w) n += __popcll(words[w] & low_bits(drafted - 32 * w));
      }
      win_begin = s.cached + n - a.window;
    }
  }
  __device__ uint64_t word(const TreeArgs& a, int w) const { return w >= 0 && w < a.words ? words[w] : 0u; }
  // the tokens of the page from position p0 on, one bit each
  __device__ uint64_t page(const TreeArgs& a, const TreeSegment& s, int p0) const {
    uint64_t old = low_bits(s.cached - p0);
    if (a.window > 0) old &= ~low_bits(win_begin - p0) | low_bits(a.sinks - p0);
    if (p0 + kPage <= s.cached) return old;
    const int drafted = s.len - s.cached, j0 = p0 - s.cached;     // j0 > -64
    uint64_t tree;
    if (!words) {
      tree = j0 >= 0 ? low_bits(chain - j0) : low_bits(chain) << -j0;
    } else if (j0 < 0) {
      tree = (word(a, 0) | word(a, 1) << 32) & low_bits(drafted);
      tree <<= -j0;
    } else {
      const int w = j0 >> 5, sh = j0 & 31;
      const uint64_t lo = word(a, w) | word(a, w + 1) << 32;
      tree = sh ? lo >> sh | word(a, w + 2) << (64 - sh) : lo;
      tree &= low_bits(drafted - j0);
    }
    return old | tree;
  }
};

template <bool E4M3>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  } else {
    // the biased byte under the exponent of 1024 is 1024 + 128 + c; the subtraction is exact
    const uint32_t b = w ^ 0x80808080u;
    const uint32_t l = __byte_perm(b, 0x64646464u, 0x4140), h = __byte_perm(b, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(l), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(h), "r"(0x64806480u));
  }
}

// The E4M3 NaN codes (0x7F, 0xFF) of a word as a mask of their bytes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  const uint32_t x = (w & 0x7F7F7F7Fu) + 0x01010101u;      // bit 7 of a byte is set where its low bits were all ones
  return (x & 0x80808080u) >> 7;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Raw blocks in, FP16 tiles out. Block e of a worker is page e / 2's K (e even) or V.
template <int D, int NT, bool E4M3>
__device__ void role_dequant(const TreeArgs& a, const Sync& sy, int seg_b, int seg_e, int t, uint32_t base, volatile int* nan_seen) {
  using C = Cfg<D, NT>;
  constexpr int kItems = C::kRaw / 16 / C::kDQ;            // 16 codes each
  static_assert(kItems * C::kDQ * 16 == C::kRaw, "every thread the same number of items");
  constexpr int kBlockRow = kPage * D;
  Walk cur(a, seg_b, seg_e);
  if (cur.done()) return;
  // thread 0 loads kRS - 1 blocks ahead of the conversion; its page id is read a page before it is needed
  Walk ld = cur;
  int32_t ld_page = t == 0 ? ld.page(a) : 0;
  int loaded = 0;                                          // blocks issued (thread 0)
  const uint32_t raw = base + C::OFF_RAW;
  auto issue = [&]() {
    if (ld.done()) return true;
    const int slot = loaded % C::kRS;
    if (loaded >= C::kRS && !sy.wait(C::B_RAW_EMPTY + slot, (loaded / C::kRS - 1) & 1, false, 1)) return false;
    const bool v = loaded & 1;
    // of a request's last page only the tokens that it has
    const int p0 = ld.local() * kPage;
    const uint32_t bytes = in_pool(a, ld_page) ? min(kPage, ld.s.len - p0) * D : 0;
    const uint32_t bar = sy.bar(C::B_RAW_FULL + slot);
    if (bytes) {
      tc::mbar_arrive_expect_tx(bar, bytes);
      const int64_t block = (static_cast<int64_t>(ld_page) * 2 + (v ? 1 : 0)) * a.kv_heads + ld.s.kv_head;
      tc::bulk_load(raw + slot * C::kRaw, a.kv + block * kBlockRow, bytes, bar);
    } else {
      tc::mbar_arrive(bar);
    }
    if (v) {
      ld.next(a);
      if (!ld.done()) ld_page = ld.page(a);
    }
    ++loaded;
    return true;
  };
  bool ok = true;
  if (t == 0)
    for (int i = 0; i < C::kRS - 1 && ok; ++i) ok = issue();
  int32_t page = cur.page(a);
  int e = 0;
  for (int g = 0; !cur.done() && ok; ++g) {
    Walk nx = cur;
    nx.next(a);
    const int32_t npage = nx.done() ? 0 : nx.page(a);
    const int p0 = cur.local() * kPage;
    const int valid = in_pool(a, page) ? min(kPage, cur.s.len - p0) : 0;
    const bool masked = E4M3 && by_row(a, cur.s, p0);
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind, ++e) {
      if (t == 0 && !issue()) { ok = false; break; }
      const int slot = e % C::kRS;
      if (!sy.wait(C::B_RAW_FULL + slot, (e / C::kRS) & 1, false, 1)) { ok = false; break; }
      uint4 w[kItems];
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int q = t + C::kDQ * i;
        w[i] = q / (D / 16) < valid ? lds128(raw + slot * C::kRaw + 16 * q) : make_uint4(0, 0, 0, 0);
      }
      tc::mbar_arrive(sy.bar(C::B_RAW_EMPTY + slot));
      if (kind == 1 && masked) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          uint32_t* x = reinterpret_cast<uint32_t*>(&w[i]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t bad = nan_bytes(x[k]);
            if (bad) {
              x[k] &= ~(bad * 0xFFu);
              *nan_seen = 1;
            }
          }
        }
      }
      const int slots = kind == 0 ? C::kKS : C::kVS, s = g % slots;
      const uint32_t full = kind == 0 ? C::B_K_FULL : C::B_V_FULL, empty = kind == 0 ? C::B_K_EMPTY : C::B_V_EMPTY;
      if (g >= slots && !sy.wait(empty + s, (g / slots - 1) & 1, false, 1)) { ok = false; break; }
      const uint32_t tile = base + (kind == 0 ? C::OFF_K : C::OFF_V) + s * C::kTile;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int q = t + C::kDQ * i, row = q / (D / 16), col = q % (D / 16), atom = col / 4, chunk = 2 * (col % 4);
        uint32_t o[8];
        codes_to_f16<E4M3>(w[i].x, o[0], o[1]);
        codes_to_f16<E4M3>(w[i].y, o[2], o[3]);
        codes_to_f16<E4M3>(w[i].z, o[4], o[5]);
        codes_to_f16<E4M3>(w[i].w, o[6], o[7]);
        // the lanes of an odd atom write their second half first: eight lanes, eight bank groups
        const int odd = D > 64 ? atom & 1 : 0;
        const uint32_t at = tile + atom * C::kAtom;
        const uint4 h0 = make_uint4(o[0], o[1], o[2], o[3]), h1 = make_uint4(o[4], o[5], o[6], o[7]);
        sts128_relaxed(at + tc::sw128_offset(row, chunk + odd), odd ? h1 : h0);
        sts128_relaxed(at + tc::sw128_offset(row, chunk + 1 - odd), odd ? h0 : h1);
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(sy.bar(full + s));
    }
    cur = nx;
    page = npage;
  }
  // after a timeout: the copies in flight land before the CTA may end
  if (t == 0 && !ok)
    for (; e < loaded; ++e) tc::mbar_wait(sy.bar(C::B_RAW_FULL + e % C::kRS), (e / C::kRS) & 1);
}

template <int D, int NT>
__device__ void role_qk(const TreeArgs& a, const Sync& sy, int seg_b, int seg_e, int tile, uint32_t base, uint32_t tbase) {
  using C = Cfg<D, NT>;
  constexpr uint32_t kIdesc = tc::idesc_f16(128, kPage, 0, 0);
  const tc::Desc2 kd = tc::split_desc(tc::smem_desc(base + C::OFF_K, 16, 1024, tc::kSwizzle128));
  const uint32_t q = tbase + C::TM_Q + tile * (D / 2);
  int n = 0, segs = 0;                          // pages of this tile, segments of this tile
  Walk w(a, seg_b, seg_e);
  for (int g = 0; !w.done(); ++g) {
    const int slot = g % C::kKS;
    const bool first = w.j == 0, mine = w.s.rows > tile * kTreeTile;
    if (!sy.wait(C::B_K_FULL + slot, (g / C::kKS) & 1, false, 2)) break;
    if (mine) {
      const int b = n % C::kSB;
      // the buffer's last P has been read
      if (n >= C::kSB && !sy.wait(C::B_O_DONE + tile * C::kSB + b, (n / C::kSB - 1) & 1, false, 2)) break;
      if (first && !sy.wait(C::B_Q_FULL + tile, segs++ & 1, false, 2)) break;
      tc::tc_fence_after();
      const uint32_t s = tbase + C::TM_S + (tile * C::kSB + b) * kPage;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t bd = kd.at(slot * C::kTile + (k >> 2) * C::kAtom + 32 * (k & 3));
        if (k == 0) tc::mma_ts_k<false>(s, q, bd, kIdesc);
        else tc::mma_ts_k<true>(s, q + 8 * k, bd, kIdesc);
      }
      tc::mma_commit(sy.bar(C::B_S_FULL + tile * C::kSB + b));
      tc::mma_commit(sy.bar(C::B_K_EMPTY + slot));
      ++n;
    } else {
      tc::mbar_arrive(sy.bar(C::B_K_EMPTY + slot));
    }
    w.next(a);
  }
  tc::mma_commit(sy.bar(C::B_FINAL));
}

template <int D, int NT>
__device__ void role_pv(const TreeArgs& a, const Sync& sy, int seg_b, int seg_e, int tile, uint32_t base, uint32_t tbase) {
  using C = Cfg<D, NT>;
  constexpr uint32_t kIdesc = tc::idesc_f16(128, D, 0, 1);
  const tc::Desc2 vd = tc::split_desc(tc::smem_desc(base + C::OFF_V, C::kAtom, 1024, tc::kSwizzle128));
  const uint32_t o = tbase + tile * D;
  int n = 0;
  Walk w(a, seg_b, seg_e);
  for (int g = 0; !w.done(); ++g) {
    const int slot = g % C::kVS;
    const bool first = w.j == 0, mine = w.s.rows > tile * kTreeTile;
    if (!sy.wait(C::B_V_FULL + slot, (g / C::kVS) & 1, false, 4)) break;
    if (mine) {
      const int b = n % C::kSB;
      if (!sy.wait(C::B_P_FULL + tile * C::kSB + b, (n / C::kSB) & 1, false, 4)) break;
      tc::tc_fence_after();
      const uint32_t p = tbase + C::TM_S + (tile * C::kSB + b) * kPage;
#pragma unroll
      for (int k = 0; k < 4; ++k) {              // 16 tokens each
        const uint64_t bd = vd.at(slot * C::kTile + 2048 * k);
        if (k == 0 && first) tc::mma_ts_k<false>(o, p, bd, kIdesc);
        else tc::mma_ts_k<true>(o, p + 8 * k, bd, kIdesc);
      }
      tc::mma_commit(sy.bar(C::B_O_DONE + tile * C::kSB + b));
      tc::mma_commit(sy.bar(C::B_V_EMPTY + slot));
      ++n;
    } else {
      tc::mbar_arrive(sy.bar(C::B_V_EMPTY + slot));
    }
    w.next(a);
  }
  tc::mma_commit(sy.bar(C::B_FINAL));
}

__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Dims of V whose code is NaN at a token that the row sees, in the pages that are masked by row: the output is NaN there.
template <int D>
__device__ __noinline__ bool sees_nan(const TreeArgs& a, const TreeSegment& s, const RowMask& mask, int dim) {
  for (int j = 0; j < s.num_pages; ++j) {
    const int v = s.page_begin + j, local = v < s.sink_pages ? v : s.win_page + (v - s.sink_pages), p0 = local * kPage;
    if (!by_row(a, s, p0)) continue;
    const int32_t page = a.kv_indices[s.page0 + local];
    if (!in_pool(a, page)) continue;
    const uint8_t* block = a.kv + ((static_cast<int64_t>(page) * 2 + 1) * a.kv_heads + s.kv_head) * (kPage * D);
    for (uint64_t m = mask.page(a, s, p0); m; m &= m - 1)
      if ((block[(__ffsll(m) - 1) * D + dim] & 0x7F) == 0x7F) return true;
  }
  return false;
}

template <int D, int NT, bool E4M3>
__device__ void role_softmax(const TreeArgs& a, const Sync& sy, int seg_b, int seg_e, int tile, int row, uint32_t tbase, volatile int* nan_seen) {
  using C = Cfg<D, NT>;
  const uint32_t tl = tbase + (static_cast<uint32_t>(row & ~31) << 16);   // the warp's quarter of the lanes
  const int group = a.heads / a.kv_heads;
  auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, sy.wait(bar, parity, false, 8)); };
  int n = 0;                                     // pages of this tile so far
  for (int si = seg_b; si < seg_e; ++si) {
    const TreeSegment s = load_segment(a.segs + si);
    const int at = tile * kTreeTile + row;       // row of the block
    if (s.rows <= tile * kTreeTile) continue;
    const bool live = at < s.rows;
    const int t = (s.row0 + at) / group;         // drafted token and query head
    const int64_t head = static_cast<int64_t>(s.tok0 + t) * a.heads + s.kv_head * group + (s.row0 + at) % group;
    auto local = [&](int j) {
      const int v = s.page_begin + j;
      return v < s.sink_pages ? v : s.win_page + (v - s.sink_pages);
    };
    float m = -INFINITY, l = 0.0f, r = kNoRef;
    // the page ids and scales of the pages to come are read ahead of their use
    auto page_id = [&](int j) { return j < s.num_pages ? a.kv_indices[s.page0 + local(j)] : -1; };
    int32_t id = page_id(0), next_id = page_id(1);
    const float* scales = a.kv_scale + s.kv_head;
    auto k_scale = [&](int32_t p) { return in_pool(a, p) ? scales[static_cast<int64_t>(p) * 2 * a.kv_heads] : 0.0f; };
    auto v_scale = [&](int32_t p) { return in_pool(a, p) ? scales[static_cast<int64_t>(p) * 2 * a.kv_heads + a.kv_heads] : 0.0f; };
    float sk = k_scale(id), sv = v_scale(id);
    RowMask mask;
    mask.init(a, s, live ? t : 0);
    // ---- Q: 2^e brings the row's largest |q| to [2^14, 2^15), where FP16 holds 8 bits down to 2^-29 of it ----
    const uint4* src = reinterpret_cast<const uint4*>(a.q + head * D);
    uint32_t top = 0;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      const uint4 v = live ? src[i] : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
    }
    const int e = top == 0 ? 0 : min(126, 14 + 127 - static_cast<int>(top >> 7));
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    const float q_scale = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {         // 32 dims, 16 columns
      uint32_t x[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = live ? src[4 * c + i] : make_uint4(0, 0, 0, 0);
        x[4 * i] = dev::bf16x2_to_f16x2(v.x ^ a.flip, up);
        x[4 * i + 1] = dev::bf16x2_to_f16x2(v.y ^ a.flip, up);
        x[4 * i + 2] = dev::bf16x2_to_f16x2(v.z ^ a.flip, up);
        x[4 * i + 3] = dev::bf16x2_to_f16x2(v.w ^ a.flip, up);
      }
      __syncwarp();
      tc::tmem_st16(tl + C::TM_Q + tile * (D / 2) + 16 * c, x);
    }
    tc::tmem_wait_st();
    tc::tc_fence_before();
    tc::mbar_arrive(sy.bar(C::B_Q_FULL + tile));

    for (int j = 0; j < s.num_pages; ++j, ++n) {
      const int p0 = local(j) * kPage, b = n % C::kSB;
      const bool masked = by_row(a, s, p0) || !in_pool(a, id);
      const float zs = sk * q_scale, vs = sv;
      uint64_t seen = ~0ull;
      if (masked) seen = in_pool(a, id) ? mask.page(a, s, p0) : 0;
      id = next_id;
      next_id = page_id(j + 2);
      sk = k_scale(id);
      sv = v_scale(id);
      if (!wait(C::B_S_FULL + tile * C::kSB + b, (n / C::kSB) & 1)) return;
      tc::tc_fence_after();
      const uint32_t ts = tl + C::TM_S + (tile * C::kSB + b) * kPage;
      uint32_t x0[32], x1[32];
      tc::tmem_ld32(ts, x0);
      tc::tmem_ld32(ts + 32, x1);
      tc::tmem_wait_ld();
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (masked) {
        const uint32_t s0 = static_cast<uint32_t>(seen), s1 = static_cast<uint32_t>(seen >> 32);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (!(s0 >> i & 1)) x0[i] = 0xff800000u;
          if (!(s1 >> i & 1)) x1[i] = 0xff800000u;
        }
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], fmaxf(__uint_as_float(x0[i]), __uint_as_float(x1[i])));
      const float top_s = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      // a scale of 0 makes every visible logit 0, not -inf * 0
      const float z = top_s == -INFINITY ? -INFINITY : top_s * zs;
      const float m_new = fmaxf(m, z);
      const float back = m_new == -INFINITY ? 0.0f : m_new;
      l *= dev::fast_exp2(m - back);
      m = m_new;
      const float c = z + lg2(vs);             // -inf where the page adds nothing to O
      const bool renew = c > r + kSlack;
      if (__any_sync(0xffffffffu, renew && j > 0)) {
        // O of the pages before, once they are all in
        if (!wait(C::B_O_DONE + tile * C::kSB + (n - 1) % C::kSB, ((n - 1) / C::kSB) & 1)) return;
        tc::tc_fence_after();
        const float f = renew ? dev::fast_exp2(r - c) : 1.0f;
#pragma unroll 1
        for (int k = 0; k < D / 16; ++k) {
          uint32_t o[16];
          tc::tmem_ld16(tl + tile * D + 16 * k, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tc::tmem_st16(tl + tile * D + 16 * k, o);
        }
      }
      if (renew) r = c;
      // held below 2^126: where that cuts, a weight is below 2^-70 of the largest
      const float F = fminf(vs * dev::fast_exp2(fminf(back - r + kLift, 126.0f)), 0x1p126f);
      float l0 = 0.0f, l1 = 0.0f;
      uint32_t pk[16];
      // masked places hold -inf: with a scale of 0 their product is NaN, so they are cleared by the mask
      const float neg = zs > 0.0f ? zs : 0.0f;
      auto half = [&](const uint32_t (&x)[32], uint32_t bits, uint32_t dst) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float p0v = dev::fast_exp2(fmaf(__uint_as_float(x[2 * i]), neg, -back));
          float p1v = dev::fast_exp2(fmaf(__uint_as_float(x[2 * i + 1]), neg, -back));
          if (masked) {
            p0v = bits >> (2 * i) & 1 ? p0v : 0.0f;
            p1v = bits >> (2 * i + 1) & 1 ? p1v : 0.0f;
          }
          l0 += p0v;
          l1 += p1v;
          pk[i] = dev::pack_f16x2(p0v * F, p1v * F);
        }
        tc::tmem_st16(dst, pk);
      };
      half(x0, static_cast<uint32_t>(seen), ts);
      half(x1, static_cast<uint32_t>(seen >> 32), ts + 16);
      l += l0 + l1;
      tc::tmem_wait_st();
      tc::tc_fence_before();
      tc::mbar_arrive(sy.bar(C::B_P_FULL + tile * C::kSB + b));
    }
    if (!wait(C::B_O_DONE + tile * C::kSB + (n - 1) % C::kSB, ((n - 1) / C::kSB) & 1)) return;
    tc::tc_fence_after();
    // ---- the segment's end: O 2^(r - 6 - m) / l; nothing visible: 0 and -inf ----
    const bool none = m == -INFINITY && l == 0.0f;      // (l is NaN where every logit is)
    const float lse2 = none ? -INFINITY : m + log2f(l);
    const float f = none || r == kNoRef ? 0.0f : dev::fast_exp2(r - kLift - m) / l;
    const bool nans = E4M3 && *nan_seen != 0 && live;
    const int64_t slot = static_cast<int64_t>(s.partial) * (NT * kTreeTile) + at;
#pragma unroll 1
    for (int k = 0; k < D / 16; ++k) {
      uint32_t o[16];
      tc::tmem_ld16(tl + tile * D + 16 * k, o);
      tc::tmem_wait_ld();
      float y[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = none ? 0.0f : __uint_as_float(o[i]) * f;
      if (nans)
        for (int i = 0; i < 16; ++i)
          if (sees_nan<D>(a, s, mask, 16 * k + i)) y[i] = __uint_as_float(0x7FC00000u);
      if (live) {
        if (s.partial < 0) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + head * D + 16 * k);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            dst[u] = make_uint4(dev::pack_bf16x2(y[8 * u], y[8 * u + 1]), dev::pack_bf16x2(y[8 * u + 2], y[8 * u + 3]),
                                dev::pack_bf16x2(y[8 * u + 4], y[8 * u + 5]), dev::pack_bf16x2(y[8 * u + 6], y[8 * u + 7]));
        } else {
          float4* dst = reinterpret_cast<float4*>(a.part_o + slot * D + 16 * k);
#pragma unroll
          for (int u = 0; u < 4; ++u) dst[u] = make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
        }
      }
      __syncwarp();
    }
    tc::tc_fence_before();
    if (live) {
      if (s.partial >= 0) a.part_lse[slot] = lse2;
      else if (a.lse) a.lse[head] = none ? -INFINITY : lse2 * 0.69314718055994531f;
    }
  }
}

template <int D, int NT, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, Cfg<D, NT>::kCtas) tree_kernel(const TreeArgs a) {
  using C = Cfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = dev::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5;
  Sync sy;
  sy.bars = base + C::OFF_BAR;
  sy.abort = reinterpret_cast<volatile int*>(sbase + C::OFF_ABORT);
  sy.status = a.status;
  volatile int* nan_seen = reinterpret_cast<volatile int*>(sbase + C::OFF_NAN);
  if (tid == 0) {
    for (int i = 0; i < C::kRS; ++i) { tc::mbar_init(sy.bar(C::B_RAW_FULL + i), 1); tc::mbar_init(sy.bar(C::B_RAW_EMPTY + i), C::kDQ); }
    for (int i = 0; i < C::kKS; ++i) { tc::mbar_init(sy.bar(C::B_K_FULL + i), C::kDQ); tc::mbar_init(sy.bar(C::B_K_EMPTY + i), NT); }
    for (int i = 0; i < C::kVS; ++i) { tc::mbar_init(sy.bar(C::B_V_FULL + i), C::kDQ); tc::mbar_init(sy.bar(C::B_V_EMPTY + i), NT); }
    for (int i = 0; i < NT * C::kSB; ++i) {
      tc::mbar_init(sy.bar(C::B_S_FULL + i), 1);
      tc::mbar_init(sy.bar(C::B_P_FULL + i), kTreeTile);
      tc::mbar_init(sy.bar(C::B_O_DONE + i), 1);
    }
    for (int i = 0; i < NT; ++i) tc::mbar_init(sy.bar(C::B_Q_FULL + i), kTreeTile);
    tc::mbar_init(sy.bar(C::B_FINAL), 2 * NT);      // one commit per issuing thread
    *sy.abort = 0;
    *nan_seen = 0;
    tc::fence_mbar_init();
  }
  if (warp == C::kQkWarp) {
    tc::tmem_alloc(base + C::OFF_TSLOT, C::kCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(sbase + C::OFF_TSLOT);
  dev::wait_for_previous();
  dev::allow_dependents();
  const int seg_b = a.worker_ptr[blockIdx.x], seg_e = a.worker_ptr[blockIdx.x + 1];

  if (warp < C::kSmWarps) {
    role_softmax<D, NT, E4M3>(a, sy, seg_b, seg_e, warp / 4, tid & 127, tbase, nan_seen);
  } else if (warp < C::kQkWarp) {
    role_dequant<D, NT, E4M3>(a, sy, seg_b, seg_e, tid - 32 * C::kSmWarps, base, nan_seen);
  } else if ((tid & 31) == 0) {
    if (warp < C::kPvWarp) role_qk<D, NT>(a, sy, seg_b, seg_e, warp - C::kQkWarp, base, tbase);
    else role_pv<D, NT>(a, sy, seg_b, seg_e, warp - C::kPvWarp, base, tbase);
    sy.wait(C::B_FINAL, 0, false, 16);              // every product has completed before tensor memory is released
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == C::kQkWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tbase, C::kCols);
  }
}

// Joins the partials of blocks that were cut: WARPS warps of a CTA share a row's partials, each takes every WARPS-th one, and
// their sums are added in order. Grid: (rows of a block / rows of a CTA, joins).
constexpr int kJoinThreads = 256;
template <int D, int WARPS>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeArgs a) {
  constexpr int kRows = kJoinThreads / 32 / WARPS, V = D / 32;
  __shared__ float sums[kJoinThreads / 32][D + 1];
  dev::wait_for_previous();
  dev::allow_dependents();
  const TreeJoin* jp = a.joins + blockIdx.y;
  const int first = jp->first, count = jp->count, rows = jp->rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, member = warp % WARPS;
  const int row = blockIdx.x * kRows + warp / WARPS;
  const int pitch = a.tiles * kTreeTile;
  if (static_cast<int>(blockIdx.x) * kRows >= rows) return;
  const bool live = row < rows;
  const float* lse = a.part_lse + static_cast<int64_t>(first) * pitch + row;
  float m = -INFINITY, total = 0.0f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  if (live) {
    for (int i = lane; i < count; i += 32) m = fmaxf(m, lse[static_cast<int64_t>(i) * pitch]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float back = m == -INFINITY ? 0.0f : m;
#pragma unroll 4
    for (int i = member; i < count; i += WARPS) {
      const float w = dev::fast_exp2(lse[static_cast<int64_t>(i) * pitch] - back);
      const float* src = a.part_o + (static_cast<int64_t>(first + i) * pitch + row) * D + lane * V;
      float x[V];
      if constexpr (V == 2) *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
      else
#pragma unroll
        for (int v = 0; v < V; v += 4) *reinterpret_cast<float4*>(x + v) = *reinterpret_cast<const float4*>(src + v);
      total += w;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(w, x[v], acc[v]);
    }
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) sums[warp][lane * V + v] = acc[v];
    if (lane == 0) sums[warp][D] = total;
    __syncthreads();
    if (member != 0) return;
#pragma unroll 1
    for (int w = 1; w < WARPS; ++w) {
      total += sums[warp + w][D];
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += sums[warp + w][lane * V + v];
    }
  }
  if (!live) return;
  const int group = a.heads / a.kv_heads, at = jp->row0 + row;
  const int64_t head = static_cast<int64_t>(jp->tok0 + at / group) * a.heads + jp->kv_head * group + at % group;
  const float inv = m == -INFINITY ? 0.0f : 1.0f / total;
  uint32_t o[V / 2];
#pragma unroll
  for (int v = 0; v < V; v += 2) o[v / 2] = dev::pack_bf16x2(acc[v] * inv, acc[v + 1] * inv);
  uint16_t* dst = a.out + head * D + lane * V;
  if constexpr (V == 2) *reinterpret_cast<uint32_t*>(dst) = o[0];
  else if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
  else *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  if (lane == 0 && a.lse) a.lse[head] = m == -INFINITY ? -INFINITY : (m + log2f(total)) * 0.69314718055994531f;
}

template <int D, int NT, bool E4M3>
cudaError_t launch_attend(const TreeArgs& a, cudaStream_t s) {
  using C = Cfg<D, NT>;
  const cudaError_t e = cudaFuncSetAttribute(tree_kernel<D, NT, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_overlapped(tree_kernel<D, NT, E4M3>, static_cast<unsigned>(a.num_workers), C::kThreads, C::kSmem, s, a);
}

template <int D>
cudaError_t launch_dim(const TreeArgs& a, cudaStream_t s) {
  const bool e4m3 = a.cache_dtype == QKVP_CACHE_E4M3;
  cudaError_t e;
  if constexpr (D == 256) {
    e = e4m3 ? launch_attend<D, 1, true>(a, s) : launch_attend<D, 1, false>(a, s);
  } else {
    if (a.tiles == 1) e = e4m3 ? launch_attend<D, 1, true>(a, s) : launch_attend<D, 1, false>(a, s);
    else e = e4m3 ? launch_attend<D, 2, true>(a, s) : launch_attend<D, 2, false>(a, s);
  }
  if (e != cudaSuccess || a.num_joins == 0) return e;
  const int rows = a.tiles * kTreeTile;
  const bool wide = a.max_join > 16;
  const int per = kJoinThreads / 32 / (wide ? 8 : 1);
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>((rows + per - 1) / per), static_cast<unsigned>(a.num_joins));
  c.blockDim = dim3(kJoinThreads);
  c.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&c, tree_join_kernel<D, 8>, a) : cudaLaunchKernelEx(&c, tree_join_kernel<D, 1>, a);
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
  switch (a.dim) {
    case 64: return launch_dim<64>(a, s);
    case 128: return launch_dim<128>(a, s);
    case 256: return launch_dim<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qkvp
