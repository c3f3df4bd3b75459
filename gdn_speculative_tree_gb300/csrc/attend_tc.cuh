// attend_tc.cuh -- what the tensor-core kernels of treewy_attend share: e4m3
// operands and their terms, the plan of the work, and the loading warp.
//
// The pages are the products' operands as they are: an e4m3 operand costs no
// conversion, and an f32 or bf16 one becomes two 8-bit terms x = hi + lo, whose
// products go into one f32 sum at twice the rate of a product in bf16.
// Queries, and the draft's keys and values, are two e4m3 terms in units of
// their row's power of two: hi has four significant bits, lo the next four and
// a sign, so that a bf16 value is exact but for the smallest of its row.
//
// A tile is 128 tokens.  The weights of the softmax are
//
//   w = 2^(s + log2(the page's value scale) - m + 7.75)
//
// with one reference m per row for the running maximum of s + log2(scale): they
// have the size of what they contribute, however far the pages' scales lie
// apart.  m follows the maximum only when that has grown by more than 2 (the
// output and the sum are then brought down), so weights stay within 2^8.75 =
// 431, e4m3's 448.  Their hi is e4m3 (four significant bits, steps of 2^-9 below
// 2^-6) and lo e5m2 (three, down to 2^-16): a weight is off by 2^-8 of itself or by
// 2^-14, which is 2^-21 of a row's largest (2^-17 where attend_tc_kernel leaves
// room above it), and a smaller one than that by 2^-3 of itself or 2^-17.  So
// tokens beside one that has most of the weight are about as exact as bf16 would
// have them.  (hi in e5m2 and lo in e4m3 ends at 2^-10, with weights of up to 2^11:
// 2^-16 of the largest with the headroom of 2^5 that brings the output down least.)
//
// Work: the items (request, key head, 128 rows at most) are runs of tiles, the
// draft's own keys first; all runs in a row are cut into equal pieces, one for
// each CTA, and an item that lies in several pieces is joined by
// attend_join_kernel.  Many items of several row tiles each go to a CTA apiece
// instead, the row tiles of one context side by side, so that L2 serves it to
// all of them.
#pragma once
#include "cache_device.cuh"
#include "treewy_internal.h"

namespace treewy {

constexpr int kTile = 128;                      // tokens, and rows at most
constexpr int kGroups = kTile / 16;             // the smallest page is 16 tokens
constexpr int kMaxListed = 640;                 // requests whose tiles are put in a row
constexpr int kMaxPieces = 152;                 // CTAs that share the row
constexpr float kGrowth = 1.f, kBias = 7.75f;   // weights are within e4m3: 2^(kGrowth + kBias) <= 448
constexpr float kLeast = 1e-37f;                // of a score's factor: -inf times it stays -inf
constexpr uint32_t kHalf = 128 * 128;           // bytes of 128 rows of 128
constexpr unsigned kFull = 0xffffffffu;

// Drafts of at most kFewRows rows (nodes times query heads of a key head) are
// another kernel's (attend_few.cu): 64 of them, contexts of 1000 to 4000, take
// 94 us there at 16 rows (146 in attend_tc_kernel), 140 at 20 (131), and with
// places for 32 of them it took 162 at 32 rows (133).
constexpr int kFewRows = 16;

struct Consts {
  float ks[kGroups], lv[kGroups], il[kGroups];  // key scale, log2 of the value scale, 1 / value scale
  int bad;
};

// What every request, or the CTA's own one, brings.
struct PlanSmem {
  int scan[32];
  int base[kMaxListed + 1], lo[kMaxListed], len[kMaxListed];  // tiles before it, rows, context
  uint8_t nodes[kMaxListed];
};

template <int S>
struct RingSmem {
  Consts c[S];
  uint64_t kfull[S], kfree[S], vfull[S], vfree[S], cfull[S];
  uint64_t deadline;
  int fail;
};

// The draft of the CTA's item.
struct DraftSmem {
  unsigned long long seen[kMaxNodes];  // the nodes that a node sees
  unsigned long long no_number;        // nodes with a value that is none
  float rowf[kFewRows];                // (few rows) a row's unit of the queries, times the scores' factor
  float ks[kMaxNodes], lv[kMaxNodes], il[kMaxNodes];
  int parent[kMaxNodes];
  int bad_tree;
};

// A bounded wait: every wait of the CTA gives up at the same time.
template <typename Smem>
__device__ __forceinline__ bool wait(Smem& s, uint64_t* bar, uint32_t parity) {
  while (!mbar_try_wait(bar, parity & 1u)) {
    if (*reinterpret_cast<volatile int*>(&s.fail) != 0 || globaltimer_ns() > s.deadline) {
      *reinterpret_cast<volatile int*>(&s.fail) = 1;
      return false;
    }
  }
  return true;
}
// The same for a converged warp, whose lanes agree.
template <typename Smem>
__device__ __forceinline__ bool wait_warp(Smem& s, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(s, bar, parity));
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(bar);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// e4m3 x e4m3 -> f32, A in shared memory or in TMEM (four codes per column).
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D f32, M = 128, e4m3 operands; `a_mn`, `b_mn`: the operand's rows run along the sum.
__device__ __forceinline__ uint32_t idesc_f8(uint32_t N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((N >> 3) << 17) | (8u << 24);
}
constexpr uint32_t kAE5m2 = 1u << 7, kBE5m2 = 1u << 10;  // that operand is e5m2
// V: rows of 128 bytes along the sum, 128-byte swizzle, blocks of 128 columns kHalf bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  uint64_t d = smem_desc_sw128(addr, 1024);
  d &= ~(static_cast<uint64_t>(0x3FFFu) << 16);
  return d | (static_cast<uint64_t>(kHalf >> 4) << 16);
}

// 32 TMEM columns of this thread's lane; complete after tmem_wait32.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_wait32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t at, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::
          "r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
// Eight values of a row of d bf16 at column c (zeros behind d).
// (one by one where rows do not start on 16 bytes)
__device__ __forceinline__ uint4 load_row8_odd(const uint16_t* row, int c, int d) {
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    u[e] = (c + 2 * e < d ? __ldg(row + c + 2 * e) : 0u) | (c + 2 * e + 1 < d ? static_cast<uint32_t>(__ldg(row + c + 2 * e + 1)) << 16 : 0u);
  return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ uint4 load_row8(const uint16_t* row, int c, int d) {
  return c < d ? __ldg(reinterpret_cast<const uint4*>(row + c)) : make_uint4(0, 0, 0, 0);
}

// Two weights as hi + lo: of their f16, hi is the e4m3 nearest to it, and lo the
// upper byte of the rest (e5m2 is f16 without its last eight bits) after rounding.
// `lo` has the bytes in places 1 and 3.
__device__ __forceinline__ void weight_terms(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  uint32_t h, rest;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
  hi = e4m3x2_of_f16x2(h);
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h), "r"(e4m3x2_to_f16x2(hi)));
  lo = rest + 0x00800080u;
}

// The largest of a row's |bf16|, by one warp (lane: eight of them).
__device__ __forceinline__ uint32_t row_largest(const uint4& x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  return __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
}
// What is not finite out of eight values; its places (all bits of a value).
__device__ __forceinline__ void take_out(uint4& x, uint4& bad) {
  auto one = [](uint32_t& u) {
    const uint32_t b = ((u & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((u & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
    u &= ~b;
    return b;
  };
  bad = make_uint4(one(x.x), one(x.y), one(x.z), one(x.w));
}

// A row's terms, by one warp (lane: eight columns, as bf16): codes of
// x 2^(7 - E), 2^E the largest exponent of the row; returns E - 7.  What is not
// finite becomes NaN, or zero where `clear`; `none`: there is some.
__device__ __forceinline__ int row_terms(uint4 x, bool clear, uint2& hi, uint2& lo, bool& none) {
  uint32_t top = row_largest(x);
  uint4 bad = make_uint4(0, 0, 0, 0);
  none = top >= 0x7f80u;
  if (none) {
    take_out(x, bad);
    top = row_largest(x);
  }
  const int E = max(static_cast<int>(top >> 7) - 127, -100);
  const float f = __uint_as_float(static_cast<uint32_t>(127 + 7 - E) << 23);
  uint32_t h[4], l[4];
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t y, rest;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(__uint_as_float(u[e] & 0xffff0000u) * f), "f"(__uint_as_float(u[e] << 16) * f));
    h[e] = e4m3x2_of_f16x2(y);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(y), "r"(e4m3x2_to_f16x2(h[e])));  // exactly; of the code, which has fewer bits where y is small
    l[e] = e4m3x2_of_f16x2(rest);
  }
  hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
  if (none && !clear) {
    auto codes = [](uint32_t a, uint32_t b) {
      return (a & 0x7fu) | ((a >> 8) & 0x7f00u) | ((b & 0x7fu) << 16) | ((b << 8) & 0x7f000000u);
    };
    hi.x |= codes(bad.x, bad.y), hi.y |= codes(bad.z, bad.w);
  }
  return E - 7;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Columns 8 lane .. 8 lane + 7 of row `row` of an operand of 128-byte rows
// (128-byte swizzle), blocks of 128 columns `block` bytes apart.
__device__ __forceinline__ uint2* operand8(unsigned char* tile, int row, int lane, uint32_t block) {
  return reinterpret_cast<uint2*>(tile + (lane >> 4) * block + row * 128 + (((lane & 15) >> 1) ^ (row & 7)) * 16 + (lane & 1) * 8);
}

struct Params {
  treewy_attn a;
  int G, tiles_m;        // query heads per key head; row tiles of the largest draft
  int listed;            // tiles in a row (1) or an item per CTA (0)
  int rows_cap;          // rows of a partial result
  int wide_q, wide_k, wide_v, wide_o;  // rows start on 16 bytes
  float* part_o;         // [kMaxPieces][2][rows_cap][d]
  float* part_lse;       // [kMaxPieces][2][rows_cap]; infinity: refused
  int* record;           // [kMaxPieces][8]: the item that begins in a piece and ends in a later one
  // of attend_split_kernel: terms e4m3 [2][Hkv][T][G][d] (G = 1: keys and values), and their units' exponents
  uint8_t *q_terms, *k_terms, *v_terms;
  int16_t *q_units, *k_units, *v_units;
  int* order;            // requests as they are begun where an item is a CTA's, or NULL: in their own order
};

// The tiles of one item that a CTA takes.
struct Segment {
  int r, h, m, t0, t1, tiles;
  int lo, N, len;
};

__device__ __forceinline__ int tiles_of(int len) { return 1 + len / kTile + (len % kTile != 0); }
__device__ __forceinline__ int row_tiles(const Params& p, int N) { return (N * p.G + kTile - 1) / kTile; }

// Walks a CTA's segments; every role walks them for itself.  kTilesOfRows: a
// context may have several row tiles.
template <bool kTilesOfRows>
struct Walk {
  int u, end, r, item, t;  // tile, the end of the part; request, item (head, row tile) and tile of the next segment
  __device__ __forceinline__ bool next(const Params& p, const PlanSmem& cs, Segment& s) {
    if (u >= end) return false;
    if (p.listed) {
      while (cs.base[r + 1] <= u) ++r, item = 0;
    }
    const int k = p.listed ? r : 0;
    s.r = r, s.lo = cs.lo[k], s.N = cs.nodes[k], s.len = cs.len[k], s.tiles = tiles_of(s.len);
    const int mt = !kTilesOfRows ? 1 : p.listed ? row_tiles(p, s.N) : p.tiles_m;
    s.h = kTilesOfRows ? item / mt : item;
    s.m = item - s.h * mt;
    s.t0 = t, s.t1 = p.listed ? min(s.tiles, t + (end - u)) : s.tiles;
    u += s.t1 - s.t0, ++item, t = 0;
    return true;
  }
};

// Where a CTA's part begins and ends.
template <bool kTilesOfRows>
struct Part {
  Walk<kTilesOfRows> walk;
  int each, more;  // tiles of a piece; how many pieces have one more
};
// The piece that a tile lies in.
template <bool M>
__device__ __forceinline__ int piece_of(const Part<M>& p, int u) {
  const int big = p.more * (p.each + 1);
  return u < big ? u / (p.each + 1) : p.more + (u - big) / p.each;
}

// All threads call it (THREADS of them, after the barriers' set-up); ends with
// a __syncthreads.
template <int THREADS, bool kTilesOfRows, int S>
__device__ __forceinline__ Part<kTilesOfRows> make_plan(const Params& p, PlanSmem& cs, RingSmem<S>& ring) {
  const treewy_attn& a = p.a;
  const treewy_cache& c = a.cache;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  Part<kTilesOfRows> part = {{0, 0, 0, 0, 0}, 1, 0};
  if (p.listed) {
    int carry = 0;
    if (t == 0) cs.base[0] = 0;
#pragma unroll 1
    for (int r0 = 0; r0 < a.R; r0 += THREADS) {
      const int r = r0 + t;
      int v = 0;
      if (r < a.R) {
        const CacheRequest q = cache_request(c, a.node_offset, r, a.T, a.max_nodes, a.max_context);
        if (q.err != 0 && blockIdx.x == 0) atomicOr(a.status + r, q.err);
        cs.lo[r] = q.lo, cs.nodes[r] = static_cast<uint8_t>(q.N), cs.len[r] = q.len;
        v = q.N == 0 ? 0 : c.Hkv * row_tiles(p, q.N) * tiles_of(q.len);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += y;
      }
      if (lane == 31) cs.scan[warp] = v;
      __syncthreads();
      int before = carry;
      const int used = min(THREADS / 32, (a.R - r0 + 31) / 32);
#pragma unroll 1
      for (int w = 0; w < used; ++w) {
        const int x = cs.scan[w];
        if (w < warp) before += x;
        carry += x;
      }
      if (r < a.R) cs.base[r + 1] = before + v;
      __syncthreads();
    }
    const int pieces = min(static_cast<int>(gridDim.x), carry), w = blockIdx.x;  // none of them empty
    if (w < pieces) {
      part.each = carry / pieces, part.more = carry - part.each * pieces;
      part.walk.u = w * part.each + min(w, part.more);
      part.walk.end = part.walk.u + part.each + (w < part.more ? 1 : 0);
      int lo = 0, hi = a.R;  // base[lo] <= u < base[hi]
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cs.base[mid] <= part.walk.u) lo = mid;
        else hi = mid;
      }
      part.walk.r = lo;
      const int in = part.walk.u - cs.base[lo], tiles = tiles_of(cs.len[lo]);
      part.walk.item = in / tiles, part.walk.t = in - part.walk.item * tiles;
    }
    // until it is written: no item begins here and ends elsewhere, and no part is any good
    if (t == 0) p.record[8 * blockIdx.x] = 0;
#pragma unroll 1
    for (int i = t; i < 2 * p.rows_cap; i += THREADS) p.part_lse[2 * static_cast<int64_t>(blockIdx.x) * p.rows_cap + i] = INFINITY;
  } else {
    const int per = c.Hkv * p.tiles_m, item = static_cast<int>(blockIdx.x % per);
    int r = static_cast<int>(blockIdx.x / per);
    if (p.order != nullptr) r = min(max(__ldcg(p.order + r), 0), a.R - 1);
    const CacheRequest q = cache_request(c, a.node_offset, r, a.T, a.max_nodes, a.max_context);
    if (q.err != 0 && item == 0 && t == 0) atomicOr(a.status + r, q.err);
    if (t == 0) cs.lo[0] = q.lo, cs.nodes[0] = static_cast<uint8_t>(q.N), cs.len[0] = q.len;
    part.walk.r = r, part.walk.item = item;
    if (item % p.tiles_m < row_tiles(p, q.N)) part.walk.end = 1;
  }
  if (t == 0) {  // a second, and a hundred times what a tile takes
    ring.fail = 0;
    ring.deadline = globaltimer_ns() + 1000000000ull +
                    100000ull * static_cast<uint64_t>(p.listed ? part.walk.end - part.walk.u : tiles_of(cs.len[0]));
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  return part;
}

// A loading warp: the keys (or the values, with the pages' scales) of every
// tile of the CTA's segments into the ring's stages (K's halves of 128 columns,
// then V's).  Lane i has the i-th of 32 pages of the context, and the next
// 32's, asked for ahead.  begin(g) comes before a segment's tiles, draft(g, gt,
// slot, again) in the place of the draft's; false: a wait of theirs gave up.
// Returns the tiles up to which copies have been started.
template <bool kValues, int NH, bool M, int S, typename Cs, typename Begin, typename Draft>
__device__ __forceinline__ int load_pages(const Params& p, Cs& cs, RingSmem<S>& rs, Walk<M> walk, unsigned char* ring, const CUtensorMap& map,
                                          Begin begin, Draft draft) {
  const treewy_cache& c = p.a.cache;
  constexpr uint32_t kStage = 2 * NH * kHalf;
  const int lane = threadIdx.x & 31, P = c.page_len, per = kTile / P;
  uint64_t* const full = kValues ? rs.vfull : rs.kfull;
  uint64_t* const free = kValues ? rs.vfree : rs.kfree;
  int armed = 0, gt = 0, slot = 0;
  asm volatile("fence.proxy.async.global;" ::: "memory");  // pages and terms that an earlier kernel wrote
  uint32_t again = 1;  // parity of the stage's use before
  Segment g;
#pragma unroll 1
  while (walk.next(p, cs.plan, g)) {
    if (!begin(g)) return armed;
    const int32_t* table = c.page_table + static_cast<int64_t>(g.r) * c.max_pages;
    const int pages = g.len / P + (g.len % P != 0);
    auto entry = [&](int i) { return i < pages ? __ldg(table + i) : -1; };
    auto scale = [&](const float* x, int page) {
      return page >= 0 && page < c.num_pages ? __ldg(x + static_cast<int64_t>(page) * c.Hkv + g.h) : 1.f;
    };
    int src = 32, p0 = (g.t0 - 1) * per;  // the lane that has the tile's first page; its number
    int page = 0, next = 0;
    float ks = 0.f, vs = 1.f, next_ks = 0.f, next_vs = 1.f;
    bool begun = false;
#pragma unroll 1
    for (int j = g.t0; j < g.t1; ++j, ++gt) {
      if (gt >= S && !wait_warp(rs, &free[slot], again)) return armed;
      if (j == 0) {
        if (!draft(g, gt, slot, again)) return armed;
        if constexpr (kValues) {
          if (lane < kGroups) rs.c[slot].ks[lane] = 1.f, rs.c[slot].lv[lane] = rs.c[slot].il[lane] = 0.f;
          if (lane == 0) rs.c[slot].bad = 0;
          warp_arrive(&rs.cfull[slot]);
        }
      } else {
        if (src == 32) {
          page = begun ? next : entry(p0 + lane);
          next = entry(p0 + 32 + lane);
          if constexpr (kValues) {
            if (!begun) next_ks = scale(c.k_scale, page), next_vs = scale(c.v_scale, page);
            ks = next_ks, vs = next_vs;
          }
          begun = true, src = 0;
        }
        const bool mine = lane >= src && lane < src + per && p0 + lane - src < pages;
        const bool in = mine && page >= 0 && page < c.num_pages;
        const unsigned load = __ballot_sync(kFull, in);
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], __popc(load) * P * 128u * NH);
        armed = gt + 1;
        __syncwarp();
        if (in) {
          unsigned char* to = ring + slot * kStage + (kValues ? NH * kHalf : 0) + (lane - src) * P * 128;
#pragma unroll
          for (int x = 0; x < NH; ++x) tma_load_3d(to + x * kHalf, &map, &full[slot], x * 128, 0, page * c.Hkv + g.h);
        }
        __syncwarp();
        if constexpr (kValues) {
          const int at = src + min(lane, kGroups - 1) * 16 / P;
          const float gk = __shfl_sync(kFull, ks, at), gv = __shfl_sync(kFull, vs, at);
          const bool bad = __any_sync(kFull, mine && !in);
          if (lane < kGroups) {
            const float lv = log2f(gv);
            rs.c[slot].ks[lane] = gk;
            rs.c[slot].lv[lane] = lv;
            rs.c[slot].il[lane] = ex2(-lv);
          }
          if (lane == 0) rs.c[slot].bad = bad;
          warp_arrive(&rs.cfull[slot]);
          if (src == per) next_ks = scale(c.k_scale, next), next_vs = scale(c.v_scale, next);
        }
        src += per;
      }
      p0 += per;
      if (++slot == S) slot = 0, again ^= 1;
    }
  }
  return armed;
}

// At the end of a CTA whose waits have given up: what is in flight ends first
// (a draft's tile among the last ones may never be filled).
template <int S>
__device__ __forceinline__ void drain_copies(uint64_t (&full)[S], int armed) {
  for (int i = 0; i < S && i < armed; ++i) mbar_wait_for(&full[(armed - 1 - i) % S], ((armed - 1 - i) / S) & 1, 20000000ull);
}

// Zeros in the 128-byte rows [lo, hi) of `blocks` blocks, by THREADS threads (this one: t).
template <int THREADS>
__device__ __forceinline__ void zero_rows(unsigned char* tile, int blocks, uint32_t block, int lo, int hi, int t) {
#pragma unroll 1
  for (int x = 0; x < blocks; ++x)
#pragma unroll 1
    for (int i = lo * 8 + t; i < hi * 8; i += THREADS) *reinterpret_cast<uint4*>(tile + x * block + i * 16) = make_uint4(0, 0, 0, 0);
}

// What one thread says of a finished segment: the status, and where it is a
// part of an item, what the joining kernel needs.
template <bool M>
__device__ __forceinline__ void report(const Params& p, const Part<M>& part, const Walk<M>& walk, const Segment& g, int rows, bool bad_tree, bool bad) {
  if (bad) atomicOr(p.a.status + g.r, bad_tree ? TREEWY_STATUS_BAD_TREE : TREEWY_STATUS_BAD_PAGE);
  if (g.t0 != 0 || g.t1 == g.tiles) return;
  int4* rec = reinterpret_cast<int4*>(p.record + 8 * blockIdx.x);
  rec[1] = make_int4(g.h, g.m, g.lo, 0);
  rec[0] = make_int4(1, piece_of(part, walk.u + (g.tiles - g.t1) - 1), rows, 0);  // the piece of the item's last tile
}

// By the lanes of a warp.
template <int S>
__device__ __forceinline__ void init_ring(RingSmem<S>& rs, int lane) {
  if (lane >= S) return;
  mbar_init(&rs.kfull[lane], 1);
  mbar_init(&rs.kfree[lane], 1);
  mbar_init(&rs.vfull[lane], 1);
  mbar_init(&rs.vfree[lane], 1);
  mbar_init(&rs.cfull[lane], 1);
}

cudaError_t launch_attend_few(const Params& p, const CUtensorMap& k, const CUtensorMap& v, unsigned grid, cudaStream_t stream);

}  // namespace treewy
