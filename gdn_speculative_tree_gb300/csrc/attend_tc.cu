// attend_tc.cu -- attention over pages of e4m3 keys and values and the draft's
// own ones on the 5th-generation tensor cores (tcgen05, TMEM, TMA), for bf16
// rows and outputs and head sizes that are multiples of 16.
//
// The pages are the products' operands as they are: an e4m3 operand costs no
// conversion, and an f32 or bf16 one becomes two e4m3 terms x = hi + lo, whose
// two products go into one accumulator at twice the rate of bf16's.  hi has
// four significant bits, lo the next four and a sign, so that a bf16 value in
// units of its row's power of two is exact but for the smallest of the row.
//
// A tile is 128 rows, (node, query head) pairs that share a key head, times
// 128 tokens.  TMEM lanes are rows, so that a softmax thread owns half a row:
//
//   S = Q K^T          Q's terms and K in shared memory, S in TMEM, twice
//   w = 2^(s + log2(page's value scale) - m + 5)   two terms, back in TMEM
//   O += w V           V in shared memory as it is stored (rows along the sum)
//
// with one reference m per row for the running maximum of s + log2(scale): the
// weights then have the size of what they contribute, however far the pages'
// scales lie apart.  m follows the maximum only when that has grown by more
// than 2^3 (O and the sum are then brought down): weights stay within 2^8, and
// their terms' last step, 2^-9, within 2^-14 of the row's largest weight.
//
// The draft is a tile of its own, the first of an item (request, key head, 128
// rows): its keys and values, in units of a power of two for each, take two
// tokens of the tile each, one per term, and the ancestors are a mask of bits.
//
//   warps 0-7   queries and draft to e4m3; softmax; outputs
//   warp 8      page table, scales and pages (TMA)
//   warp 9      issues the products: S of the next tile before O of this one
//
// Drafts of at most 32 rows leave most lanes of a tile empty, and the softmax
// of the rest to two warps (TMEM lanes belong to warps).  There (kSmall) Q's
// rows are in shared memory four times, so that every quarter of the lanes has
// all of S: each of the eight warps takes 16 tokens of every row, and the
// weights go to shared memory instead of TMEM, as the product's left operand.
//
// Work: the items' tiles in a row, cut into equal pieces, one for each CTA; an
// item that lies in several pieces is joined by attend_join_kernel.  Many
// items of several row tiles each go to a CTA apiece instead, the row tiles
// of one context side by side, so that L2 serves it to all of them.
#include "cache_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

constexpr int kTile = 128;                      // tokens, and rows
constexpr int kSoftWarps = 8, kLoadWarp = kSoftWarps, kMmaWarp = kLoadWarp + 1;
constexpr int kSoftThreads = 32 * kSoftWarps, kThreads = 32 * (kMmaWarp + 1);
constexpr int kGroups = kTile / 16;             // the smallest page is 16 tokens
constexpr int kMaxListed = 768;                 // requests whose tiles are put in a row
constexpr int kMaxPieces = 152;                 // CTAs that share the row
constexpr float kGrowth = 3.f, kBias = 5.f;     // 2^(kGrowth + kBias) <= 448
constexpr float kLeast = 1e-37f;                // of a score's factor: -inf times it stays -inf
constexpr uint32_t kHalf = 128 * 128;           // bytes of 128 rows of 128
constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;
constexpr unsigned kFull = 0xffffffffu;

// NH: halves of 128 columns of a head; kSmall: at most 32 rows.
template <int NH, bool kSmall>
struct Shape {
  static constexpr uint32_t kWBlock = 32 * 128;                      // a term of the weights of 32 rows
  static constexpr uint32_t kWBytes = kSmall ? 4 * kWBlock : 0;      // two tiles, two terms
  static constexpr uint32_t kQBytes = 2 * NH * kHalf;                // behind them: products read 128 rows of weights
  static constexpr uint32_t kStage = 2 * NH * kHalf;                 // K, then V
  static constexpr int kStages = NH == 2 ? 2 : 5;
  static constexpr uint32_t kBytes = kWBytes + kQBytes + kStages * kStage + 1024;
};

struct Consts {
  float ks[kGroups], lv[kGroups], il[kGroups];  // key scale, log2 of the value scale, 1 / value scale
  int bad;
};

struct AttendSmem {
  Consts c[5];
  uint64_t kfull[5], kfree[5], vfull[5], vfree[5], cfull[5];
  uint64_t sfull[2], pready[2], pvdone[2], qready, drain;
  uint64_t deadline;
  unsigned long long seen[kMaxNodes];  // the nodes that a node sees
  unsigned long long no_number;        // nodes with a value that is none
  float rowf[kTile];            // a row's unit of the queries, times the scores' factor
  float ks[kMaxNodes], lv[kMaxNodes], il[kMaxNodes];  // of the draft
  float top[2][2 * kTile];      // maxima (and sums) of the parts of rows; two sets in turn
  int parent[kMaxNodes];
  int bad_tree;
  uint32_t tmem;
  int fail;
  int scan[kThreads / 32];
  // of every request, or of the CTA's own: tiles before it, rows, context
  int base[kMaxListed + 1], lo[kMaxListed], len[kMaxListed];
  uint8_t nodes[kMaxListed];
};

// A bounded wait: every wait of the CTA gives up at the same time.
__device__ __forceinline__ bool wait(AttendSmem& s, uint64_t* bar, uint32_t parity) {
  while (!mbar_try_wait(bar, parity & 1u)) {
    if (*reinterpret_cast<volatile int*>(&s.fail) != 0 || globaltimer_ns() > s.deadline) {
      *reinterpret_cast<volatile int*>(&s.fail) = 1;
      return false;
    }
  }
  return true;
}
// The same for a converged warp, whose lanes agree.
__device__ __forceinline__ bool wait_warp(AttendSmem& s, uint64_t* bar, uint32_t parity) {
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
__device__ __forceinline__ uint32_t idesc_f8(uint32_t N, bool b_mn) {  // A, B e4m3 (0), D f32, M = 128
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((N >> 3) << 17) | (8u << 24);
}
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
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
// Eight values of a row of d bf16 at column c (zeros behind d).
__device__ __forceinline__ uint4 load_row8(const uint16_t* row, int c, int d, bool wide) {
  if (wide) return c < d ? __ldg(reinterpret_cast<const uint4*>(row + c)) : make_uint4(0, 0, 0, 0);
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    u[e] = (c + 2 * e < d ? __ldg(row + c + 2 * e) : 0u) | (c + 2 * e + 1 < d ? static_cast<uint32_t>(__ldg(row + c + 2 * e + 1)) << 16 : 0u);
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Two values in f16 as hi + lo: hi the four leading bits, lo the next.
__device__ __forceinline__ void split_f16x2(uint32_t h, uint32_t& hi, uint32_t& lo) {
  const uint32_t top = (h + 0x00400040u) & 0xff80ff80u;  // half a unit of the fourth bit up, the rest off
  uint32_t rest;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(h), "r"(top));
  hi = e4m3x2_of_f16x2(top);
  lo = e4m3x2_of_f16x2(rest);
}

// Two weights as hi + lo: f16 first, of which hi has the four leading bits and
// lo the rest, rounded (2^-8 of the weight in all, 2^-9 where hi leaves e4m3's
// normal range).
__device__ __forceinline__ void weight_terms(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
  split_f16x2(h, hi, lo);
}

// A row's terms, by one warp (lane: eight columns, as bf16): codes of
// x 2^(7 - E), 2^E the largest exponent of the row, and the unit 2^(E - 7).
// What is not finite becomes NaN, or zero where `clear`; `none`: there is some.
__device__ __forceinline__ float row_terms(uint4 x, bool clear, uint2& hi, uint2& lo, bool& none) {
  uint32_t u[4] = {x.x, x.y, x.z, x.w};
  auto largest = [&] {
    const uint32_t m = __vmaxu2(__vmaxu2(u[0] & 0x7fff7fffu, u[1] & 0x7fff7fffu), __vmaxu2(u[2] & 0x7fff7fffu, u[3] & 0x7fff7fffu));
    return __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
  };
  uint32_t top = largest(), bad[4] = {0, 0, 0, 0};
  none = top >= 0x7f80u;
  if (none) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bad[e] = ((u[e] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((u[e] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
      u[e] &= ~bad[e];
    }
    top = largest();
  }
  const int E = max(static_cast<int>(top >> 7) - 127, -100);
  const float f = __uint_as_float(static_cast<uint32_t>(127 + 7 - E) << 23);
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(__uint_as_float(u[e] & 0xffff0000u) * f), "f"(__uint_as_float(u[e] << 16) * f));
    split_f16x2(y, h[e], l[e]);
    if (!clear) h[e] |= (bad[e] & 0x7fu) | ((bad[e] >> 8) & 0x7f00u);
  }
  hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
  return __uint_as_float(static_cast<uint32_t>(127 - 7 + E) << 23);
}

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
  int wide_q, wide_k, wide_v, wide_o;
  float* part_o;         // [kMaxPieces][2][rows_cap][d]
  float* part_lse;       // [kMaxPieces][2][rows_cap]
  int* record;           // [kMaxPieces][8]: the item that begins in a piece and ends in a later one
  int* part_bad;         // [kMaxPieces][2]
};

// The tiles of one item that a CTA takes.
struct Segment {
  int r, h, m, t0, t1, tiles;
  int lo, N, len;
};

__device__ __forceinline__ int tiles_of(int len) { return 1 + (len + kTile - 1) / kTile; }
__device__ __forceinline__ int row_tiles(const Params& p, int N) { return (N * p.G + kTile - 1) / kTile; }

// Walks a CTA's segments; every role walks them for itself.
struct Walk {
  int u, end, r;
  __device__ bool next(const Params& p, const AttendSmem& cs, Segment& s) {
    if (u >= end) return false;
    int k = 0;
    if (p.listed) {
      while (cs.base[r + 1] <= u) ++r;
      k = s.r = r;
    } else {
      s.r = static_cast<int>(blockIdx.x / (p.a.cache.Hkv * p.tiles_m));
    }
    s.lo = cs.lo[k], s.N = cs.nodes[k], s.len = cs.len[k], s.tiles = tiles_of(s.len);
    if (p.listed) {
      const int in = u - cs.base[r], item = in / s.tiles, mt = row_tiles(p, s.N);
      s.h = item / mt, s.m = item % mt, s.t0 = in % s.tiles, s.t1 = min(s.tiles, s.t0 + (end - u));
    } else {
      const int item = static_cast<int>(blockIdx.x % (p.a.cache.Hkv * p.tiles_m));
      s.h = item / p.tiles_m, s.m = item % p.tiles_m, s.t0 = 0, s.t1 = s.tiles;
    }
    u += s.t1 - s.t0;
    return true;
  }
};

template <int NH, bool kSmall>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using Sh = Shape<NH, kSmall>;
  constexpr int S = Sh::kStages;
  extern __shared__ unsigned char raw_smem[];
  __shared__ AttendSmem cs;
  unsigned char* wts = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  unsigned char* smem = wts + Sh::kWBytes;
  unsigned char* ring = smem + Sh::kQBytes;
  const treewy_attn& a = p.a;
  const treewy_cache& c = a.cache;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, d = c.d, G = p.G;

  // ---- set-up, while the kernel before may still run
  if (t == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&cs.kfull[i], 1);
      mbar_init(&cs.kfree[i], 1);
      mbar_init(&cs.vfull[i], 1);
      mbar_init(&cs.vfree[i], 1);
      mbar_init(&cs.cfull[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&cs.sfull[i], 1);
      mbar_init(&cs.pready[i], kSoftWarps);
      mbar_init(&cs.pvdone[i], 1);
    }
    mbar_init(&cs.qready, 1);
    mbar_init(&cs.drain, 1);
    fence_mbarrier_init();
    cs.fail = 0;
    cs.base[0] = 0;
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&cs.tmem, kTmemCols);
    tmem_relinquish();
  }
  after_previous();

  // ---- this CTA's part
  Walk begin = {0, 1, 0};
  int total = 1, pieces = 1;
  bool none_here = false;
  if (p.listed) {
    int carry = 0;
    for (int r0 = 0; r0 < a.R; r0 += kThreads) {
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
      for (int w = 0; w < kThreads / 32; ++w) {
        const int x = cs.scan[w];
        if (w < warp) before += x;
        carry += x;
      }
      if (r < a.R) cs.base[r + 1] = before + v;
      __syncthreads();
    }
    total = carry;
    pieces = min(static_cast<int>(gridDim.x), total);  // none of them empty
    none_here = static_cast<int>(blockIdx.x) >= pieces;
    if (!none_here) {
      begin.u = static_cast<int>(static_cast<int64_t>(blockIdx.x) * total / pieces);
      begin.end = static_cast<int>(static_cast<int64_t>(blockIdx.x + 1) * total / pieces);
      int lo = 0, hi = a.R;  // base[lo] <= u < base[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cs.base[mid] <= begin.u) lo = mid;
        else hi = mid;
      }
      begin.r = lo;
    }
    if (t == 0) {
      p.record[8 * blockIdx.x] = 0;
      p.part_bad[2 * blockIdx.x] = p.part_bad[2 * blockIdx.x + 1] = 1;
    }
  } else {
    const int per = c.Hkv * p.tiles_m, r = static_cast<int>(blockIdx.x / per), item = static_cast<int>(blockIdx.x % per);
    const CacheRequest q = cache_request(c, a.node_offset, r, a.T, a.max_nodes, a.max_context);
    if (q.err != 0 && item == 0 && t == 0) atomicOr(a.status + r, q.err);
    if (t == 0) cs.lo[0] = q.lo, cs.nodes[0] = static_cast<uint8_t>(q.N), cs.len[0] = q.len;
    none_here = item % p.tiles_m >= row_tiles(p, q.N);
  }
  if (t == 0) {  // a second, and a hundred times what a tile takes
    cs.deadline = globaltimer_ns() + 1000000000ull +
                  100000ull * static_cast<uint64_t>(p.listed ? begin.end - begin.u : 1 + a.max_context / kTile);
  }
  if (none_here) begin.end = begin.u;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = cs.tmem;
  const float factor = a.scale * 1.4426950408889634f;  // scores in powers of two

  Walk walk = begin;
  Segment g;
  int armed_k = 0, armed_v = 0;  // tiles up to which the loading warp has started copies
  int gt = 0;  // tiles so far

  if (warp == kLoadWarp) {
    // ---- pages: lane i has the i-th of 32 pages of the context
    const int P = c.page_len, per = kTile / P;
    bool ok = true;
    while (ok && walk.next(p, cs, g)) {
      const int32_t* table = c.page_table + static_cast<int64_t>(g.r) * c.max_pages;
      const int pages = (g.len + P - 1) / P;
      auto entry = [&](int i) { return i < pages ? __ldg(table + i) : -1; };
      auto scale = [&](const float* x, int page) {
        return page >= 0 && page < c.num_pages ? __ldg(x + static_cast<int64_t>(page) * c.Hkv + g.h) : 1.f;
      };
      int first = -1;  // page index of lane 0's
      int page = 0, next = 0;
      float ks = 0.f, vs = 1.f, next_ks = 0.f, next_vs = 1.f;
      for (int j = g.t0; j < g.t1; ++j, ++gt) {
        const int slot = gt % S;
        const uint32_t again = (gt / S + 1) & 1;
        unsigned char* stage = ring + slot * Sh::kStage;
        if (j == 0) {  // the draft's tile: the softmax warps fill it
          if (gt >= S) ok = wait_warp(cs, &cs.kfree[slot], again) && wait_warp(cs, &cs.vfree[slot], again);
          if (!ok) break;
          if (lane == 0) cs.c[slot].bad = 0;
          warp_arrive(&cs.cfull[slot]);
          continue;
        }
        const int p0 = (j - 1) * per;  // the tile's first page
        if (first < 0) {
          first = p0;
          page = entry(p0 + lane);
          next = entry(p0 + 32 + lane);
          ks = scale(c.k_scale, page), vs = scale(c.v_scale, page);
        } else if (p0 >= first + 32) {  // the next 32, asked for ahead
          first = p0;
          page = next, ks = next_ks, vs = next_vs;
          next = entry(p0 + 32 + lane);
        }
        const int src = p0 - first;  // the lane that has it
        const bool mine = lane >= src && lane < src + per && first + lane < pages;
        const bool in = page >= 0 && page < c.num_pages;
        const unsigned load = __ballot_sync(kFull, mine && in), wanted = __ballot_sync(kFull, mine);
        const uint32_t bytes = __popc(load) * P * 128u * NH;
        const int z = page * c.Hkv + g.h;
        const uint32_t to = (lane - src) * P * 128;
        if (gt >= S) ok = wait_warp(cs, &cs.kfree[slot], again);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&cs.kfull[slot], bytes);
        armed_k = gt + 1;
        __syncwarp();
        if (mine && in) {
#pragma unroll
          for (int x = 0; x < NH; ++x) tma_load_3d(stage + x * kHalf + to, &kmap, &cs.kfull[slot], x * 128, 0, z);
        }
        __syncwarp();
        if (gt >= S) ok = wait_warp(cs, &cs.vfree[slot], again);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&cs.vfull[slot], bytes);
        armed_v = gt + 1;
        __syncwarp();
        if (mine && in) {
#pragma unroll
          for (int x = 0; x < NH; ++x) tma_load_3d(stage + (NH + x) * kHalf + to, &vmap, &cs.vfull[slot], x * 128, 0, z);
        }
        __syncwarp();
        const int at = src + min(lane, kGroups - 1) * 16 / P;
        const float gk = __shfl_sync(kFull, ks, at), gv = __shfl_sync(kFull, vs, at);
        if (lane < kGroups) {
          const float lv = log2f(gv);
          cs.c[slot].ks[lane] = gk;
          cs.c[slot].lv[lane] = lv;
          cs.c[slot].il[lane] = ex2(-lv);
        }
        if (lane == 0) cs.c[slot].bad = load != wanted;
        warp_arrive(&cs.cfull[slot]);
        // the scales of the pages that were asked for with the last 32
        if (src == (per == 32 ? 0 : per)) next_ks = scale(c.k_scale, next), next_vs = scale(c.v_scale, next);
      }
    }
  } else if (warp == kMmaWarp) {
    // ---- products
    const uint32_t id_s = idesc_f8(kTile, false), id_o = idesc_f8(d, true);
    const uint32_t q0 = smem_addr(smem), r0 = smem_addr(ring), w0 = smem_addr(wts);
    int seg = 0;
    bool ok = true;
    while (ok && walk.next(p, cs, g)) {
      ok = wait_warp(cs, &cs.qready, seg & 1);
      ++seg;
      auto scores = [&](int tile) {  // S of the CTA's tile number `tile`
        const int slot = tile % S;
        if (!wait_warp(cs, &cs.kfull[slot], (tile / S) & 1)) return false;
        tc_fence_after_sync();
        if (elect_one()) {
          const uint32_t s = tmem + kColS + (tile & 1) * kTile, k0 = r0 + slot * Sh::kStage;
          uint32_t acc = 0;
#pragma unroll
          for (int x = 0; x < NH; ++x) {
            const int steps = (min(128, d - 128 * x) + 31) / 32;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= steps) continue;
              const uint64_t b = smem_desc_sw128(k0 + x * kHalf + k * 32, 1024);
#pragma unroll
              for (int term = 0; term < 2; ++term) {
                mma_f8(s, smem_desc_sw128(q0 + (term * NH + x) * kHalf + k * 32, 1024), b, id_s, acc);
                acc = 1;
              }
            }
          }
          mma_commit(&cs.sfull[tile & 1]);
          mma_commit(&cs.kfree[slot]);
        }
        __syncwarp();
        return true;
      };
      ok = ok && scores(gt);
      for (int j = g.t0; ok && j < g.t1; ++j, ++gt) {
        if (j + 1 < g.t1) ok = scores(gt + 1);
        const int slot = gt % S;
        ok = ok && wait_warp(cs, &cs.vfull[slot], (gt / S) & 1) && wait_warp(cs, &cs.pready[gt & 1], (gt >> 1) & 1);
        if (!ok) break;
        tc_fence_after_sync();
        const int n = j == 0 ? (kSmall ? (g.N + 7) / 8 * 16 : g.N > 32 ? kTile : kTile / 2) : min(kTile, g.len - (j - 1) * kTile);
        if (elect_one()) {
          const uint32_t w = tmem + kColS + (gt & 1) * kTile, v0 = r0 + slot * Sh::kStage + NH * kHalf;
          uint32_t acc = j != g.t0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (32 * k >= n) continue;
            const uint64_t b = desc_mn(v0 + k * 4096);
#pragma unroll
            for (int term = 0; term < 2; ++term) {
              if constexpr (kSmall)
                mma_f8(tmem + kColO, smem_desc_sw128(w0 + (2 * (gt & 1) + term) * Sh::kWBlock + k * 32, 1024), b, id_o, acc);
              else
                mma_f8_ts(tmem + kColO, w + term * 32 + k * 8, b, id_o, acc);
              acc = 1;
            }
          }
          mma_commit(&cs.vfree[slot]);
          mma_commit(&cs.pvdone[gt & 1]);
        }
        __syncwarp();
      }
    }
  } else {
    // ---- softmax: warps w and w + 4 have lanes 32 (w % 4) ..; a thread has kCols tokens of a row
    constexpr int kCols = kSmall ? 16 : 64, kNodes = kCols / 2;
    const int part = warp & 3, hf = warp >> 2, row = kSmall ? lane : part * 32 + lane;
    const int share = kSmall ? part * 2 + hf : hf, tok0 = share * kCols;  // which part of the row
    const uint32_t lanes = tmem + (static_cast<uint32_t>(part * 32) << 16);
    const int out_cols = (d / 16 + 1) / 2 * 16;  // O's columns of the first half
    const int col0 = hf ? out_cols : 0, col1 = hf ? d : out_cols;
    const bool has_o = !kSmall || part == 0;  // O is in lanes 0-31 there
    auto all_sync = [] { named_bar_sync<1, kSoftThreads>(); };
    auto row_sync = [&] {  // among the warps that share rows
      if constexpr (kSmall) named_bar_sync<1, kSoftThreads>();
      else asm volatile("bar.sync %0, 64;" ::"r"(2 + part) : "memory");
    };
    // `op` over the parts of this thread's row
    auto over_row = [&](int set, float v, auto op) {
      constexpr int kPitch = kSmall ? 32 : kTile;
      cs.top[set][share * kPitch + row] = v;
      row_sync();
#pragma unroll
      for (int i = 0; i < (kSmall ? 8 : 2); ++i) {
        const float y = cs.top[set][i * kPitch + row];
        v = i == 0 ? y : op(v, y);
      }
      return v;
    };
    while (walk.next(p, cs, g)) {
      // queries and tree
      const int row0 = g.m * kTile, rows = min(kTile, g.N * G - row0);
      if (t == 0) cs.bad_tree = 0, cs.no_number = 0;
      all_sync();
      if (t < g.N) {
        const int q = a.parent != nullptr ? __ldg(a.parent + g.lo + t) : t - 1;
        const bool wrong = q < -1 || q >= t;
        if (wrong) cs.bad_tree = 1;
        cs.parent[t] = wrong ? -1 : q;
      }
      constexpr int kBatch = 8;  // rows of a warp that are loaded together
      for (int i0 = warp; i0 < rows; i0 += kSoftWarps * kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int i = i0 + e * kSoftWarps, rr = row0 + i, node = rr / G;
          if (i < rows)
            x[e] = load_row8(static_cast<const uint16_t*>(a.q) + (static_cast<int64_t>(g.lo) + node) * a.q_stride +
                                 static_cast<int64_t>(g.h * G + rr - node * G) * d,
                             8 * lane, d, p.wide_q);
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          const int i = i0 + e * kSoftWarps;
          if (i >= rows) continue;
          uint2 hi, lo;
          bool none;
          const float unit = row_terms(x[e], false, hi, lo, none);
          if (8 * lane < NH * 128) {
#pragma unroll
            for (int copy = 0; copy < (kSmall ? 4 : 1); ++copy) {
              *operand8(smem, 32 * copy + i, lane, kHalf) = hi;
              *operand8(smem + NH * kHalf, 32 * copy + i, lane, kHalf) = lo;
            }
          }
          if (lane == 0) cs.rowf[i] = unit * factor;
        }
      }
      if (g.t0 == 0) {
        wait_warp(cs, &cs.cfull[gt % S], (gt / S) & 1);  // the stage is free
        unsigned char* stage = ring + (gt % S) * Sh::kStage;
#pragma unroll
        for (int value = 0; value < 2; ++value) {
          const uint16_t* from = static_cast<const uint16_t*>(value ? a.v : a.k) +
                                 static_cast<int64_t>(g.lo) * (value ? a.v_stride : a.k_stride) + static_cast<int64_t>(g.h) * d;
          uint4 x[kMaxNodes / kSoftWarps];
#pragma unroll
          for (int e = 0; e < kMaxNodes / kSoftWarps; ++e) {
            const int n = warp + e * kSoftWarps;
            x[e] = make_uint4(0, 0, 0, 0);
            if (n < g.N) x[e] = load_row8(from + n * (value ? a.v_stride : a.k_stride), 8 * lane, d, value ? p.wide_v : p.wide_k);
          }
#pragma unroll
          for (int e = 0; e < kMaxNodes / kSoftWarps; ++e) {
            const int n = warp + e * kSoftWarps, token = n / kNodes * kCols + n % kNodes;
            uint2 hi = make_uint2(0, 0), lo = hi;
            float unit = 1.f;
            bool none = false;
            // a value that is no number would reach the nodes that do not see it: weights of zero times it
            if (n < g.N) unit = row_terms(x[e], value != 0, hi, lo, none);
            if (8 * lane < NH * 128) {
              unsigned char* tile = stage + (value ? NH * kHalf : 0);
              *operand8(tile, token, lane, kHalf) = hi;
              *operand8(tile, token + kNodes, lane, kHalf) = lo;
            }
            if (lane == 0) {
              if (value) {
                if (none) atomicOr(&cs.no_number, 1ull << n);
                const float lv = log2f(unit);
                cs.lv[n] = lv;
                cs.il[n] = ex2(-lv);
              } else {
                cs.ks[n] = unit;
              }
            }
          }
        }
      }
      fence_proxy_async_smem();
      all_sync();
      if (t == 0) {
        arrive(&cs.qready);
        if (g.t0 == 0) {
          arrive(&cs.kfull[gt % S]);
          arrive(&cs.vfull[gt % S]);
        }
      }
      if (t < g.N) {  // the nodes that node t sees
        unsigned long long m = 0;
        for (int q = t; q >= 0; q = cs.parent[q]) m |= 1ull << q;
        cs.seen[t] = m;
      }
      all_sync();

      bool bad = cs.bad_tree != 0;
      const int bad_bit = bad ? TREEWY_STATUS_BAD_TREE : TREEWY_STATUS_BAD_PAGE;
      const bool alive = kSmall || part * 32 < rows;
      const float rowf = row < rows ? cs.rowf[row] : 0.f;
      const int node = min(row0 + row, g.N * G - 1) / G;
      const uint32_t seen = static_cast<uint32_t>(cs.seen[node] >> (kNodes * share));
      float m = -INFINITY, sum = 0.f;
      for (int j = g.t0; j < g.t1; ++j, ++gt) {
        const int slot = gt % S, b = gt & 1;
        const Consts& cc = cs.c[slot];
        // after a wait that gave up a warp still comes by every barrier of threads
        bool ok = wait_warp(cs, &cs.sfull[b], (gt >> 1) & 1) && wait_warp(cs, &cs.cfull[slot], (gt / S) & 1);
        tc_fence_after_sync();
        bad |= cc.bad != 0;
        const int n = j == 0 ? kTile : min(kTile, g.len - (j - 1) * kTile);
        if (n < kTile && ok) ok = wait_warp(cs, &cs.vfull[slot], (gt / S) & 1);
        if (n < kTile && ok) {  // values behind the context: anything, so none
          const int end = (n + 31) & ~31;
          unsigned char* v = ring + slot * Sh::kStage + NH * kHalf;
          for (int i = n * 8 + t; i < end * 8; i += kSoftThreads)
#pragma unroll
            for (int x = 0; x < NH; ++x) *reinterpret_cast<uint4*>(v + x * kHalf + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        if (alive) {
          const uint32_t sc = lanes + kColS + b * kTile;
          uint32_t r[kCols];
          float* s = reinterpret_cast<float*>(r);
          if (ok) {
            if constexpr (kSmall) {
              uint32_t(&r16)[16] = *reinterpret_cast<uint32_t(*)[16]>(r);
              tmem_ld16_async(sc + tok0, r16);
              tmem_wait16(r16);
            } else {
              tmem_ld32(sc + tok0, r);
              tmem_ld32(sc + tok0 + 32, r + 32);
              tmem_wait32(r);
              tmem_wait32(r + 32);
            }
          }
          float top = -INFINITY;
          if (j == 0) {
#pragma unroll
            for (int i = 0; i < kNodes; ++i) {
              const int q = share * kNodes + i;
              const float y = (s[i] + s[kNodes + i]) * (cs.ks[q] * rowf) + cs.lv[q];
              s[i] = (seen >> i) & 1 ? y : -INFINITY;
              top = fmaxf(top, s[i]);
            }
          } else {
            if (n < kTile) {
#pragma unroll
              for (int i = 0; i < kCols; ++i) s[i] = tok0 + i < n ? s[i] : -INFINITY;
            }
#pragma unroll
            for (int q = 0; q < kCols / 16; ++q) {
              float x = s[16 * q];
#pragma unroll
              for (int i = 1; i < 16; ++i) x = fmaxf(x, s[16 * q + i]);
              const int at = share * (kCols / 16) + q;
              top = fmaxf(top, fmaf(x, fmaxf(cc.ks[at] * rowf, kLeast), cc.lv[at]));
            }
          }
          top = over_row(b, top, [](float x, float y) { return fmaxf(x, y); });
          if (j == g.t0) {
            m = top;
          } else {
            const bool grown = top > m + kGrowth;
            if (__any_sync(kFull, grown)) {
              const float down = grown ? ex2(m - top) : 1.f;
              if (grown) m = top;
              sum *= down;
              if (has_o) {
                wait_warp(cs, &cs.pvdone[(gt - 1) & 1], ((gt - 1) >> 1) & 1);
                tc_fence_after_sync();
                for (int x = col0; x < col1; x += 16) {
                  uint32_t o[16];
                  tmem_ld16_async(lanes + kColO + x, o);
                  tmem_wait16(o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * down);
                  tmem_st16(lanes + kColO + x, o);
                }
                tmem_wait_st();
              }
            }
          }
          const float off = kBias - m;
          uint32_t hi[kCols / 4], lo[kCols / 4];
          if (j == 0) {
#pragma unroll
            for (int i = 0; i < kNodes; ++i) {
              s[i] = ex2(s[i] + off);
              sum = fmaf(s[i], cs.il[share * kNodes + i], sum);
            }
#pragma unroll
            for (int i = 0; i < kNodes / 4; ++i) {
              uint32_t h0, l0, h1, l1;
              weight_terms(s[4 * i], s[4 * i + 1], h0, l0);
              weight_terms(s[4 * i + 2], s[4 * i + 3], h1, l1);
              hi[i] = hi[i + kNodes / 4] = h0 | (h1 << 16);  // the value's two terms have one weight
              lo[i] = lo[i + kNodes / 4] = l0 | (l1 << 16);
            }
          } else {
#pragma unroll
            for (int q = 0; q < kCols / 16; ++q) {
              const int at = share * (kCols / 16) + q;
              const float f = fmaxf(cc.ks[at] * rowf, kLeast), e = cc.lv[at] + off;
              float part_sum = 0.f;
#pragma unroll
              for (int i = 16 * q; i < 16 * q + 16; ++i) {
                s[i] = ex2(fmaf(s[i], f, e));
                part_sum += s[i];
              }
              sum = fmaf(part_sum, cc.il[at], sum);
            }
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i) {
              uint32_t h0, l0, h1, l1;
              weight_terms(s[4 * i], s[4 * i + 1], h0, l0);
              weight_terms(s[4 * i + 2], s[4 * i + 3], h1, l1);
              hi[i] = h0 | (h1 << 16);
              lo[i] = l0 | (l1 << 16);
            }
          }
          if constexpr (kSmall) {
            unsigned char* w = wts + 2 * b * Sh::kWBlock + row * 128 + ((share ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(w) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(w + Sh::kWBlock) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            fence_proxy_async_smem();
          } else {
            tmem_st16(sc + hf * 16, hi);
            tmem_st16(sc + 32 + hf * 16, lo);
            tmem_wait_st();
          }
          tc_fence_before_sync();
        }
        warp_arrive(&cs.pready[b]);
      }

      // ---- outputs
      const bool whole = g.t0 == 0 && g.t1 == g.tiles;
      const bool ok = wait_warp(cs, &cs.pvdone[(gt - 1) & 1], ((gt - 1) >> 1) & 1);
      tc_fence_after_sync();
      // not the set of the last tile, which another warp may still read
      if (alive) sum = over_row(gt & 1, sum, [](float x, float y) { return x + y; });
      const float inv = 1.f / sum;
      if (ok && alive && has_o) {
        const int head = g.h * G + (row0 + row) % G;
        const int64_t out = ((static_cast<int64_t>(g.lo) + node) * a.Hq + head) * d;
        const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (g.t0 == 0 ? 1 : 0);
        float* po = p.part_o + (piece * p.rows_cap + row) * d;
        const bool write = row < rows && !bad;
        const unsigned long long none = g.t0 == 0 && write ? cs.no_number & cs.seen[node] : 0;
        for (int x = col0; x < col1; x += 16) {
          uint32_t o[16];
          tmem_ld16_async(lanes + kColO + x, o);
          tmem_wait16(o);
          float y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(o[i]) * inv;
          for (unsigned long long q = none; q != 0; q &= q - 1) {  // values of the node's path that are no numbers
            const uint16_t* v = static_cast<const uint16_t*>(a.v) + (static_cast<int64_t>(g.lo) + __ffsll(q) - 1) * a.v_stride +
                                static_cast<int64_t>(g.h) * d + x;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if ((v[i] & 0x7f80) == 0x7f80) y[i] = NAN;
          }
          uint32_t u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
          const uint4 u0 = make_uint4(u[0], u[1], u[2], u[3]), u1 = make_uint4(u[4], u[5], u[6], u[7]);
          if (!whole) {
            if (!write) continue;
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(po + x + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          } else if (!kSmall && p.wide_o) {  // by way of the queries' place, so that rows are written as such
            unsigned char* to = smem + row * (NH * 256);
            *reinterpret_cast<uint4*>(to + (((x >> 3) ^ (row & 7)) << 4)) = u0;
            *reinterpret_cast<uint4*>(to + (((x >> 3) + 1 ^ (row & 7)) << 4)) = u1;
          } else if (!write) {
            continue;
          } else if (p.wide_o) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + out + x);
            to[0] = u0;
            to[1] = u1;
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) static_cast<__nv_bfloat16*>(a.o)[out + x + i] = __float2bfloat16_rn(y[i]);
          }
        }
        if (write && !whole && hf == 0) p.part_lse[piece * p.rows_cap + row] = m + log2f(sum);
        tc_fence_before_sync();
      }
      if (!kSmall && whole && p.wide_o) {
        all_sync();
        if (ok && !bad) {
          for (int i = warp; i < rows; i += kSoftWarps) {
            const int rr = row0 + i, at = rr / G;
            uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) +
                                                 ((static_cast<int64_t>(g.lo) + at) * a.Hq + g.h * G + rr - at * G) * d);
            if (8 * lane < d) to[lane] = *reinterpret_cast<const uint4*>(smem + i * (NH * 256) + ((lane ^ (i & 7)) << 4));
          }
        }
      }
      if (ok) {
        if (t == 0 && bad) atomicOr(a.status + g.r, bad_bit);
        if (t == 0 && !whole) {
          if (g.t0 == 0) {
            // the piece in which the item's last tile lies
            const int64_t last = static_cast<int64_t>(walk.u) + (g.tiles - g.t1) - 1;
            int* rec = p.record + 8 * blockIdx.x;
            rec[1] = static_cast<int>(((last + 1) * pieces - 1) / total);
            rec[2] = g.r, rec[3] = g.h, rec[4] = g.m, rec[5] = rows;
            rec[0] = 1;
          }
          p.part_bad[2 * blockIdx.x + (g.t0 == 0 ? 1 : 0)] = bad;
        }
      }
    }
  }

  __syncthreads();
  if (cs.fail != 0) {
    if (t == 0) {  // some of these may be written
      walk = begin;
      while (walk.next(p, cs, g)) atomicOr(a.status + g.r, TREEWY_STATUS_TIMEOUT);
    }
    // copies and products in flight end before the CTA does (a draft's tile among these may never be filled)
    if (warp == kLoadWarp) {
      for (int i = 0; i < S; ++i) {
        if (armed_k > i) mbar_wait_for(&cs.kfull[(armed_k - 1 - i) % S], ((armed_k - 1 - i) / S) & 1, 20000000ull);
        if (armed_v > i) mbar_wait_for(&cs.vfull[(armed_v - 1 - i) % S], ((armed_v - 1 - i) / S) & 1, 20000000ull);
      }
    }
    if (warp == kMmaWarp) {
      if (elect_one()) mma_commit(&cs.drain);
      __syncwarp();
      mbar_wait_for(&cs.drain, 0, 100000000ull);
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// An item that lies in several pieces: its parts' outputs, each normed with
// its own sum, by the weights 2^lse.  A CTA per row: eight warps take the
// parts in turn, a lane eight columns.
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ Params p) {
  after_previous();
  __shared__ float acc[8][256], wsum[8];
  __shared__ int refused;
  const int w = blockIdx.y, row = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31, d = p.a.cache.d;
  const int* rec = p.record + 8 * w;
  if (rec[0] == 0 || row >= rec[5]) return;
  const int parts = rec[1] - w + 1;
  if (t == 0) refused = 0;
  __syncthreads();
  float top = -INFINITY;
  auto piece_of = [&](int i) { return 2 * static_cast<int64_t>(w + i) + (i == 0 ? 1 : 0); };
  for (int i = t; i < parts; i += 256)
    if (p.part_bad[piece_of(i)] != 0) refused = 1;
  for (int i = lane; i < parts; i += 32) {
    const float lse = p.part_lse[piece_of(i) * p.rows_cap + row];
    top = lse > top || lse != lse ? lse : top;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  float sum = 0.f, y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = 0.f;
#pragma unroll 4
  for (int i = warp; i < parts; i += 8) {
    const int64_t at = piece_of(i) * p.rows_cap + row;
    const float f = exp2f(p.part_lse[at] - top);
    sum += f;
    if (8 * lane < d) {
      const float4* o = reinterpret_cast<const float4*>(p.part_o + at * d + 8 * lane);
      const float4 u = o[0], v = o[1];
      y[0] = fmaf(f, u.x, y[0]); y[1] = fmaf(f, u.y, y[1]); y[2] = fmaf(f, u.z, y[2]); y[3] = fmaf(f, u.w, y[3]);
      y[4] = fmaf(f, v.x, y[4]); y[5] = fmaf(f, v.y, y[5]); y[6] = fmaf(f, v.z, y[6]); y[7] = fmaf(f, v.w, y[7]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[warp][8 * lane + e] = y[e];
  if (lane == 0) wsum[warp] = sum;
  __syncthreads();
  if (refused || t >= d) return;
  float z = 0.f, n = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) z += acc[i][t], n += wsum[i];
  const int rr = rec[4] * kTile + row;
  const int64_t node = static_cast<int64_t>(__ldg(p.a.node_offset + rec[2])) + rr / p.G;
  static_cast<__nv_bfloat16*>(p.a.o)[(node * p.a.Hq + rec[3] * p.G + rr % p.G) * d + t] = __float2bfloat16_rn(z / n);
}

int row_tiles_of(const treewy_attn& a) {
  return static_cast<int>((static_cast<int64_t>(a.max_nodes) * (a.Hq / a.cache.Hkv) + kTile - 1) / kTile);
}
// Whether the tiles are put in a row: where there is one row tile to a
// context, or too few items to fill the SMs several times over.
bool listed(const treewy_attn& a) {
  const int mt = row_tiles_of(a);
  const int64_t items = static_cast<int64_t>(a.R) * a.cache.Hkv * mt;
  return a.R <= kMaxListed && (mt == 1 || items <= 4 * kMaxPieces) && items * (2 + a.max_context / kTile) < (int64_t(1) << 31);
}
int rows_cap(const treewy_attn& a) {
  return static_cast<int>(std::min<int64_t>(kTile, static_cast<int64_t>(a.max_nodes) * (a.Hq / a.cache.Hkv)));
}

bool make_map(CUtensorMap* map, const void* codes, const treewy_cache& c) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.page_len),
                              static_cast<cuuint64_t>(c.num_pages * c.Hkv)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.d) * c.page_len};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(c.page_len), 1}, ones[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NH, bool kSmall>
cudaError_t launch(const Params& p, const CUtensorMap& k, const CUtensorMap& v, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(attend_tc_kernel<NH, kSmall>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NH, kSmall>::kBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_after_smem(attend_tc_kernel<NH, kSmall>, dim3(grid), kThreads, Shape<NH, kSmall>::kBytes, stream, p, k, v);
}

}  // namespace

bool attend_on_tensor_cores(const treewy_attn& a) {
  return a.qkv_dtype == TREEWY_DTYPE_BF16 && a.o_dtype == TREEWY_DTYPE_BF16 && a.cache.d % 16 == 0 &&
         (a.flags & TREEWY_FLAG_FORCE_GENERIC) == 0;
}

uint64_t attend_workspace(const treewy_attn& a) {
  if (a.R == 0 || !attend_on_tensor_cores(a) || !listed(a)) return 0;
  return static_cast<uint64_t>(kMaxPieces) * (2ull * rows_cap(a) * (a.cache.d + 1) * 4 + 8 * 4 + 2 * 4);
}

cudaError_t launch_attend_tc(const treewy_attn& a, cudaStream_t stream) {
  Params p = {};
  p.a = a;
  p.G = a.Hq / a.cache.Hkv;
  p.tiles_m = row_tiles_of(a);
  p.listed = listed(a) ? 1 : 0;
  p.rows_cap = rows_cap(a);
  auto wide = [](const void* x, int64_t stride) { return reinterpret_cast<uintptr_t>(x) % 16 == 0 && stride % 8 == 0 ? 1 : 0; };
  p.wide_q = wide(a.q, a.q_stride), p.wide_k = wide(a.k, a.k_stride), p.wide_v = wide(a.v, a.v_stride), p.wide_o = wide(a.o, 0);
  if (p.listed) {
    const size_t rows = static_cast<size_t>(kMaxPieces) * 2 * p.rows_cap;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_lse = p.part_o + rows * a.cache.d;
    p.record = reinterpret_cast<int*>(p.part_lse + rows);
    p.part_bad = p.record + 8 * kMaxPieces;
  }
  unsigned grid;
  if (p.listed) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    grid = static_cast<unsigned>(std::min(sms, kMaxPieces));
  } else {
    const int64_t items = static_cast<int64_t>(a.cache.Hkv) * p.tiles_m;
    if (items > 0x7fffffff / a.R) return cudaErrorNotSupported;
    grid = static_cast<unsigned>(items * a.R);
  }
  CUtensorMap k, v;
  // a cache without pages has none to read: its requests are short or refused
  treewy_cache c = a.cache;
  if (c.num_pages == 0) c.num_pages = 1, c.k = c.v = const_cast<void*>(a.q);
  if (!make_map(&k, c.k, c) || !make_map(&v, c.v, c)) return cudaErrorUnknown;
  const bool two = a.cache.d > 128, small = static_cast<int64_t>(a.max_nodes) * p.G <= 32;
  cudaError_t e = two ? (small ? launch<2, true>(p, k, v, grid, stream) : launch<2, false>(p, k, v, grid, stream))
                      : (small ? launch<1, true>(p, k, v, grid, stream) : launch<1, false>(p, k, v, grid, stream));
  if (e != cudaSuccess || !p.listed) return e;
  return launch_after(attend_join_kernel, dim3(p.rows_cap, grid), 256, stream, p);
}

}  // namespace treewy
