// attend_few.cu -- attention over pages of e4m3 keys and values and the
// draft's own ones on the 5th-generation tensor cores, as attend_tc.cu, for
// drafts of at most 16 rows (nodes times query heads of a key head): single
// tokens and chains.
//
// Such a call reads its context at the rate of HBM or should.  Rows of 128
// would be mostly empty, so the tile lies on its side: TMEM lanes are tokens,
// and the columns are rows (of the queries, hi and lo terms side by side):
//
//   S^T = K Q^T     M = 128 tokens, N = 2 NR, from the page as it is
//   w               a thread has one token of four rows; their terms go to
//                   shared memory, a byte each
//   O^T += V^T w^T  M = 128 columns of the head (V's rows run along the sum)
//
// A product of N = 16 takes an eighth of the time of one of 128, and the
// softmax of a tile is spread over 256 or 512 threads.
//
// The draft's keys and values are the terms' rows 0 .. 15 (hi) and 64 .. 79
// (lo) of a tile: the keys' products are added up in S^T, and the weights of
// the first lanes stand for both tokens of a value.
//
// A context's tiles are few where there are many heads, so that what comes
// before and after them counts: four warps of their own make the next item's
// queries and draft while the softmax goes through this one's tiles, and write
// the last one's outputs (queries, drafts and O are there twice).
//
// Bound by HBM with long contexts: 64 tokens on 8 key heads of 128 over 8000
// tokens 165 us, 6.4 TB/s or 0.94 of a copy; 64 tokens on 2 key heads of 256
// over 2000 to 8000, 62 us (5.3 TB/s, the joining 5 of it); 256K tokens of one
// request 57 us (4.7 TB/s).  With 16 rows by the softmax: drafts of 4 nodes over
// 1000 to 4000 tokens of 8 heads of 128, 94 us (3.6 TB/s), a tile a chain of
// 2,200 cycles (S, maxima, a barrier, weights).  A lone request: the launches
// and the way from the lengths to the first products (12 us at 1500 tokens).
//
//   8 or 16 warps  softmax
//   two            page table, scales and pages (TMA): keys, and values
//   two            issue the products, S two or up to four tiles ahead of O
//   four           queries and draft to e4m3; outputs
#include "attend_tc.cuh"

namespace treewy {
namespace {

constexpr int kSideWarps = 4, kSideThreads = 32 * kSideWarps;
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;

// NH: halves of 128 columns of a head; NR: rows, 8 or 16.
template <int NH, int NR>
struct Shape {
  static constexpr int kRowsOf = 4, kGroups = NR / kRowsOf;          // rows of a thread; of warps that share a tile's tokens
  static constexpr int kSoftWarps = 4 * kGroups, kLoadWarp = kSoftWarps, kMmaWarp = kLoadWarp + 2, kSideWarp = kMmaWarp + 2;
  static constexpr int kThreads = 32 * (kSideWarp + kSideWarps);
  static constexpr uint32_t kRowBytes = 2 * NR * 128;                // hi and lo rows of 128 bytes
  static constexpr int kCols = 16;                                   // of a product of the weights, 16 at least
  static constexpr uint32_t kWBlock = kCols * 128;                   // a term of a tile's weights
  static constexpr uint32_t kWBytes = 4 * kWBlock;                   // of two tiles
  static constexpr uint32_t kQBytes = NH * kRowBytes;                // of an item; two of them
  static constexpr uint32_t kStage = 2 * NH * kHalf;                 // K, then V
  static constexpr int kStages = NH == 2 ? (NR == 8 ? 3 : 2) : 6;
  // What the softmax waits for besides S costs it most where tiles are small (a wait, met by all of its warps, is some 200
  // cycles of a tile's 2,200 for heads of up to 128).  There S comes behind the products that free the weights' place, and
  // behind the tile's constants, so that it stands for both: drafts of 4 nodes 94 us against 106 with waits of their own.
  // For heads of 256 the stages are few: S up to four tiles ahead frees K's sooner (one long context 56 us against 58),
  // and with two stages the constants would hold S up (drafts of 4: 138 us against 148).
  static constexpr bool kInOrder = NH == 1, kWithConsts = kStages > 2;
  static constexpr int kAhead = kInOrder ? 2 : 4;                    // tiles of S
  static constexpr uint32_t kBytes = kWBytes + 2 * kQBytes + kStages * kStage + 1024;
};

// What belongs to an item: two of them in turn.
struct ItemSmem {
  DraftSmem draft;
  alignas(16) float sum[4][kFewRows];  // of the quarters of the lanes
  float ref[kFewRows], inv[kFewRows];  // the rows' references, and one over their sums
  int64_t out[kFewRows];               // where a row's output begins
  uint32_t seen[kFewRows];             // the nodes that a row sees
  int bad;                             // a page of it
};

template <int S, int kAhead>
struct FewSmem {
  RingSmem<S> ring;
  uint64_t sfull[kAhead], sread[kAhead], pready[2], pvdone[2], drain[2];
  // A stage is there for an item's draft (or it has none).  The loading warp is ahead of who fills them by its stages at
  // most, so that with eight barriers none is two phases on before it is waited for.
  uint64_t place[8];
  uint64_t ready[2], free[2], done[2], odone[2], ofree[2];  // items: made, their place free, their softmax done, O, O written
  alignas(16) float top[2][4][kFewRows];  // maxima of the quarters of rows; two sets in turn
  uint32_t tmem;
  ItemSmem item[2];
  PlanSmem plan;
};

// 4 or 8 TMEM columns of this thread's lane; complete after ld_wait.
template <int N>
__device__ __forceinline__ void ld_cols(uint32_t at, uint32_t* r) {
  static_assert(N == 4 || N == 8, "columns");
  if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
  } else {
    tmem_ld8_async(at, *reinterpret_cast<uint32_t(*)[8]>(r));
  }
}
template <int N>
__device__ __forceinline__ void ld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sums over a warp of N values that every lane has: lane l gets that of value
// l / (32 / N), in a few exchanges of ever fewer values.
template <int N>
__device__ __forceinline__ float sum_lanes(float (&v)[N], int lane) {
  int bit = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1, bit >>= 1) {
    const bool upper = lane & bit;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float other = __shfl_xor_sync(kFull, upper ? v[i] : v[n + i], bit);
      v[i] = (upper ? v[n + i] : v[i]) + other;
    }
  }
#pragma unroll
  for (; bit > 0; bit >>= 1) v[0] += __shfl_xor_sync(kFull, v[0], bit);
  return v[0];
}

// A part of an item's queries, and of the draft's keys and values where it has
// them, as terms: by one of the four warps (number w).  All of its rows, or the
// first eight, are loaded at once, and converted one at a time: little code,
// which a CTA meets for the first time here.
// place(kind, i, ..) writes row i of the queries (kind 0), keys (1) or values (2).
template <int NR, typename Place>
__device__ __forceinline__ void fill_rows(const Params& p, DraftSmem& ds, const Segment& g, int rows, float factor, int w, Place place) {
  constexpr int kBatch = 8;
  const treewy_attn& a = p.a;
  const int lane = threadIdx.x & 31, d = a.cache.d, G = p.G;
  const int total = rows + (g.t0 == 0 ? 2 * g.N : 0), each = (total + kSideWarps - 1) / kSideWarps, end = min(total, (w + 1) * each);
  const bool wide = p.wide_q && p.wide_k && p.wide_v;
  const int batch = wide ? kBatch : 1;
#pragma unroll 1
  for (int b0 = w * each; b0 < end; b0 += batch) {
    const int many = min(batch, end - b0);
    // lane i finds the i-th row
    const int e = min(b0 + (lane & (kBatch - 1)), total - 1), n = e - rows, in = e < rows ? e / G : n >> 1;
    const int64_t token = static_cast<int64_t>(g.lo) + in;
    const uint16_t* row = e < rows ? static_cast<const uint16_t*>(a.q) + token * a.q_stride + (static_cast<int64_t>(g.h) * G + e - in * G) * d
                                   : static_cast<const uint16_t*>(n & 1 ? a.v : a.k) + token * (n & 1 ? a.v_stride : a.k_stride) +
                                         static_cast<int64_t>(g.h) * d;
    const unsigned long long at = reinterpret_cast<unsigned long long>(row);
    uint4 x[kBatch];
    if (wide) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint16_t* from = reinterpret_cast<const uint16_t*>(__shfl_sync(kFull, at, i));
        if (i < many) x[i] = load_row8(from, 8 * lane, d);
      }
    } else {
      x[0] = load_row8_odd(reinterpret_cast<const uint16_t*>(__shfl_sync(kFull, at, 0)), 8 * lane, d);
    }
#pragma unroll 1
    for (int e0 = 0; e0 < many; ++e0) {
      const int r = b0 + e0, kind = r < rows ? 0 : 1 + ((r - rows) & 1), to = kind == 0 ? r : (r - rows) >> 1;
      uint2 hi, lo;
      bool none;
      // a value that is no number would reach the nodes that do not see it: weights of zero times it
      const int unit = row_terms(x[0], kind == 2, hi, lo, none);
      place(kind, to, hi, lo);
      if (lane == 0) {
        if (kind == 0) {
          ds.rowf[to] = pow2(unit) * factor;
        } else if (kind == 1) {
          ds.ks[to] = pow2(unit);
        } else {
          if (none) atomicOr(&ds.no_number, 1ull << to);
          ds.lv[to] = static_cast<float>(unit);
          ds.il[to] = pow2(-unit);
        }
      }
#pragma unroll
      for (int i = 0; i + 1 < kBatch; ++i) x[i] = x[i + 1];
    }
  }
}

template <int NH, int NR>
__global__ void __launch_bounds__(Shape<NH, NR>::kThreads, 1)
    attend_few_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using Sh = Shape<NH, NR>;
  constexpr int S = Sh::kStages, kAhead = Sh::kAhead, NT = Sh::kRowsOf, kThreads = Sh::kThreads, kSoftWarps = Sh::kSoftWarps, kSoftThreads = 32 * kSoftWarps;
  constexpr int kLoadWarp = Sh::kLoadWarp, kMmaWarp = Sh::kMmaWarp, kSideWarp = Sh::kSideWarp;
  extern __shared__ unsigned char raw_smem[];
  __shared__ FewSmem<S, kAhead> cs;
  RingSmem<S>& rs = cs.ring;
  unsigned char* wts = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  unsigned char* qs = wts + Sh::kWBytes;
  unsigned char* ring = qs + 2 * Sh::kQBytes;
  const treewy_attn& a = p.a;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, d = a.cache.d, G = p.G;

  // ---- set-up, while the kernel before may still run
  if (warp == 0) {
    init_ring(rs, lane);
    if (lane < 8) mbar_init(&cs.place[lane], 1);
    if (lane < kAhead) {
      mbar_init(&cs.sfull[lane], 1);
      mbar_init(&cs.sread[lane], kSoftWarps);
    }
    if (lane < 2) {
      mbar_init(&cs.pready[lane], kSoftWarps);
      mbar_init(&cs.pvdone[lane], 1);
      mbar_init(&cs.ready[lane], kSideWarps);
      mbar_init(&cs.free[lane], kSoftWarps);
      mbar_init(&cs.done[lane], kSoftWarps);
      mbar_init(&cs.odone[lane], 1);
      mbar_init(&cs.ofree[lane], kSideWarps);
      mbar_init(&cs.drain[lane], 1);
    }
    fence_mbarrier_init();
    if (lane == 0) {
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&cs.tmem, kTmemCols);
    tmem_relinquish();
  }
  after_previous();
  const Part<false> mine = make_plan<kThreads, false>(p, cs.plan, rs);
  const uint32_t tmem = cs.tmem;

  Walk<false> walk = mine.walk;
  Segment g;
  int armed = 0;
  int gt = 0;   // tiles so far
  int slot = 0;      // their stage
  uint32_t use = 0;  // and the parity of its use
  auto next_stage = [&] {
    if (++slot == S) slot = 0, use ^= 1;
  };
  int seg = 0;  // items, or parts of them, so far: the k-th uses place k & 1 for the k / 2-th time

  if (warp == kLoadWarp) {
    armed = load_pages<false, NH>(p, cs, rs, walk, ring, kmap, [](const Segment&) { return true; },
                                     [](const Segment&, int, int, uint32_t) { return true; });
  } else if (warp == kLoadWarp + 1) {
    // the draft's tile is filled by other warps, once both its stages are free
    static_assert(S < 8, "drafts whose stage is there and that are not filled yet");
    armed = load_pages<true, NH>(
        p, cs, rs, walk, ring, vmap,
        [&](const Segment& s) {
          if (s.t0 != 0) warp_arrive(&cs.place[seg & 7]);
          ++seg;
          return true;
        },
        [&](const Segment&, int tile, int slot, uint32_t again) {
          if (tile >= S && !wait_warp(rs, &rs.kfree[slot], again)) return false;
          warp_arrive(&cs.place[(seg - 1) & 7]);
          return true;
        });
  } else if (warp == kMmaWarp) {
    // ---- S^T = K Q^T
    const uint32_t id_s = idesc_f8(2 * NR, false, false), r0 = smem_addr(ring);
    bool ok = true;
#pragma unroll 1
    for (; ok && walk.next(p, cs.plan, g); ++seg) {
      const uint32_t q0 = smem_addr(qs) + (seg & 1) * Sh::kQBytes;
      ok = wait_warp(rs, &cs.ready[seg & 1], (seg >> 1) & 1);
#pragma unroll 1
      for (int j = g.t0; ok && j < g.t1; ++j, ++gt) {
        const int b = gt % kAhead;
        if constexpr (Sh::kInOrder) ok = gt < 2 || wait_warp(rs, &cs.pvdone[b], ((gt - 2) >> 1) & 1);
        else ok = gt < kAhead || wait_warp(rs, &cs.sread[b], (gt / kAhead - 1) & 1);
        if constexpr (Sh::kWithConsts) ok = ok && wait_warp(rs, &rs.cfull[slot], use);
        ok = ok && wait_warp(rs, &rs.kfull[slot], use);
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
          uint32_t acc = 0, k0 = r0 + slot * Sh::kStage;
#pragma unroll 1
          for (int term = 0; term < (j == 0 ? 2 : 1); ++term, k0 += 64 * 128) {  // the draft's lo rows
#pragma unroll
            for (int x = 0; x < NH; ++x) {
              const int steps = (min(128, d - 128 * x) + 31) / 32;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k >= steps) continue;
                mma_f8(tmem + kColS + b * (2 * NR), smem_desc_sw128(k0 + x * kHalf + k * 32, 1024),
                       smem_desc_sw128(q0 + x * Sh::kRowBytes + k * 32, 1024), id_s, acc);
                acc = 1;
              }
            }
          }
          mma_commit(&cs.sfull[b]);
          mma_commit(&rs.kfree[slot]);
        }
        __syncwarp();
        next_stage();
      }
    }
  } else if (warp == kMmaWarp + 1) {
    // ---- O^T += V^T w^T
    const uint32_t id_o = idesc_f8(Sh::kCols, true, false), r0 = smem_addr(ring), w0 = smem_addr(wts);
    bool ok = true;
#pragma unroll 1
    for (; ok && walk.next(p, cs.plan, g); ++seg) {
      const uint32_t o0 = tmem + kColO + (seg & 1) * (NH * Sh::kCols);
      ok = seg < 2 || wait_warp(rs, &cs.ofree[seg & 1], ((seg >> 1) - 1) & 1);
#pragma unroll 1
      for (int j = g.t0; ok && j < g.t1; ++j, ++gt) {
        ok = wait_warp(rs, &rs.vfull[slot], use) && wait_warp(rs, &cs.pready[gt & 1], (gt >> 1) & 1);
        if (!ok) break;
        tc_fence_after_sync();
        // 32 tokens each: the draft's are the first and the third
        const int n = min(kTile, g.len - (j - 1) * kTile), steps = j == 0 ? 5 : (1 << ((n + 31) / 32)) - 1;
        if (elect_one()) {
          const uint32_t w = w0 + (gt & 1) * (2 * Sh::kWBlock), v0 = r0 + slot * Sh::kStage + NH * kHalf;
#pragma unroll
          for (int x = 0; x < NH; ++x) {
            uint32_t acc = j != g.t0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (((steps >> k) & 1) == 0) continue;
              const uint64_t v = desc_mn(v0 + x * kHalf + k * 4096);
              mma_f8(o0 + x * Sh::kCols, v, smem_desc_sw128(w + k * 32, 1024), id_o, acc);
              mma_f8(o0 + x * Sh::kCols, v, smem_desc_sw128(w + Sh::kWBlock + k * 32, 1024), id_o | kBE5m2, 1);
              acc = 1;
            }
          }
          mma_commit(&rs.vfree[slot]);
          mma_commit(&cs.pvdone[gt & 1]);
          if (j + 1 == g.t1) mma_commit(&cs.odone[seg & 1]);
        }
        __syncwarp();
        next_stage();
      }
    }
  } else if (warp < kSoftWarps) {
    // ---- softmax: a warp has the tokens 32 (w % 4) .. of a part of the rows
    const int quarter = warp & 3, row0 = (warp >> 2) * NT, token = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    auto all_sync = [] { named_bar_sync<1, kSoftThreads>(); };
#pragma unroll 1
    for (; walk.next(p, cs.plan, g); ++seg) {
      ItemSmem& it = cs.item[seg & 1];
      const DraftSmem& ds = it.draft;
      const uint32_t o0 = lanes + kColO + (seg & 1) * (NH * Sh::kCols) + row0;
      wait_warp(rs, &cs.ready[seg & 1], (seg >> 1) & 1);
      float m[NT], sum[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) m[i] = -INFINITY, sum[i] = 0.f;
      const int t0 = g.t0, t1 = g.t1, N = g.N, len = g.len;
#pragma unroll 1
      for (int j = t0; j < t1; ++j, ++gt, next_stage()) {
        const int b = gt & 1;
        const Consts& cc = rs.c[slot];
        // after a wait that gave up a warp still comes by every barrier of threads
        bool ok = wait_warp(rs, &cs.sfull[gt % kAhead], (gt / kAhead) & 1);
        if constexpr (!Sh::kWithConsts) ok = wait_warp(rs, &rs.cfull[slot], use) && ok;
        tc_fence_after_sync();
        if (cc.bad != 0) it.bad = 1;
        const bool draft_tile = j == 0;
        const int n = draft_tile ? N : min(kTile, len - (j - 1) * kTile);
        if (!draft_tile && n < kTile && ok) ok = wait_warp(rs, &rs.vfull[slot], use);
        if (!draft_tile && n < kTile && ok) {  // values behind the context: anything, so none
          unsigned char* v = ring + slot * Sh::kStage + NH * kHalf;
#pragma unroll 1
          for (int i = n * 8 + t; i < ((n + 31) & ~31) * 8; i += kSoftThreads)
#pragma unroll
            for (int x = 0; x < NH; ++x) *reinterpret_cast<uint4*>(v + x * kHalf + i * 16) = make_uint4(0, 0, 0, 0);
        }
        uint32_t r[2 * NT];
        if (ok) {
          const uint32_t sc = lanes + kColS + gt % kAhead * (2 * NR) + row0;
          ld_cols<NT>(sc, r);
          ld_cols<NT>(sc + NR, r + NT);
          ld_wait<2 * NT>(r);
          tc_fence_before_sync();
        }
        if constexpr (!Sh::kInOrder) warp_arrive(&cs.sread[gt % kAhead]);
        const float ks = draft_tile ? ds.ks[lane] : cc.ks[token >> 4], lv = draft_tile ? ds.lv[lane] : cc.lv[token >> 4];
        const float il = draft_tile ? (token < n ? ds.il[lane] : 0.f) : cc.il[token >> 4];
        float s[NT], top[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float x = __uint_as_float(r[i]) + __uint_as_float(r[NT + i]);
          const float y = fmaf(x, fmaxf(ks * ds.rowf[row0 + i], kLeast), lv);
          const bool live = token < n && (!draft_tile || ((it.seen[row0 + i] >> lane) & 1));
          s[i] = live ? y : -INFINITY;
          top[i] = warp_max(s[i]);
        }
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < NT; i += 4) *reinterpret_cast<float4*>(&cs.top[b][quarter][row0 + i]) = make_float4(top[i], top[i + 1], top[i + 2], top[i + 3]);
        }
        all_sync();
        bool grown = false;
#pragma unroll
        for (int i = 0; i < NT; i += 4) {
          float4 x = *reinterpret_cast<const float4*>(&cs.top[b][0][row0 + i]);
#pragma unroll
          for (int q = 1; q < 4; ++q) {
            const float4 y = *reinterpret_cast<const float4*>(&cs.top[b][q][row0 + i]);
            x = make_float4(fmaxf(x.x, y.x), fmaxf(x.y, y.y), fmaxf(x.z, y.z), fmaxf(x.w, y.w));
          }
          top[i] = x.x, top[i + 1] = x.y, top[i + 2] = x.z, top[i + 3] = x.w;
#pragma unroll
          for (int e = 0; e < 4; ++e) grown |= top[i + e] > m[i + e] + kGrowth;
        }
        // the weights' place is read no more
        if constexpr (!Sh::kInOrder)
          if (gt >= 2) wait_warp(rs, &cs.pvdone[b], ((gt - 2) >> 1) & 1);
        if (j == t0) {
#pragma unroll
          for (int i = 0; i < NT; ++i) m[i] = top[i];
        } else if (grown) {  // the same in all warps that have these rows
          wait_warp(rs, &cs.pvdone[b ^ 1], ((gt - 1) >> 1) & 1);
          tc_fence_after_sync();
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const bool more = top[i] > m[i] + kGrowth;
            const float down = more ? ex2(m[i] - top[i]) : 1.f;
            if (more) m[i] = top[i];
            sum[i] *= down;
            top[i] = down;
          }
#pragma unroll 1
          for (int x = 0; x < NH; ++x) {  // halves of the head's columns
            uint32_t o[NT];
            ld_cols<NT>(o0 + x * Sh::kCols, o);
            ld_wait<NT>(o);
#pragma unroll
            for (int i = 0; i < NT; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * top[i]);
            tmem_st4(o0 + x * Sh::kCols, o);
          }
          tmem_wait_st();
        }
        unsigned char* w = wts + b * (2 * Sh::kWBlock);
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
          const float w0 = ex2(s[i] + (kBias - m[i])), w1 = ex2(s[i + 1] + (kBias - m[i + 1]));
          sum[i] = fmaf(w0, il, sum[i]);
          sum[i + 1] = fmaf(w1, il, sum[i + 1]);
          uint32_t hi, lo;
          weight_terms(w0, w1, hi, lo);
          if (!draft_tile || quarter == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = row0 + i + e;
              unsigned char* at = w + row * 128 + (((token >> 4) ^ (row & 7)) << 4) + (token & 15);
              at[0] = static_cast<unsigned char>(hi >> (8 * e));
              at[Sh::kWBlock] = static_cast<unsigned char>(lo >> (16 * e + 8));
              if (draft_tile) {  // a value's two terms have one weight
                at = w + row * 128 + ((((token + 64) >> 4) ^ (row & 7)) << 4) + (token & 15);
                at[0] = static_cast<unsigned char>(hi >> (8 * e));
                at[Sh::kWBlock] = static_cast<unsigned char>(lo >> (16 * e + 8));
              }
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        warp_arrive(&cs.pready[b]);
      }
      const float part = sum_lanes<NT>(sum, lane);  // of row row0 + lane / (32 / NT)
      if (lane % (32 / NT) == 0) it.sum[quarter][row0 + lane / (32 / NT)] = part;
      if (quarter == 0 && lane == 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i) it.ref[row0 + i] = m[i];
      }
      warp_arrive(&cs.done[seg & 1]);
      if (lane == 0) arrive(&cs.free[seg & 1]);
    }
  } else {
    // ---- the next item's queries and draft, the last one's outputs
    const int quarter = warp & 3, u = t - 32 * kSideWarp;
    const float factor = a.scale * 1.4426950408889634f;  // scores in powers of two
    auto side_sync = [] { named_bar_sync<2, kSideThreads>(); };
    Walk<false> behind = walk;
    int tiles = 0;  // up to the item that is made
    bool more = true;
#pragma unroll 1
    for (;; ++seg) {
      more = more && walk.next(p, cs.plan, g);
      if (more) {
        ItemSmem& it = cs.item[seg & 1];
        DraftSmem& ds = it.draft;
        const int rows = g.N * G, at = tiles % S;
        unsigned char *q = qs + (seg & 1) * Sh::kQBytes, *draft = ring + at * Sh::kStage;
        const int parent = u < g.N ? (a.parent != nullptr ? __ldg(a.parent + g.lo + u) : u - 1) : -1;
        if (seg >= 2) wait_warp(rs, &cs.free[seg & 1], ((seg >> 1) - 1) & 1);
        if (u == 0) ds.bad_tree = 0, ds.no_number = 0, it.bad = 0;
        zero_rows<kSideThreads>(q, NH, Sh::kRowBytes, rows, NR, u);
        zero_rows<kSideThreads>(q, NH, Sh::kRowBytes, NR + rows, 2 * NR, u);
        if (u >= rows && u < NR) ds.rowf[u] = 0.f;
        side_sync();
        if (u < g.N) {
          const bool wrong = parent < -1 || parent >= u;
          if (wrong) ds.bad_tree = 1;
          ds.parent[u] = wrong ? -1 : parent;
        }
        bool placed = false;
        auto stage_is_there = [&] {
          if (!placed) wait_warp(rs, &cs.place[seg & 7], (seg >> 3) & 1);
          placed = true;
        };
        fill_rows<NR>(p, ds, g, rows, factor, warp - kSideWarp, [&](int kind, int i, uint2 hi, uint2 lo) {
          if (kind != 0) stage_is_there();
          unsigned char* tile = kind == 0 ? q : kind == 1 ? draft : draft + NH * kHalf;
          const uint32_t block = kind == 0 ? Sh::kRowBytes : kHalf;
          if (8 * lane < NH * 128) {
            *operand8(tile, i, lane, block) = hi;
            *operand8(tile, i + (kind == 0 ? NR : 64), lane, block) = lo;
          }
        });
        stage_is_there();
        if (g.t0 == 0) {  // what the draft's tile has behind its values
          zero_rows<kSideThreads>(draft + NH * kHalf, NH, kHalf, g.N, 32, u);
          zero_rows<kSideThreads>(draft + NH * kHalf, NH, kHalf, 64 + g.N, 96, u);
          if (u >= g.N && u < 32) ds.ks[u] = 1.f, ds.lv[u] = ds.il[u] = 0.f;
        }
        fence_proxy_async_smem();
        side_sync();
        if (u < NR) {
          uint32_t m = 0;
#pragma unroll 1
          for (int n = min(u, rows - 1) / G; n >= 0; n = ds.parent[n]) m |= 1u << n;
          it.seen[u] = m;
        }
        if (g.t0 == 0 && u == 0) {
          arrive(&rs.kfull[at]);
          arrive(&rs.vfull[at]);
        }
        warp_arrive(&cs.ready[seg & 1]);
        tiles += g.t1 - g.t0;
      }
      if (seg == 0) continue;
      if (!behind.next(p, cs.plan, g)) break;
      // ---- outputs of the one before
      const int k = seg - 1;
      ItemSmem& it = cs.item[k & 1];
      const int rows = g.N * G;
      const bool whole = g.t0 == 0 && g.t1 == g.tiles;
      bool ok = wait_warp(rs, &cs.done[k & 1], (k >> 1) & 1);
      ok = wait_warp(rs, &cs.odone[k & 1], (k >> 1) & 1) && ok;
      tc_fence_after_sync();
      const bool bad_tree = it.draft.bad_tree != 0, bad = bad_tree || it.bad != 0;
      const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (g.t0 == 0 ? 1 : 0);
      if (u < NR) {
        const float total = it.sum[0][u] + it.sum[1][u] + it.sum[2][u] + it.sum[3][u];
        const int node = u / G;
        it.inv[u] = 1.f / total;
        it.out[u] = whole ? ((static_cast<int64_t>(g.lo) + node) * a.Hq + g.h * G + u - node * G) * d : (piece * p.rows_cap + u) * d;
        if (!whole && ok && !bad && u < rows) p.part_lse[piece * p.rows_cap + u] = it.ref[u] + log2f(total);
      }
      side_sync();
      if (ok && !bad) {
#pragma unroll 1
        for (int x = 0; x < NH * (NR / 8); ++x) {
          const int half = x / (NR / 8), r0 = x % (NR / 8) * 8, col = half * 128 + quarter * 32 + lane;
          if (r0 >= rows) continue;
          uint32_t o[8];
          ld_cols<8>(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kColO + ((k & 1) * NH + half) * Sh::kCols + r0, o);
          ld_wait<8>(o);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (r0 + i >= rows || col >= d) continue;
            const float y = __uint_as_float(o[i]) * it.inv[r0 + i];
            if (whole) static_cast<__nv_bfloat16*>(a.o)[it.out[r0 + i] + col] = __float2bfloat16_rn(y);
            else p.part_o[it.out[r0 + i] + col] = y;
          }
        }
        if (g.t0 == 0 && it.draft.no_number != 0) {  // values of the rows' paths that are no numbers
#pragma unroll 1
          for (int x = 0; x < rows * NH; ++x) {
            const int row = x / NH, col = x % NH * 128 + quarter * 32 + lane;
            if (col >= d) continue;
#pragma unroll 1
            for (uint32_t n = it.seen[row] & static_cast<uint32_t>(it.draft.no_number); n != 0; n &= n - 1) {
              const uint16_t v = static_cast<const uint16_t*>(a.v)[(static_cast<int64_t>(g.lo) + __ffs(n) - 1) * a.v_stride +
                                                                   static_cast<int64_t>(g.h) * d + col];
              if ((v & 0x7f80) != 0x7f80) continue;
              if (whole) static_cast<__nv_bfloat16*>(a.o)[it.out[row] + col] = __float2bfloat16_rn(NAN);
              else p.part_o[it.out[row] + col] = NAN;
            }
          }
        }
        tc_fence_before_sync();
      }
      if (ok && u == 0) report(p, mine, behind, g, rows, bad_tree, bad);
      side_sync();  // before this place is made anew
      warp_arrive(&cs.ofree[k & 1]);
    }
  }

  __syncthreads();
  if (rs.fail != 0) {
    if (t == 0) {  // some of these may be written
      walk = mine.walk;
      while (walk.next(p, cs.plan, g)) atomicOr(a.status + g.r, TREEWY_STATUS_TIMEOUT);
    }
    if (warp == kLoadWarp) drain_copies(rs.kfull, armed);
    if (warp == kLoadWarp + 1) drain_copies(rs.vfull, armed);
    if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      uint64_t* drain = &cs.drain[warp - kMmaWarp];
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait_for(drain, 0, 100000000ull);
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int NH, int NR>
cudaError_t launch(const Params& p, const CUtensorMap& k, const CUtensorMap& v, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(attend_few_kernel<NH, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NH, NR>::kBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_after_smem(attend_few_kernel<NH, NR>, dim3(grid), Shape<NH, NR>::kThreads, Shape<NH, NR>::kBytes, stream, p, k, v);
}

template <int NH>
cudaError_t by_rows(const Params& p, const CUtensorMap& k, const CUtensorMap& v, unsigned grid, cudaStream_t stream) {
  const int rows = p.a.max_nodes * p.G;
  // 64 single tokens of eight heads a key head: 64 us with 8 rows, 67 with 16
  return rows <= 8 ? launch<NH, 8>(p, k, v, grid, stream) : launch<NH, 16>(p, k, v, grid, stream);
}

}  // namespace

cudaError_t launch_attend_few(const Params& p, const CUtensorMap& k, const CUtensorMap& v, unsigned grid, cudaStream_t stream) {
  return p.a.cache.d > 128 ? by_rows<2>(p, k, v, grid, stream) : by_rows<1>(p, k, v, grid, stream);
}

}  // namespace treewy
