// attend_tc.cu -- attention over pages of e4m3 keys and values and the draft's
// own ones on the 5th-generation tensor cores (tcgen05, TMEM, TMA), for bf16
// rows and outputs, head sizes that are multiples of 16, and drafts of more
// than 16 rows; and what joins the pieces of an item.
//
// attend_split_kernel makes the terms of all queries and of the drafts' keys and
// values, once for every tile that reads them; attend_tc_kernel then loads them
// as it loads pages.
//
// A tile is 128 rows, (node, query head) pairs that share a key head, times
// 128 tokens.  TMEM lanes are rows:
//
//   S = Q K^T          Q's terms and K in shared memory, S in TMEM, twice (three
//                      times for heads of up to 128, where O leaves room)
//   w                  two terms, back in TMEM in the place of S
//   O += w V           V in shared memory as it is stored (rows along the sum)
//
// Two sets of eight warps take tiles in turn, so that one's loads and waits fall
// into the other's arithmetic; a thread has half a row of its set's tile.  The
// sets share the rows' references: a tile's weights wait for the maxima of the
// tile before it, not for its weights.  The first reference comes from a
// segment's first two tiles, the draft's own one being small.
//
// The draft's keys and values take two tokens of its tile each, one per term
// (n and 64 + n); the ancestors are a mask of bits.
//
// Bound by the way of a tile through its set where the tensor pipe could take
// twice as many (48 % busy): S, maxima, the reference, weights, O, and only then
// the next S in its place, O taking all of TMEM that S does not for heads of
// 256.  A tile's two products are 2,048 cycles, and a set takes 6,500 for one,
// 3,100 of them waiting for S.  256 trees of 16 to 64 nodes over 500 to 4000
// tokens: 470 us, 811 TFLOP/s (counted once, not by term); all of 64 nodes over
// 4000: 952 us, 1,137 TFLOP/s, 0.58 of a dense bf16 product's rate; with heads
// of 128, whose softmax is as long, 787 us, 688 TFLOP/s (828 us with two tiles
// of S).
//
//   warps 0-15   softmax, outputs
//   warps 16, 17 page table, scales, pages and terms (TMA): keys, and values
//   warp 18      issues the products: S of the next tiles before O of this one
#include "attend_tc.cuh"

namespace treewy {
namespace {

constexpr int kSets = 2, kSetWarps = 8, kSoftWarps = kSets * kSetWarps, kLoadWarp = kSoftWarps, kMmaWarp = kLoadWarp + 2;
constexpr int kSoftThreads = 32 * kSoftWarps, kThreads = 32 * (kMmaWarp + 1);
constexpr int kParts = kSoftWarps / 4;  // warps that share 32 rows
constexpr uint32_t kColO = 0, kTmemCols = 512;
// The first reference is the largest of a segment's first two tiles where a token stands out there: where some 16 tokens
// in a row have none within 2^-kFar of it.  Then the others need the weights' bits, and few rows see a larger one later.
// Elsewhere it is 2^kRoom above, so that a maximum that grows brings the output down less often: that waits for the tile
// before.  Wide trees 470 us; 478 and 519 with kFar = 6 and 4, 527 without room for any row; with room for all of them
// (471) the outputs of 32,000 tokens beside a first one of a third of the weight are more than 0.008 off.
constexpr float kFar = 8.f, kRoom = 4.f;

// Terms of every row: a warp takes four rows of a token (its query heads, then
// key heads, keys and values) at a time.  Units are the exponents of a row's
// power of two, kNone above them where a value's row has something that is no
// number.  Bound by HBM: every row is read and written once (the wide trees'
// 210 MB in 47 us), where every CTA would convert them for its own tile.
//
// Its first CTA also finds the order in which the requests are begun where an
// item is a CTA's: the longest context first, so that the last CTAs are short
// (256 trees 470 us, 490 in their own order; 100 of them 183 and 221).
constexpr int kNone = 1024, kSplitThreads = 256, kSplitRows = 4, kMaxOrdered = 1024;
__global__ void __launch_bounds__(kSplitThreads) attend_split_kernel(const __grid_constant__ Params p, int groups) {
  after_previous();
  const treewy_attn& a = p.a;
  const int lane = threadIdx.x & 31, d = a.cache.d, G = p.G, Hkv = a.cache.Hkv, heads = a.Hq + 2 * Hkv;
  const unsigned T = static_cast<unsigned>(a.T), jobs = T * groups;
  if (p.order != nullptr && blockIdx.x == 0) {
    __shared__ int length[kMaxOrdered];
    for (int r = threadIdx.x; r < a.R; r += kSplitThreads) length[r] = __ldg(a.cache.length + r);
    __syncthreads();
    for (int r = threadIdx.x; r < a.R; r += kSplitThreads) {
      const int mine = length[r];
      int before = 0;
#pragma unroll 8
      for (int s = 0; s < a.R; ++s) before += length[s] > mine || (length[s] == mine && s < r);
      p.order[before] = r;
    }
  }
#pragma unroll 1
  for (unsigned job = blockIdx.x * (kSplitThreads / 32) + (threadIdx.x >> 5); job < jobs; job += gridDim.x * (kSplitThreads / 32)) {
    const unsigned token = job / groups;
    const int first = static_cast<int>(job - token * groups) * kSplitRows;
    uint4 x[kSplitRows];
#pragma unroll
    for (int e = 0; e < kSplitRows; ++e) {
      const int head = first + e;
      if (head >= heads) continue;
      const int kind = head < a.Hq ? 0 : head < a.Hq + Hkv ? 1 : 2, h = head - (kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + Hkv);
      const uint16_t* from = static_cast<const uint16_t*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                             token * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + static_cast<int64_t>(h) * d;
      const bool wide = kind == 0 ? p.wide_q : kind == 1 ? p.wide_k : p.wide_v;
      x[e] = wide ? load_row8(from, 8 * lane, d) : load_row8_odd(from, 8 * lane, d);
    }
#pragma unroll
    for (int e = 0; e < kSplitRows; ++e) {
      const int head = first + e;
      if (head >= heads) continue;
      const int kind = head < a.Hq ? 0 : head < a.Hq + Hkv ? 1 : 2, h = head - (kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + Hkv);
      const unsigned g = kind == 0 ? G : 1, hk = h / g, to = (hk * T + token) * g + (h - hk * g);
      uint2 hi, lo;
      bool none;
      // a value that is no number would reach the nodes that do not see it: weights of zero times it
      int unit = row_terms(x[e], kind == 2, hi, lo, none);
      if (kind == 2 && none) unit += kNone;
      uint8_t* terms = (kind == 0 ? p.q_terms : kind == 1 ? p.k_terms : p.v_terms) + static_cast<int64_t>(to) * d + 8 * lane;
      if (8 * lane < d) {
        *reinterpret_cast<uint2*>(terms) = hi;
        *reinterpret_cast<uint2*>(terms + static_cast<int64_t>(T) * (kind == 0 ? a.Hq : Hkv) * d) = lo;
      }
      if (lane == 0) (kind == 0 ? p.q_units : kind == 1 ? p.k_units : p.v_units)[to] = static_cast<int16_t>(unit);
    }
  }
}

// NH: halves of 128 columns of a head.
template <int NH>
struct Shape {
  static constexpr uint32_t kQBytes = 2 * NH * kHalf, kStage = 2 * NH * kHalf;  // hi and lo; K and V
  static constexpr int kStages = NH == 2 ? 2 : 5;
  static constexpr int kScores = NH == 2 ? 2 : 3;      // tiles of S
  static constexpr uint32_t kColS = kTmemCols - kScores * kTile;
  static constexpr uint32_t kBytes = kQBytes + kStages * kStage + 1024;
};

template <int S>
struct AttendSmem {
  RingSmem<S> ring;
  uint64_t sfull[3], mdone[2], pready[2], pvdone[2], qfull, qfree, drain;
  float ref[kTile], first[kSets][kTile], half[kSets][2][kTile], low[kSets][2][kTile], sum[kParts][kTile];  // of the rows
  uint32_t tmem;
  int bad[2];                    // a page of the segment's: two in turn, as warps still read the last one's
  Segment segment;               // the softmax warps' current one
  DraftSmem draft;
  PlanSmem plan;
};

struct Maps {
  CUtensorMap k, v;              // pages
  CUtensorMap q_terms, k_terms, v_terms;
};

// Parents of the segment's nodes; who sees whom.
__device__ __forceinline__ void load_tree(const Params& p, DraftSmem& ds, const Segment& g, int t) {
  if (t >= g.N) return;
  const int q = p.a.parent != nullptr ? __ldg(p.a.parent + g.lo + t) : t - 1;
  const bool wrong = q < -1 || q >= t;
  if (wrong) ds.bad_tree = 1;
  ds.parent[t] = wrong ? -1 : q;
}
__device__ __forceinline__ void see(DraftSmem& ds, const Segment& g, int t) {
  if (t >= g.N) return;
  unsigned long long m = 0;
#pragma unroll 1
  for (int q = t; q >= 0; q = ds.parent[q]) m |= 1ull << q;
  ds.seen[t] = m;
}

template <int NH>
__global__ void __launch_bounds__(kThreads, 1) attend_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  using Sh = Shape<NH>;
  constexpr int S = Sh::kStages, B = Sh::kScores;
  extern __shared__ unsigned char raw_smem[];
  __shared__ AttendSmem<S> cs;
  RingSmem<S>& rs = cs.ring;
  DraftSmem& ds = cs.draft;
  unsigned char* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  unsigned char* ring = smem + Sh::kQBytes;
  const treewy_attn& a = p.a;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, d = a.cache.d, G = p.G;

  // ---- set-up, while the kernel before may still run
  if (warp == 0) {
    init_ring(rs, lane);
    if (lane < 3) mbar_init(&cs.sfull[lane], 1);
    if (lane < 2) {
      mbar_init(&cs.mdone[lane], kSetWarps);
      mbar_init(&cs.pready[lane], kSetWarps);
      mbar_init(&cs.pvdone[lane], 1);
    }
    if (lane == 0) {
      mbar_init(&cs.qfull, 1);
      mbar_init(&cs.qfree, kSoftWarps);
      mbar_init(&cs.drain, 1);
    }
    fence_mbarrier_init();
    if (lane == 0) {
      prefetch_tensormap(&maps.k);
      prefetch_tensormap(&maps.v);
      prefetch_tensormap(&maps.q_terms);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&cs.tmem, kTmemCols);
    tmem_relinquish();
  }
  after_previous();
  const Part<true> mine = make_plan<kThreads, true>(p, cs.plan, rs);
  const uint32_t tmem = cs.tmem;

  Walk<true> walk = mine.walk;
  Segment g;
  int armed = 0;
  int queries = 0;  // segments whose queries have been sent for
  int gt = 0;  // tiles so far

  if (warp == kLoadWarp) {
    armed = load_pages<false, NH>(
        p, cs, rs, walk, ring, maps.k,
        [&](const Segment& s) {
          if (queries > 0 && !wait_warp(rs, &cs.qfree, (queries - 1) & 1)) return false;
          ++queries;
          if (lane == 0) {
            mbar_arrive_expect_tx(&cs.qfull, 2 * NH * kHalf);
            const int row = static_cast<int>((static_cast<int64_t>(s.h) * a.T + s.lo) * G + s.m * kTile);
#pragma unroll
            for (int x = 0; x < 2 * NH; ++x) tma_load_3d(smem + x * kHalf, &maps.q_terms, &cs.qfull, x % NH * 128, row, x / NH);
          }
          __syncwarp();
          return true;
        },
        [&](const Segment& s, int tile, int slot, uint32_t) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&rs.kfull[slot], NH * kHalf);
            for (int x = 0; x < 2 * NH; ++x)
              tma_load_3d(ring + slot * Sh::kStage + x % NH * kHalf + x / NH * (kHalf / 2), &maps.k_terms, &rs.kfull[slot], x % NH * 128,
                          static_cast<int>(s.h * a.T + s.lo), x / NH);
          }
          __syncwarp();
          return true;
        });
  } else if (warp == kLoadWarp + 1) {
    armed = load_pages<true, NH>(
        p, cs, rs, walk, ring, maps.v, [](const Segment&) { return true; },
        [&](const Segment& s, int tile, int slot, uint32_t) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&rs.vfull[slot], NH * kHalf);
            for (int x = 0; x < 2 * NH; ++x)
              tma_load_3d(ring + slot * Sh::kStage + (NH + x % NH) * kHalf + x / NH * (kHalf / 2), &maps.v_terms, &rs.vfull[slot],
                          x % NH * 128, static_cast<int>(s.h * a.T + s.lo), x / NH);
          }
          __syncwarp();
          return true;
        });
  } else if (warp == kMmaWarp) {
    // ---- products
    const uint32_t id_s = idesc_f8(kTile, false, false), id_o = idesc_f8(d, false, true);
    const uint32_t q0 = smem_addr(smem), r0 = smem_addr(ring);
    int seg = 0, tile = 0;  // tile: whose S is next
    bool ok = true;
#pragma unroll 1
    while (ok && walk.next(p, cs.plan, g)) {
      ok = wait_warp(rs, &cs.qfull, seg & 1);
      ++seg;
      // S of B - 1 tiles ahead, then O of this one
      const int end = gt + g.t1 - g.t0;
#pragma unroll 1
      for (int j = g.t0 - (B - 1); ok && j < g.t1; ++j) {
        if (tile < end) {
          const int slot = tile % S;
          ok = wait_warp(rs, &rs.kfull[slot], (tile / S) & 1);
          if (!ok) break;
          tc_fence_after_sync();
          if (elect_one()) {
            const uint32_t s = tmem + Sh::kColS + tile % B * kTile, k0 = r0 + slot * Sh::kStage;
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
            mma_commit(&cs.sfull[tile % B]);
            mma_commit(&rs.kfree[slot]);
          }
          __syncwarp();
          ++tile;
        }
        if (j < g.t0) continue;
        const int slot = gt % S;
        ok = wait_warp(rs, &rs.vfull[slot], (gt / S) & 1) && wait_warp(rs, &cs.pready[gt & 1], (gt >> 1) & 1);
        if (!ok) break;
        tc_fence_after_sync();
        const int n = j == 0 ? kTile : min(kTile, g.len - (j - 1) * kTile);
        if (elect_one()) {
          const uint32_t w = tmem + Sh::kColS + gt % B * kTile, v0 = r0 + slot * Sh::kStage + NH * kHalf;
          uint32_t acc = j != g.t0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (32 * k >= n) continue;
            const uint64_t b = desc_mn(v0 + k * 4096);
#pragma unroll
            for (int term = 0; term < 2; ++term) {
              mma_f8_ts(tmem + kColO, w + k / 2 * 64 + k % 2 * 16 + term * 8, b, term == 0 ? id_o : id_o | kAE5m2, acc);
              acc = 1;
            }
          }
          mma_commit(&rs.vfree[slot]);
          mma_commit(&cs.pvdone[gt & 1]);
        }
        __syncwarp();
        ++gt;
      }
    }
  } else {
    // ---- softmax: a warp has lanes 32 (w % 4) .. and half of the tokens, of its set's tiles (even or odd ones)
    const int quarter = warp & 3, hf = (warp >> 2) & 1, set = warp >> 3, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float factor = a.scale * 1.4426950408889634f;  // scores in powers of two
    auto all_sync = [] { named_bar_sync<1, kSoftThreads>(); };
    int turn = 0;
    auto pair_sync = [&] { asm volatile("bar.sync %0, 64;" ::"r"(2 + (warp & 3) + 4 * set) : "memory"); };
#pragma unroll 1
    for (; walk.next(p, cs.plan, g); turn ^= 1) {
      // tree and units
      const int rows = min(kTile, g.N * G - g.m * kTile);
      if (t == 0) ds.bad_tree = 0, ds.no_number = 0, cs.bad[turn] = 0, cs.segment = g;
      all_sync();
      load_tree(p, ds, g, t);
      if (t < kMaxNodes) {
        const bool in = t < g.N;
        const int64_t at = static_cast<int64_t>(g.h) * a.T + g.lo + t;
        int v = in ? p.v_units[at] : 0;
        ds.ks[t] = in ? pow2(p.k_units[at]) : 1.f;
        if (v >= kNone / 2) v -= kNone, atomicOr(&ds.no_number, 1ull << t);
        ds.lv[t] = static_cast<float>(v);
        ds.il[t] = in ? pow2(-v) : 0.f;
      }
      float rowf = 0.f;
      if (row < rows) rowf = pow2(p.q_units[(static_cast<int64_t>(g.h) * a.T + g.lo) * G + g.m * kTile + row]) * factor;
      all_sync();
      see(ds, g, t);
      all_sync();

      const bool bad_tree = ds.bad_tree != 0, alive = quarter * 32 < rows;
      float m = -INFINITY, sum = 0.f;
      const int t0 = g.t0, t1 = g.t1, len = g.len;
#pragma unroll 1
      for (int j = t0; j < t1; ++j, ++gt) {
        const int slot = gt % S;
        const Consts& cc = rs.c[slot];
        if ((gt & 1) != set) continue;
        // after a wait that gave up a warp still comes by every barrier of threads
        const uint32_t sc = lanes + Sh::kColS + gt % B * kTile;
        bool ok = wait_warp(rs, &cs.sfull[gt % B], (gt / B) & 1) && wait_warp(rs, &rs.cfull[slot], (gt / S) & 1);
        // the set's last product, so that none of its phases is missed (with two tiles of S, S itself came behind it)
        if (B > 2 && gt >= 2) wait_warp(rs, &cs.pvdone[set], ((gt - 2) >> 1) & 1);
        tc_fence_after_sync();
        if (cc.bad != 0) cs.bad[turn] = 1;
        const int n = j == 0 ? kTile : min(kTile, len - (j - 1) * kTile);
        if (n < kTile && ok) ok = wait_warp(rs, &rs.vfull[slot], (gt / S) & 1);
        if (n < kTile && ok) {  // values behind the context: anything, so none
          unsigned char* v = ring + slot * Sh::kStage + NH * kHalf;
#pragma unroll 1
          for (int i = n * 8 + (t & 255); i < ((n + 31) & ~31) * 8; i += 32 * kSetWarps)
#pragma unroll
            for (int x = 0; x < NH; ++x) *reinterpret_cast<uint4*>(v + x * kHalf + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        // the tile's maxima
        float top = -INFINITY, low = INFINITY, rf = rowf;  // low: of the context's maxima by 16 tokens
        if (alive && j == 0) {  // the draft's scores go back in the place of the products; the tile's constants are 1 and 0
          rf = 1.f;
          const Segment& now = cs.segment;
          const uint32_t seen = static_cast<uint32_t>(ds.seen[min(now.m * kTile + row, now.N * G - 1) / G] >> (32 * hf));
#pragma unroll 1
          for (int x = 32 * hf; x < 32 * hf + 32; x += 16) {
            uint32_t r[2][16];
            tmem_ld16_async(sc + x, r[0]);
            tmem_ld16_async(sc + 64 + x, r[1]);
            tmem_wait16(r[0]);
            tmem_wait16(r[1]);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float y = (__uint_as_float(r[0][i]) + __uint_as_float(r[1][i])) * (ds.ks[x + i] * rowf) + ds.lv[x + i];
              const float s = (seen >> (x + i - 32 * hf)) & 1 ? y : -INFINITY;
              top = fmaxf(top, s);
              r[0][i] = __float_as_uint(s);
            }
            tmem_st16(sc + x, r[0]);
            tmem_st16(sc + 64 + x, r[0]);
          }
          tmem_wait_st();
          tc_fence_before_sync();
        } else if (alive) {
#pragma unroll 1
          for (int x = 64 * hf; x < 64 * hf + 64; x += 32) {
            uint32_t r[32];
            float* s = reinterpret_cast<float*>(r);
            tmem_ld32(sc + x, r);
            tmem_wait32(r);
            if (n < kTile) {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = x + i < n ? s[i] : -INFINITY;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float y[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                y[i] = fmaxf(fmaxf(s[16 * q + i], s[16 * q + 4 + i]), fmaxf(s[16 * q + 8 + i], s[16 * q + 12 + i]));
              const float z = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
              const float high = fmaf(z, fmaxf(cc.ks[x / 16 + q] * rowf, kLeast), cc.lv[x / 16 + q]);
              top = fmaxf(top, high);
              if (x + 16 * q + 16 <= n) low = fminf(low, high);
            }
          }
        }
        // the rows' references, in the order of the tiles; both halves of a row have read the last one before it moves on
        const bool start = j - t0 < 2;
        float now = m;
        if (!start) {
          wait_warp(rs, &cs.mdone[set ^ 1], ((gt - 1) >> 1) & 1);
          now = cs.ref[row];
        }
        cs.half[set][hf][row] = top;
        if (start) cs.low[set][hf][row] = low;
        pair_sync();
        top = fmaxf(top, cs.half[set][hf ^ 1][row]);
        if (start) low = fminf(low, cs.low[set][hf ^ 1][row]);
        bool grown = false;
        float down = 1.f;
        if (start) {  // the larger of the first two
          // The second tile's set waits for the first one's maxima before it says that its own are there: the other way
          // round the first set could go on to its next phase, of the same parity as the one before, past a warp that
          // has yet to look.
          if (j != t0) wait_warp(rs, &cs.mdone[set ^ 1], ((gt - 1) >> 1) & 1);
          if (hf == 0) cs.first[set][row] = top;
          warp_arrive(&cs.mdone[set]);
          if (t1 - t0 > 1) {
            if (j == t0) wait_warp(rs, &cs.mdone[set ^ 1], ((gt + 1) >> 1) & 1);
            top = fmaxf(top, cs.first[set ^ 1][row]);
            low = fminf(low, fminf(cs.low[set ^ 1][0][row], cs.low[set ^ 1][1][row]));
          }
          m = top - low > kFar ? top : top + kRoom;
          if (hf == 0 && j == t0) cs.ref[row] = m;  // the other set has it too, and reads this two tiles later
        } else {
          if (now != m) sum *= ex2(m - now), m = now;
          grown = top > m + kGrowth;
          if (grown) {
            down = ex2(m - top);
            sum *= down;
            m = top;
            if (hf == 0) cs.ref[row] = top;
          }
          warp_arrive(&cs.mdone[set]);
        }
        if (alive && __any_sync(kFull, grown)) {
          wait_warp(rs, &cs.pvdone[set ^ 1], ((gt - 1) >> 1) & 1);
          tc_fence_after_sync();
          const int mid = (d / 16 + 1) / 2 * 16;
#pragma unroll 1
          for (int x = hf ? mid : 0; x < (hf ? d : mid); x += 16) {
            uint32_t o[16];
            tmem_ld16_async(lanes + kColO + x, o);
            tmem_wait16(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * down);
            tmem_st16(lanes + kColO + x, o);
          }
          tmem_wait_st();
        }
        if (alive) {
          if (j == 0) tc_fence_after_sync();  // the other half's scores of the draft
          // weights, 32 tokens at a time; their terms take the place of products that have been read
#pragma unroll 1
          for (int y = 0; y < 2; ++y) {
            const int at = 64 * hf + 32 * y;
            uint32_t r[32];
            float* s = reinterpret_cast<float*>(r);
            tmem_ld32(sc + at, r);
            tmem_wait32(r);
            if (n < kTile) {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = at + i < n ? s[i] : -INFINITY;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float f = fmaxf(cc.ks[at / 16 + q] * rf, kLeast), e = cc.lv[at / 16 + q] + (kBias - m);
              float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
              uint32_t hi[4], lo[4];  // four codes each
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float* w = s + 16 * q + 4 * i;
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                  const float2 y = fma2(make_float2(w[k], w[k + 1]), make_float2(f, f), make_float2(e, e));
                  w[k] = ex2(y.x), w[k + 1] = ex2(y.y);
                  part[k / 2] = add2(part[k / 2], make_float2(w[k], w[k + 1]));
                }
                uint32_t h0, l0, h1, l1;
                weight_terms(w[0], w[1], h0, l0);
                weight_terms(w[2], w[3], h1, l1);
                hi[i] = h0 | (h1 << 16);
                lo[i] = __byte_perm(l0, l1, 0x7531);
              }
              sum = fmaf((part[0].x + part[0].y) + (part[1].x + part[1].y), cc.il[at / 16 + q], sum);
              tmem_st4(sc + 64 * hf + 16 * y + 4 * q, hi);
              tmem_st4(sc + 64 * hf + 16 * y + 8 + 4 * q, lo);
            }
            if (j == 0 && hf == 0) {
#pragma unroll
              for (int i = 0; i < 32; ++i) sum = fmaf(s[i], ds.il[at + i], sum);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before_sync();
        warp_arrive(&cs.pready[set]);
      }

      // ---- outputs
      g = cs.segment;
      const int row0 = g.m * kTile, node = min(row0 + row, g.N * G - 1) / G, part = set * 2 + hf;
      const int per = (d / 16 + kParts - 1) / kParts * 16, col0 = min(d, part * per), col1 = min(d, col0 + per);  // O's columns of a warp
      const bool whole = g.t0 == 0 && g.t1 == g.tiles;
      // the last two tiles in their order: a set that did not take the last one may come here two phases early
      bool ok = gt < 2 || wait_warp(rs, &cs.pvdone[gt & 1], ((gt - 2) >> 1) & 1);
      ok = wait_warp(rs, &cs.pvdone[(gt - 1) & 1], ((gt - 1) >> 1) & 1) && ok;
      tc_fence_after_sync();
      const unsigned long long no_number = ds.no_number;  // before the next segment's
      cs.sum[part][row] = m == -INFINITY ? 0.f : sum * ex2(m - cs.ref[row]);  // a set may have had no tile
      all_sync();
      m = cs.ref[row];
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kParts; ++i) sum += cs.sum[i][row];
      const bool bad = bad_tree || cs.bad[turn] != 0;
      const float inv = 1.f / sum;
      if (ok && alive) {
        const int64_t out = ((static_cast<int64_t>(g.lo) + node) * a.Hq + g.h * G + (row0 + row) % G) * d;
        const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (g.t0 == 0 ? 1 : 0);
        float* po = p.part_o + (piece * p.rows_cap + row) * d;
        const bool write = row < min(kTile, g.N * G - row0) && !bad;
        const unsigned long long none = g.t0 == 0 && write ? no_number & ds.seen[node] : 0;
#pragma unroll 1
        for (int x = col0; x < col1; x += 16) {
          uint32_t o[16];
          tmem_ld16_async(lanes + kColO + x, o);
          tmem_wait16(o);
          float y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(o[i]) * inv;
          if (none != 0) {  // values of the node's path that are no numbers
#pragma unroll 1
            for (unsigned long long q = none; q != 0; q &= q - 1) {
              const uint16_t* v = static_cast<const uint16_t*>(a.v) + (static_cast<int64_t>(g.lo) + __ffsll(q) - 1) * a.v_stride +
                                  static_cast<int64_t>(g.h) * d + x;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if ((v[i] & 0x7f80) == 0x7f80) y[i] = NAN;
            }
          }
          if (!whole) {
            if (!write) continue;
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(po + x + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            continue;
          }
          uint32_t u[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&v);
          }
          if (p.wide_o) {  // by way of the queries' place, so that rows are written as such
            unsigned char* to = smem + row * (NH * 256);
            *reinterpret_cast<uint4*>(to + (((x >> 3) ^ (row & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
            *reinterpret_cast<uint4*>(to + ((((x >> 3) + 1) ^ (row & 7)) << 4)) = make_uint4(u[4], u[5], u[6], u[7]);
          } else if (write) {
#pragma unroll
            for (int i = 0; i < 16; ++i) static_cast<__nv_bfloat16*>(a.o)[out + x + i] = __float2bfloat16_rn(y[i]);
          }
        }
        if (write && !whole && part == 0) p.part_lse[piece * p.rows_cap + row] = m + log2f(sum);
        tc_fence_before_sync();
      }
      if (whole && p.wide_o) {
        all_sync();
        if (ok && !bad) {
          constexpr int kEach = kTile / kSoftWarps;
          int head = (row0 + warp * kEach) % G;
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.o) + ((static_cast<int64_t>(g.lo) + (row0 + warp * kEach) / G) * a.Hq + g.h * G) * d;
#pragma unroll 4
          for (int i = warp * kEach; i < min(min(kTile, g.N * G - row0), warp * kEach + kEach); ++i) {
            if (8 * lane < d)
              reinterpret_cast<uint4*>(to + head * d)[lane] = *reinterpret_cast<const uint4*>(smem + i * (NH * 256) + ((lane ^ (i & 7)) << 4));
            if (++head == G) head = 0, to += static_cast<int64_t>(a.Hq) * d;
          }
        }
      }
      if (ok && t == 0) report(p, mine, walk, g, min(kTile, g.N * G - row0), bad_tree, bad);
      fence_proxy_async_smem();  // the queries' place is read from and written to here
      warp_arrive(&cs.qfree);
    }
  }

  __syncthreads();
  if (rs.fail != 0) {
    if (t == 0) {  // some of these may be written
      walk = mine.walk;
      while (walk.next(p, cs.plan, g)) atomicOr(a.status + g.r, TREEWY_STATUS_TIMEOUT);
    }
    if (warp == kLoadWarp) {
      drain_copies(rs.kfull, armed);
      if (queries > 0) mbar_wait_for(&cs.qfull, (queries - 1) & 1, 20000000ull);
    }
    if (warp == kLoadWarp + 1) drain_copies(rs.vfull, armed);
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
// its own sum, by the weights 2^lse.  A CTA takes eight rows, a warp each, a
// lane eight columns; or one row (`many`), whose parts the warps share.  Bound
// by three loads in a row (the item, its parts' sums, their outputs): 5 us.
constexpr int kJoinRows = 8;
__global__ void __launch_bounds__(32 * kJoinRows) attend_join_kernel(const __grid_constant__ Params p, int many) {
  after_previous();
  __shared__ float acc[kJoinRows][256], wsum[kJoinRows];
  const int w = blockIdx.y, t = threadIdx.x, warp = t >> 5, lane = t & 31, d = p.a.cache.d;
  const int4 rec = *reinterpret_cast<const int4*>(p.record + 8 * w);
  const int row = many ? blockIdx.x : blockIdx.x * kJoinRows + warp;
  if (rec.x == 0 || row >= rec.z) return;
  const int4 item = *reinterpret_cast<const int4*>(p.record + 8 * w + 4);
  const int parts = rec.y - w + 1;
  auto part_of = [&](int i) { return (2 * static_cast<int64_t>(w + i) + (i == 0 ? 1 : 0)) * p.rows_cap + row; };
  float top = -INFINITY;
#pragma unroll 1
  for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.part_lse[part_of(i)]);  // NaN comes by way of the weights
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  if (top == INFINITY) return;  // a part was refused, in all of its rows
  float sum = 0.f, y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = 0.f;
#pragma unroll 8
  for (int i = many ? warp : 0; i < parts; i += many ? kJoinRows : 1) {
    const int64_t at = part_of(i);
    const float f = exp2f(p.part_lse[at] - top);
    sum += f;
    if (8 * lane < d) {
      const float4* o = reinterpret_cast<const float4*>(p.part_o + at * d + 8 * lane);
      const float4 u = o[0], v = o[1];
      y[0] = fmaf(f, u.x, y[0]); y[1] = fmaf(f, u.y, y[1]); y[2] = fmaf(f, u.z, y[2]); y[3] = fmaf(f, u.w, y[3]);
      y[4] = fmaf(f, v.x, y[4]); y[5] = fmaf(f, v.y, y[5]); y[6] = fmaf(f, v.z, y[6]); y[7] = fmaf(f, v.w, y[7]);
    }
  }
  const int rr = item.y * kTile + row, node = rr / p.G;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.o) +
                       ((static_cast<int64_t>(item.z) + node) * p.a.Hq + item.x * p.G + rr - node * p.G) * d;
  if (many) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[warp][8 * lane + e] = y[e];
    if (lane == 0) wsum[warp] = sum;
    __syncthreads();
    if (t < d) {
      float z = 0.f, n = 0.f;
#pragma unroll
      for (int i = 0; i < kJoinRows; ++i) z += acc[i][t], n += wsum[i];
      out[t] = __float2bfloat16_rn(z / n);
    }
  } else if (8 * lane < d) {
    const float inv = 1.f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) out[8 * lane + e] = __float2bfloat16_rn(y[e] * inv);
  }
}

int row_tiles_of(const treewy_attn& a) {
  return static_cast<int>((static_cast<int64_t>(a.max_nodes) * (a.Hq / a.cache.Hkv) + kTile - 1) / kTile);
}
bool few_rows(const treewy_attn& a) { return static_cast<int64_t>(a.max_nodes) * (a.Hq / a.cache.Hkv) <= kFewRows; }
// Whether the tiles are put in a row.  For few rows always: 64 drafts of 4 nodes
// on 8 key heads 94 us (an item per CTA: 114), 64 tokens 64 us (69).  Otherwise
// where there are few items, for which a CTA apiece would leave SMs idle, and
// fewer where they are row tiles of one context, which L2 then serves to
// neighbours.  16-node trees of one row tile: 57 us with 128 items (61), 70 with
// 160 (61), 94 with 256 (76); 64-node trees of 4 row tiles: 64 us with 72 items
// (73), 76 with 96 (75), 83 with 128 (75).
bool listed(const treewy_attn& a) {
  const int mt = row_tiles_of(a);
  const int64_t items = static_cast<int64_t>(a.R) * a.cache.Hkv * mt;
  return a.R <= kMaxListed && (few_rows(a) || items <= (mt == 1 ? kMaxPieces : kMaxPieces / 2)) &&
         items * (2 + a.max_context / kTile) < (int64_t(1) << 31);
}
int rows_cap(const treewy_attn& a) {
  return static_cast<int>(std::min<int64_t>(kTile, static_cast<int64_t>(a.max_nodes) * (a.Hq / a.cache.Hkv)));
}

bool make_map(CUtensorMap* map, const void* codes, int d, int rows, int64_t blocks, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(blocks)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(d) * static_cast<cuuint64_t>(rows)};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows), 1}, ones[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A 16-byte aligned address beside p, for a map that nothing is read through.
void* any16(const void* p) { return reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15)); }
uint64_t up256(uint64_t n) { return (n + 255) & ~uint64_t(255); }

// Whether the longest contexts are begun first: where an item is a CTA's, up to a number of requests behind which the last
// CTAs matter little.
bool ordered(const treewy_attn& a) { return !few_rows(a) && !listed(a) && a.R <= kMaxOrdered; }

// Where things are in the workspace: the parts of items in several pieces, then the terms.
struct Workspace {
  uint64_t record, lse, q_terms, k_terms, v_terms, q_units, k_units, v_units, order, end;
  explicit Workspace(const treewy_attn& a) {
    const uint64_t rows = listed(a) ? static_cast<uint64_t>(kMaxPieces) * 2 * rows_cap(a) : 0;
    const uint64_t T = few_rows(a) ? 0 : static_cast<uint64_t>(std::max<int64_t>(a.T, 1)), q = T * a.Hq, kv = T * a.cache.Hkv, d = a.cache.d;
    record = up256(rows * d * 4);
    lse = record + (rows > 0 ? kMaxPieces * 8 * 4 : 0);
    q_terms = up256(lse + rows * 4);
    k_terms = up256(q_terms + 2 * q * d);
    v_terms = up256(k_terms + 2 * kv * d);
    q_units = up256(v_terms + 2 * kv * d);
    k_units = up256(q_units + 2 * q);
    v_units = up256(k_units + 2 * kv);
    order = up256(v_units + 2 * kv);
    end = order + (ordered(a) ? 4 * static_cast<uint64_t>(a.R) : 0);
  }
};

template <int NH>
cudaError_t launch(const Params& p, const Maps& maps, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(attend_tc_kernel<NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NH>::kBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_after_smem(attend_tc_kernel<NH>, dim3(grid), kThreads, Shape<NH>::kBytes, stream, p, maps);
}

}  // namespace

bool attend_on_tensor_cores(const treewy_attn& a) {
  return a.qkv_dtype == TREEWY_DTYPE_BF16 && a.o_dtype == TREEWY_DTYPE_BF16 && a.cache.d % 16 == 0 &&
         (a.flags & TREEWY_FLAG_FORCE_GENERIC) == 0;
}

uint64_t attend_workspace(const treewy_attn& a) { return a.R == 0 || !attend_on_tensor_cores(a) ? 0 : Workspace(a).end; }

cudaError_t launch_attend_tc(const treewy_attn& a, cudaStream_t stream) {
  Params p = {};
  p.a = a;
  p.G = a.Hq / a.cache.Hkv;
  p.tiles_m = row_tiles_of(a);
  p.listed = listed(a) ? 1 : 0;
  p.rows_cap = rows_cap(a);
  auto wide = [](const void* x, int64_t stride) { return reinterpret_cast<uintptr_t>(x) % 16 == 0 && stride % 8 == 0 ? 1 : 0; };
  p.wide_q = wide(a.q, a.q_stride), p.wide_k = wide(a.k, a.k_stride), p.wide_v = wide(a.v, a.v_stride), p.wide_o = wide(a.o, 0);
  const Workspace at(a);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.record = reinterpret_cast<int*>(ws + at.record);
  p.part_lse = reinterpret_cast<float*>(ws + at.lse);
  p.q_terms = ws + at.q_terms, p.k_terms = ws + at.k_terms, p.v_terms = ws + at.v_terms;
  p.q_units = reinterpret_cast<int16_t*>(ws + at.q_units);
  p.k_units = reinterpret_cast<int16_t*>(ws + at.k_units);
  p.v_units = reinterpret_cast<int16_t*>(ws + at.v_units);
  if (ordered(a) && a.T > 0) p.order = reinterpret_cast<int*>(ws + at.order);  // without rows nothing writes it
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
  const bool few = few_rows(a);
  const int64_t T = std::max<int64_t>(a.T, 1);
  if (!few && T * (a.Hq + 2 * static_cast<int64_t>(a.cache.Hkv)) > 0x7fffffff) return cudaErrorNotSupported;
  Maps maps;
  // a cache without pages has none to read: its requests are short or refused
  const treewy_cache& c = a.cache;
  const int64_t blocks = std::max<int64_t>(c.num_pages, 1) * c.Hkv;
  const void* any = c.num_pages > 0 ? nullptr : a.node_offset;
  if (!make_map(&maps.k, any ? any16(any) : c.k, c.d, c.page_len, blocks, c.page_len) ||
      !make_map(&maps.v, any ? any16(any) : c.v, c.d, c.page_len, blocks, c.page_len))
    return cudaErrorUnknown;
  cudaError_t e;
  if (few) {
    e = launch_attend_few(p, maps.k, maps.v, grid, stream);
  } else {
    if (!make_map(&maps.q_terms, p.q_terms, c.d, static_cast<int>(T * a.Hq), 2, kTile) ||
        !make_map(&maps.k_terms, p.k_terms, c.d, static_cast<int>(T * c.Hkv), 2, kMaxNodes) ||
        !make_map(&maps.v_terms, p.v_terms, c.d, static_cast<int>(T * c.Hkv), 2, kMaxNodes))
      return cudaErrorUnknown;
    const int groups = (a.Hq + 2 * c.Hkv + kSplitRows - 1) / kSplitRows;
    if (a.T > 0) {
      const int64_t ctas = std::min<int64_t>((a.T * groups + 7) / 8, 16 * kMaxPieces);
      e = launch_after(attend_split_kernel, dim3(static_cast<unsigned>(ctas)), kSplitThreads, stream, p, groups);
      if (e != cudaSuccess) return e;
    }
    e = c.d > 128 ? launch<2>(p, maps, grid, stream) : launch<1>(p, maps, grid, stream);
  }
  if (e != cudaSuccess || !p.listed) return e;
  // 256K tokens of one request in 57 us, 71 by eight rows to a CTA; 64 tokens of eight rows 62.5 us against 64; but 64-node
  // trees of 8 requests 78 us against 61
  const int many = p.rows_cap <= 8 || static_cast<int64_t>(a.R) * c.Hkv * p.tiles_m * 8 <= kMaxPieces ? 1 : 0;
  return launch_after(attend_join_kernel, dim3(many ? p.rows_cap : (p.rows_cap + kJoinRows - 1) / kJoinRows, grid), 32 * kJoinRows, stream, p, many);
}

}  // namespace treewy
