// attend_tc.cu -- attention over pages of e4m3 keys and values and the draft's
// own ones on the 5th-generation tensor cores (tcgen05, TMEM, TMA), for bf16
// rows and outputs, head sizes that are multiples of 16, and drafts of more
// than 32 rows; and what joins the pieces of an item.
//
// A tile is 128 rows, (node, query head) pairs that share a key head, times
// 128 tokens.  TMEM lanes are rows, so that a softmax thread owns a part of a
// row:
//
//   S = Q K^T          Q's terms and K in shared memory, S in TMEM, twice
//   w                  two terms, back in TMEM in the place of S
//   O += w V           V in shared memory as it is stored (rows along the sum)
//
// The draft's keys and values take two tokens of its tile each, one per term;
// the ancestors are a mask of bits.
//
//   softmax warps  queries and draft to e4m3; softmax; outputs
//   loading warps  page table, scales and pages (TMA): keys, and values
//   issuing warp   the products: S of the next tile before O of this one
#include "attend_tc.cuh"

namespace treewy {
namespace {

constexpr int kSoftWarps = 8, kLoadWarp = kSoftWarps, kMmaWarp = kLoadWarp + 2;
constexpr int kSoftThreads = 32 * kSoftWarps, kThreads = 32 * (kMmaWarp + 1);
constexpr int kParts = kSoftWarps / 4, kCols = kTile / kParts, kNodes = kCols / 2;  // of a row, by warp
constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;

// NH: halves of 128 columns of a head.
template <int NH>
struct Shape {
  static constexpr uint32_t kQBytes = 2 * NH * kHalf, kStage = 2 * NH * kHalf;  // hi and lo; K and V
  static constexpr int kStages = NH == 2 ? 2 : 5;
  static constexpr uint32_t kBytes = kQBytes + kStages * kStage + 1024;
};

template <int S>
struct AttendSmem {
  RingSmem<S> ring;
  uint64_t sfull[2], pready[2], pvdone[2], qready, drain;
  float top[2][kParts * kTile];  // maxima (and sums) of the parts of rows; two sets in turn
  uint32_t tmem;
  Segment segment;               // the softmax warps' current one
  DraftSmem draft;
  PlanSmem plan;
};

template <int NH>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using Sh = Shape<NH>;
  constexpr int S = Sh::kStages;
  extern __shared__ unsigned char raw_smem[];
  __shared__ AttendSmem<S> cs;
  RingSmem<S>& rs = cs.ring;
  DraftSmem& ds = cs.draft;
  unsigned char* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  unsigned char* ring = smem + Sh::kQBytes;
  const treewy_attn& a = p.a;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, d = a.cache.d, G = p.G;

  // ---- set-up, while the kernel before may still run
  if (t == 0) {
    init_ring(rs);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&cs.sfull[i], 1);
      mbar_init(&cs.pready[i], kSoftWarps);
      mbar_init(&cs.pvdone[i], 1);
    }
    mbar_init(&cs.qready, 1);
    mbar_init(&cs.drain, 1);
    fence_mbarrier_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&cs.tmem, kTmemCols);
    tmem_relinquish();
  }
  after_previous();
  const Part mine = make_plan<kThreads>(p, cs.plan, rs);
  const uint32_t tmem = cs.tmem;

  Walk walk = mine.walk;
  Segment g;
  int armed = 0;
  int gt = 0;  // tiles so far

  if (warp == kLoadWarp) {
    armed = load_pages<false, NH, S>(p, cs, rs, walk, ring, kmap);
  } else if (warp == kLoadWarp + 1) {
    armed = load_pages<true, NH, S>(p, cs, rs, walk, ring, vmap);
  } else if (warp == kMmaWarp) {
    // ---- products
    const uint32_t id_s = idesc_f8(kTile, false, false), id_o = idesc_f8(d, false, true);
    const uint32_t q0 = smem_addr(smem), r0 = smem_addr(ring);
    int seg = 0;
    bool ok = true;
#pragma unroll 1
    while (ok && walk.next(p, cs.plan, g)) {
      ok = wait_warp(rs, &cs.qready, seg & 1);
      ++seg;
      // S of the next tile, then O of the last
#pragma unroll 1
      for (int j = g.t0 - 1; ok && j < g.t1; ++j) {
        if (j + 1 < g.t1) {
          const int tile = gt + (j >= g.t0 ? 1 : 0), slot = tile % S;
          ok = wait_warp(rs, &rs.kfull[slot], (tile / S) & 1);
          if (!ok) break;
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
            mma_commit(&rs.kfree[slot]);
          }
          __syncwarp();
        }
        if (j < g.t0) continue;
        const int slot = gt % S;
        ok = wait_warp(rs, &rs.vfull[slot], (gt / S) & 1) && wait_warp(rs, &cs.pready[gt & 1], (gt >> 1) & 1);
        if (!ok) break;
        tc_fence_after_sync();
        const int n = j == 0 ? kTile : min(kTile, g.len - (j - 1) * kTile);
        if (elect_one()) {
          const uint32_t w = tmem + kColS + (gt & 1) * kTile, v0 = r0 + slot * Sh::kStage + NH * kHalf;
          uint32_t acc = j != g.t0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (32 * k >= n) continue;
            const uint64_t b = desc_mn(v0 + k * 4096);
#pragma unroll
            for (int term = 0; term < 2; ++term) {
              mma_f8_ts(tmem + kColO, w + term * 32 + k * 8, b, term == 0 ? id_o | kAE5m2 : id_o, acc);
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
    // ---- softmax: warp w has lanes 32 (w % 4) .. and of their rows the tokens from kCols (w / 4)
    const int quarter = warp & 3, share = warp >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int per = (d / 16 + kParts - 1) / kParts * 16;  // O's columns of a warp
    const int col0 = min(d, share * per), col1 = min(d, col0 + per);
    const float factor = a.scale * 1.4426950408889634f;  // scores in powers of two
    auto all_sync = [] { named_bar_sync<1, kSoftThreads>(); };
    // `op` over the parts of this thread's row
    auto over_row = [&](int set, float v, auto op) {
      cs.top[set][share * kTile + row] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(2 + quarter), "n"(32 * kParts) : "memory");
      v = cs.top[set][row];
#pragma unroll
      for (int i = 1; i < kParts; ++i) v = op(v, cs.top[set][i * kTile + row]);
      return v;
    };
#pragma unroll 1
    while (walk.next(p, cs.plan, g)) {
      // queries and tree
      const int rows = min(kTile, g.N * G - g.m * kTile);
      if (t == 0) ds.bad_tree = 0, ds.no_number = 0, cs.segment = g;
      if (g.t0 == 0) wait_warp(rs, &rs.cfull[gt % S], (gt / S) & 1);  // the stage is free
      all_sync();
      load_tree(p, ds, g, t);
      unsigned char* draft = ring + (gt % S) * Sh::kStage;
      if (g.t0 == 0) {  // what the draft's tile has behind its values
        const int last = g.N % kNodes;
        if (last != 0) {
          const int at = g.N / kNodes * kCols;
          zero_rows<kSoftThreads>(draft + NH * kHalf, NH, kHalf, at + last, at + kNodes);
          zero_rows<kSoftThreads>(draft + NH * kHalf, NH, kHalf, at + kNodes + last, at + kCols);
        }
        zero_rows<kSoftThreads>(draft + NH * kHalf, NH, kHalf, (g.N + kNodes - 1) / kNodes * kCols, kTile);
        if (t >= g.N && t < kMaxNodes) ds.ks[t] = 1.f, ds.lv[t] = ds.il[t] = 0.f;
      }
      fill_rows<NH, kSoftWarps, 8>(p, ds, g, rows, factor, [&](int kind, int i, int ln, uint2 hi, uint2 lo) {
        unsigned char* tile = kind == 0 ? smem : kind == 1 ? draft : draft + NH * kHalf;
        const int token = i / kNodes * kCols + i % kNodes;
        *operand8(tile, kind == 0 ? i : token, ln, kHalf) = hi;
        *operand8(kind == 0 ? smem + NH * kHalf : tile, kind == 0 ? i : token + kNodes, ln, kHalf) = lo;
      });
      fence_proxy_async_smem();
      all_sync();
      if (t == 0) {
        arrive(&cs.qready);
        if (g.t0 == 0) {
          arrive(&rs.kfull[gt % S]);
          arrive(&rs.vfull[gt % S]);
        }
      }
      see(ds, g, t);
      all_sync();

      const bool bad_tree = ds.bad_tree != 0, alive = quarter * 32 < rows;
      bool bad = bad_tree;
      const float rowf = row < rows ? ds.rowf[row] : 0.f;
      float m = -INFINITY, sum = 0.f;
      const int t0 = g.t0, t1 = g.t1, len = g.len;
#pragma unroll 1
      for (int j = t0; j < t1; ++j, ++gt) {
        const int slot = gt % S, b = gt & 1;
        const Consts& cc = rs.c[slot];
        // after a wait that gave up a warp still comes by every barrier of threads
        bool ok = wait_warp(rs, &cs.sfull[b], (gt >> 1) & 1) && wait_warp(rs, &rs.cfull[slot], (gt / S) & 1);
        tc_fence_after_sync();
        bad |= cc.bad != 0;
        const int n = j == 0 ? kTile : min(kTile, len - (j - 1) * kTile);
        if (n < kTile && ok) ok = wait_warp(rs, &rs.vfull[slot], (gt / S) & 1);
        if (n < kTile && ok) {  // values behind the context: anything, so none
          const int end = (n + 31) & ~31;
          unsigned char* v = ring + slot * Sh::kStage + NH * kHalf;
#pragma unroll 1
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
#pragma unroll
            for (int x = 0; x < kCols; x += 32) tmem_ld32(sc + share * kCols + x, r + x);
#pragma unroll
            for (int x = 0; x < kCols; x += 32) tmem_wait32(r + x);
          }
          float rf = rowf;
          if (j == 0) {  // scores here; the loading warp's constants of the tile are 1 and 0
            rf = 1.f;
            const Segment& now = cs.segment;
            const uint32_t seen =
                static_cast<uint32_t>(ds.seen[min(now.m * kTile + row, now.N * G - 1) / G] >> (kNodes * share));
#pragma unroll
            for (int i = 0; i < kNodes; ++i) {
              const int q = share * kNodes + i;
              const float y = (s[i] + s[kNodes + i]) * (ds.ks[q] * rowf) + ds.lv[q];
              s[i] = s[kNodes + i] = (seen >> i) & 1 ? y : -INFINITY;
            }
          } else if (n < kTile) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) s[i] = share * kCols + i < n ? s[i] : -INFINITY;
          }
          float f[kCols / 16], top = -INFINITY;
#pragma unroll
          for (int q = 0; q < kCols / 16; ++q) {
            float x = s[16 * q];
#pragma unroll
            for (int i = 1; i < 16; ++i) x = fmaxf(x, s[16 * q + i]);
            f[q] = fmaxf(cc.ks[share * (kCols / 16) + q] * rf, kLeast);
            top = fmaxf(top, fmaf(x, f[q], cc.lv[share * (kCols / 16) + q]));
          }
          top = over_row(b, top, [](float x, float y) { return fmaxf(x, y); });
          if (j == t0) {
            m = top;
          } else {
            const bool grown = top > m + kGrowth;
            if (__any_sync(kFull, grown)) {
              const float down = grown ? ex2(m - top) : 1.f;
              if (grown) m = top;
              sum *= down;
              wait_warp(rs, &cs.pvdone[(gt - 1) & 1], ((gt - 1) >> 1) & 1);
              tc_fence_after_sync();
#pragma unroll 1
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
#pragma unroll
          for (int q = 0; q < kCols / 16; ++q) {
            const float e = cc.lv[share * (kCols / 16) + q] + (kBias - m);
            float part_sum = 0.f;
            uint32_t hi[4], lo[4];  // four codes each
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float* w = s + 16 * q + 4 * i;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                w[k] = ex2(fmaf(w[k], f[q], e));
                part_sum += w[k];
              }
              uint32_t h0, l0, h1, l1;
              weight_terms(w[0], w[1], h0, l0);
              weight_terms(w[2], w[3], h1, l1);
              hi[i] = __byte_perm(h0, h1, 0x7531);
              lo[i] = l0 | (l1 << 16);
            }
            sum = fmaf(part_sum, cc.il[share * (kCols / 16) + q], sum);
            tmem_st4(sc + share * (kCols / 4) + 4 * q, hi);
            tmem_st4(sc + 32 + share * (kCols / 4) + 4 * q, lo);
          }
          if (j == 0) {
#pragma unroll
            for (int i = 0; i < kNodes; ++i) sum = fmaf(s[i], ds.il[share * kNodes + i], sum);
          }
          tmem_wait_st();
          tc_fence_before_sync();
        }
        warp_arrive(&cs.pready[b]);
      }

      // ---- outputs
      g = cs.segment;
      const int row0 = g.m * kTile, node = min(row0 + row, g.N * G - 1) / G;
      const bool whole = g.t0 == 0 && g.t1 == g.tiles;
      const bool ok = wait_warp(rs, &cs.pvdone[(gt - 1) & 1], ((gt - 1) >> 1) & 1);
      tc_fence_after_sync();
      // not the set of the last tile, which another warp may still read
      if (alive) sum = over_row(gt & 1, sum, [](float x, float y) { return x + y; });
      const float inv = 1.f / sum;
      if (ok && alive) {
        const int64_t out = ((static_cast<int64_t>(g.lo) + node) * a.Hq + g.h * G + (row0 + row) % G) * d;
        const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (g.t0 == 0 ? 1 : 0);
        float* po = p.part_o + (piece * p.rows_cap + row) * d;
        const bool write = row < rows && !bad;
        const unsigned long long none = g.t0 == 0 && write ? ds.no_number & ds.seen[node] : 0;
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
        if (write && !whole && share == 0) p.part_lse[piece * p.rows_cap + row] = m + log2f(sum);
        tc_fence_before_sync();
      }
      if (whole && p.wide_o) {
        all_sync();
        if (ok && !bad) {
          constexpr int kEach = kTile / kSoftWarps;
          int head = (row0 + warp * kEach) % G;
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.o) + ((static_cast<int64_t>(g.lo) + (row0 + warp * kEach) / G) * a.Hq + g.h * G) * d;
#pragma unroll 4
          for (int i = warp * kEach; i < min(rows, warp * kEach + kEach); ++i) {
            if (8 * lane < d)
              reinterpret_cast<uint4*>(to + head * d)[lane] = *reinterpret_cast<const uint4*>(smem + i * (NH * 256) + ((lane ^ (i & 7)) << 4));
            if (++head == G) head = 0, to += static_cast<int64_t>(a.Hq) * d;
          }
        }
      }
      if (ok && t == 0) report(p, mine, walk, g, rows, bad_tree, bad);
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
  const int w = blockIdx.y, row = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31, d = p.a.cache.d;
  const int4 rec = *reinterpret_cast<const int4*>(p.record + 8 * w);
  if (rec.x == 0 || row >= rec.z) return;
  const int4 item = *reinterpret_cast<const int4*>(p.record + 8 * w + 4);
  const int parts = rec.y - w + 1;
  auto part_of = [&](int i) { return (2 * static_cast<int64_t>(w + i) + (i == 0 ? 1 : 0)) * p.rows_cap + row; };
  float top = -INFINITY;
#pragma unroll 1
  for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.part_lse[part_of(i)]);  // NaN comes by way of the weights
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  if (top == INFINITY) return;  // a part was refused
  float sum = 0.f, y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = 0.f;
#pragma unroll 4
  for (int i = warp; i < parts; i += 8) {
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
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[warp][8 * lane + e] = y[e];
  if (lane == 0) wsum[warp] = sum;
  __syncthreads();
  if (t >= d) return;
  float z = 0.f, n = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) z += acc[i][t], n += wsum[i];
  const int rr = item.y * kTile + row, node = rr / p.G;
  static_cast<__nv_bfloat16*>(p.a.o)[((static_cast<int64_t>(item.z) + node) * p.a.Hq + item.x * p.G + rr - node * p.G) * d + t] =
      __float2bfloat16_rn(z / n);
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

template <int NH>
cudaError_t launch(const Params& p, const CUtensorMap& k, const CUtensorMap& v, unsigned grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(attend_tc_kernel<NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NH>::kBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_after_smem(attend_tc_kernel<NH>, dim3(grid), kThreads, Shape<NH>::kBytes, stream, p, k, v);
}

}  // namespace

bool attend_on_tensor_cores(const treewy_attn& a) {
  return a.qkv_dtype == TREEWY_DTYPE_BF16 && a.o_dtype == TREEWY_DTYPE_BF16 && a.cache.d % 16 == 0 &&
         (a.flags & TREEWY_FLAG_FORCE_GENERIC) == 0;
}

uint64_t attend_workspace(const treewy_attn& a) {
  if (a.R == 0 || !attend_on_tensor_cores(a) || !listed(a)) return 0;
  return static_cast<uint64_t>(kMaxPieces) * (2ull * rows_cap(a) * (a.cache.d + 1) * 4 + 8 * 4);
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
    p.record = reinterpret_cast<int*>(p.part_o + rows * a.cache.d);
    p.part_lse = reinterpret_cast<float*>(p.record + 8 * kMaxPieces);
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
  const bool few = static_cast<int64_t>(a.max_nodes) * p.G <= kFewRows;
  const cudaError_t e = few                ? launch_attend_few(p, k, v, grid, stream)
                        : a.cache.d > 128 ? launch<2>(p, k, v, grid, stream)
                                          : launch<1>(p, k, v, grid, stream);
  if (e != cudaSuccess || !p.listed) return e;
  return launch_after(attend_join_kernel, dim3(p.rows_cap, grid), 256, stream, p);
}

}  // namespace treewy
