// attend_scan.cu -- attention over pages of e4m3 keys and values and the
// draft's own ones, in f32 on the CUDA cores (treewy_attend for f32 rows or
// outputs and for head sizes that the tensor-core kernels do not take).
//
// One pass over the tokens with the running maximum and sum of the softmax: a
// cluster of eight CTAs holds 16 (node, query head) rows that share a key head;
// its CTAs take tiles of 32 tokens in turn, the context's and then the
// draft's, through shared memory (keys and values, asked for together), and
// read each other's maxima, sums and outputs at the end.
//
// Bound by a tile's chain of loads and barriers in small calls (7 trees of 1 to
// 15 nodes, 5 heads of 80, contexts of up to 700: 23 us; 32 with keys and values
// loaded one after the other), and by the loads from shared memory of the two
// products, 128 bits for four products each, in large ones (64 requests, 16
// heads of 128, 500 to 4000 tokens: 900 us).
#include <cooperative_groups.h>

#include "cache_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

namespace cg = cooperative_groups;

constexpr int kRows = 16, kTile = 32, kThreads = 128, kRanks = 8, kMaxPad = 256;
constexpr unsigned kFull = 0xffffffffu;

struct Shared {
  int parent[kMaxNodes];
  unsigned long long seen[kMaxNodes];
  int page_of[2];
  float top[kRows], sum[kRows];
  int bad;
};

// Sixteen codes times a scale.
__device__ __forceinline__ void sixteen(float* to, const uint4& w, float f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t h0 = e4m3x2_to_f16x2(u[e] & 0xffffu), h1 = e4m3x2_to_f16x2(u[e] >> 16);
    const float2 y0 = __half22float2(*reinterpret_cast<const __half2*>(&h0)), y1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
    *reinterpret_cast<float4*>(to + 4 * e) = make_float4(y0.x * f, y0.y * f, y1.x * f, y1.y * f);
  }
}
// x, or NaN where it is not finite: an infinity counts as no number whatever it is multiplied by.
__device__ __forceinline__ float number(float x) { return fabsf(x) <= 3.4028234664e38f ? x : NAN; }
// A value of a row; four that start on four elements.
__device__ __forceinline__ float load1(const void* p, int64_t at, bool bf16) { return number(load_qkv(p, at, bf16)); }
__device__ __forceinline__ float4 load4(const void* p, int64_t at, bool bf16) {
  float4 x;
  if (bf16) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at));
    x = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
  } else {
    x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at));
  }
  return make_float4(number(x.x), number(x.y), number(x.z), number(x.w));
}

__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kThreads)
    attend_scan_kernel(const __grid_constant__ treewy_attn a, int blocks, int fours) {
  after_previous();
  extern __shared__ float4 raw_smem[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const treewy_cache& c = a.cache;
  // columns in fours, the last ones filled up with zeros; rows of the tile four floats further apart
  const int t = threadIdx.x, d = c.d, P = c.page_len, pad = (d + 3) & ~3, pitch = pad + 4;
  const unsigned item = blockIdx.x / kRanks;
  const int block = static_cast<int>(item % blocks);
  const unsigned rest = item / blocks;
  const int h = static_cast<int>(rest % c.Hkv), r = static_cast<int>(rest / c.Hkv);
  const int G = a.Hq / c.Hkv;
  // the same in all of the cluster: it leaves as one
  CacheRequest q = cache_request(c, a.node_offset, r, a.T, a.max_nodes, a.max_context);
  if (q.err == 0 && !load_parents(sh.parent, a.parent, q.lo, q.N)) q.err = TREEWY_STATUS_BAD_TREE;
  if (q.err != 0) {
    if (block == 0 && h == 0 && rank == 0 && t == 0) atomicOr(a.status + r, q.err);
    return;
  }
  const int row0 = block * kRows, live = min(kRows, q.N * G - row0);
  if (live <= 0) return;
  if (t < q.N) {  // the nodes that node t sees
    unsigned long long m = 0;
    for (int p = t; p >= 0; p = sh.parent[p]) m |= 1ull << p;
    sh.seen[t] = m;
  }
  if (t == 0) sh.bad = 0;
  float* qs = reinterpret_cast<float*>(raw_smem);  // [kRows][pad], the outputs at the end
  float* tile = qs + kRows * pad;                  // [2][kTile][pitch]: keys, values
  float* weight = tile + 2 * kTile * pitch;        // [kRows][kTile]
  const bool bf16 = a.qkv_dtype == TREEWY_DTYPE_BF16;
  if (fours) {
#pragma unroll 4
    for (int x = t; x < kRows * (pad / 4); x += kThreads) {
      const int i = x / (pad / 4), col = x % (pad / 4) * 4, rr = row0 + i;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < live) y = load4(a.q, (static_cast<int64_t>(q.lo) + rr / G) * a.q_stride + (static_cast<int64_t>(h) * G + rr % G) * d + col, bf16);
      *reinterpret_cast<float4*>(qs + i * pad + col) = y;
    }
  } else {
    for (int x = t; x < kRows * pad; x += kThreads) {
      const int i = x / pad, col = x % pad, rr = row0 + i;
      qs[x] = i < live && col < d ? load1(a.q, (static_cast<int64_t>(q.lo) + rr / G) * a.q_stride +
                                                   (static_cast<int64_t>(h) * G + rr % G) * d + col, bf16)
                                  : 0.f;
    }
  }
  const int row = t / 8, sub = t % 8;  // eight threads per row
  const int node = min(row0 + row, q.N * G - 1) / G;
  float4 acc[kMaxPad / 32];
  float top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int e = 0; e < kMaxPad / 32; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int context_tiles = q.len / kTile + (q.len % kTile != 0), tiles = context_tiles + (q.N + kTile - 1) / kTile;
  // thread t's page of a tile of the context, asked for a tile ahead (a page has 16 tokens at least: two to a tile at most)
  auto page_of = [&](int j) {
    const int64_t token = static_cast<int64_t>(j) * kTile + t * P;
    return t < 2 && j < context_tiles && t * P < kTile && token < q.len ? __ldg(c.page_table + static_cast<int64_t>(r) * c.max_pages + token / P) : 0;
  };
  int page = page_of(rank);
  for (int j = rank; j < tiles; j += kRanks) {
    const bool context = j < context_tiles;
    const int t0 = (context ? j : j - context_tiles) * kTile, n = min(kTile, (context ? q.len : q.N) - t0);
    __syncthreads();  // the tile and the weights are free
    if (context) {
      if (t < 2) {
        const bool in = page >= 0 && page < c.num_pages;
        if (!in && t * P < n) sh.bad = 1;
        sh.page_of[t] = in ? page : 0;
      }
      page = page_of(j + kRanks);
      __syncthreads();
      if (sh.bad != 0) break;  // nothing of the request is written
    }
    float* value = tile + kTile * pitch;
    if (context && d % 16 == 0) {
#pragma unroll 2
      for (int x = t; x < n * (d / 16); x += kThreads) {
        const int i = x / (d / 16), col = x % (d / 16) * 16, at = t0 + i;
        const int64_t b = static_cast<int64_t>(sh.page_of[at / P - t0 / P]) * c.Hkv + h, from = (b * P + at % P) * d + col;
        const uint4 wk = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.k) + from));
        const uint4 wv = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.v) + from));
        const float fk = __ldg(c.k_scale + b), fv = __ldg(c.v_scale + b);
        sixteen(tile + i * pitch + col, wk, fk);
        sixteen(value + i * pitch + col, wv, fv);
      }
    } else if (!context && fours) {
#pragma unroll 4
      for (int x = t; x < n * (d / 4); x += kThreads) {
        const int i = x / (d / 4), col = x % (d / 4) * 4;
        const int64_t token = static_cast<int64_t>(q.lo) + t0 + i, head = static_cast<int64_t>(h) * d + col;
        const float4 k = load4(a.k, token * a.k_stride + head, bf16), v = load4(a.v, token * a.v_stride + head, bf16);
        *reinterpret_cast<float4*>(tile + i * pitch + col) = k;
        *reinterpret_cast<float4*>(value + i * pitch + col) = v;
      }
    } else {
      for (int x = t; x < n * pad; x += kThreads) {
        const int i = x / pad, col = x % pad, at = t0 + i;
        float k = 0.f, v = 0.f;
        if (col < d && context) {
          const int64_t b = static_cast<int64_t>(sh.page_of[at / P - t0 / P]) * c.Hkv + h, from = (b * P + at % P) * d + col;
          k = e4m3_to_float(__ldg(static_cast<const uint8_t*>(c.k) + from)) * __ldg(c.k_scale + b);
          v = e4m3_to_float(__ldg(static_cast<const uint8_t*>(c.v) + from)) * __ldg(c.v_scale + b);
        } else if (col < d) {
          const int64_t token = static_cast<int64_t>(q.lo) + at, head = static_cast<int64_t>(h) * d + col;
          k = load1(a.k, token * a.k_stride + head, bf16);
          v = load1(a.v, token * a.v_stride + head, bf16);
        }
        tile[i * pitch + col] = k;
        value[i * pitch + col] = v;
      }
    }
    __syncthreads();
    float s[4] = {0.f, 0.f, 0.f, 0.f}, high = -INFINITY;  // tokens sub, sub + 8, ..
#pragma unroll 2
    for (int x = 0; x < pad; x += 4) {
      const float4 u = *reinterpret_cast<const float4*>(qs + row * pad + x);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 v = *reinterpret_cast<const float4*>(tile + (sub + 8 * e) * pitch + x);
        s[e] = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, s[e]))));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = sub + 8 * e;
      const bool sees = i < n && (context || ((sh.seen[node] >> (t0 + i)) & 1));
      s[e] = sees ? number(s[e] * a.scale) : -INFINITY;  // so that -infinity is what is not seen, and no score that has passed f32
      high = fmaxf(high, s[e]);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) high = fmaxf(high, __shfl_xor_sync(kFull, high, o));
    const float now = fmaxf(top, high);
    // a draft's tile may hold nothing that this node sees; a NaN leaves the maximum alone and comes through the weights
    const float keep = top == now ? 1.f : expf(top - now);
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float w = s[e] == -INFINITY ? 0.f : expf(s[e] - now);
      weight[row * kTile + sub + 8 * e] = w;
      part += w;
    }
    top = now;
    sum = sum * keep + part;
#pragma unroll
    for (int e = 0; e < kMaxPad / 32; ++e) acc[e] = make_float4(acc[e].x * keep, acc[e].y * keep, acc[e].z * keep, acc[e].w * keep);
    __syncwarp();  // a row's weights are its own warp's
    auto add = [&](int i) {
      const float w = weight[row * kTile + i];
#pragma unroll
      for (int e = 0; e < kMaxPad / 32; ++e) {
        const int col = 4 * sub + 32 * e;
        if (col < pad) {
          const float4 v = *reinterpret_cast<const float4*>(value + i * pitch + col);
          acc[e] = make_float4(fmaf(w, v.x, acc[e].x), fmaf(w, v.y, acc[e].y), fmaf(w, v.z, acc[e].z), fmaf(w, v.w, acc[e].w));
        }
      }
    };
    if (context) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) add(i);
    } else {  // what a node does not see adds nothing to it, whatever it is
      for (int i = 0; i < n; ++i)
        if ((sh.seen[node] >> (t0 + i)) & 1) add(i);
    }
  }
  // the ranks' parts; one that had no tile, or whose tiles no row saw, has the maximum -infinity and zeros
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  __syncthreads();
  if (sub == 0) sh.top[row] = top, sh.sum[row] = sum;
#pragma unroll
  for (int e = 0; e < kMaxPad / 32; ++e)
    if (4 * sub + 32 * e < pad) *reinterpret_cast<float4*>(qs + row * pad + 4 * sub + 32 * e) = acc[e];
  cluster.sync();
  bool bad = false;
  for (int k = 0; k < kRanks; ++k) bad |= cluster.map_shared_rank(&sh, k)->bad != 0;
  if (bad && rank == 0 && t == 0) atomicOr(a.status + r, TREEWY_STATUS_BAD_PAGE);
  for (int i = rank; !bad && i < live; i += kRanks) {
    float high = -INFINITY, total = 0.f, f[kRanks];
#pragma unroll
    for (int k = 0; k < kRanks; ++k) {
      f[k] = cluster.map_shared_rank(&sh, k)->top[i];
      high = fmaxf(high, f[k]);
    }
#pragma unroll
    for (int k = 0; k < kRanks; ++k) {
      const float part = cluster.map_shared_rank(&sh, k)->sum[i];
      // a sum that is no number comes through whatever its maximum is
      f[k] = f[k] == -INFINITY ? (part == 0.f ? 0.f : part) : expf(f[k] - high);
      total = fmaf(f[k], part, total);
    }
    const int rr = row0 + i;
    const int64_t out = ((static_cast<int64_t>(q.lo) + rr / G) * a.Hq + static_cast<int64_t>(h) * G + rr % G) * d;
    for (int col = t; col < d; col += kThreads) {
      float y = 0.f;
#pragma unroll
      for (int k = 0; k < kRanks; ++k) {
        const float* part = cluster.map_shared_rank(qs, k) + i * pad + col;
        y = fmaf(f[k], *part, y);  // a part without weight too: it has zeros, or values that are no numbers
      }
      y /= total;
      if (a.o_dtype == TREEWY_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.o)[out + col] = __float2bfloat16_rn(y);
      else static_cast<float*>(a.o)[out + col] = y;
    }
  }
  cluster.sync();  // the others may still read here
}

}  // namespace

cudaError_t launch_attend_scan(const treewy_attn& a, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(a.max_nodes) * (a.Hq / a.cache.Hkv) + kRows - 1) / kRows;
  const int64_t ctas = blocks * a.cache.Hkv * kRanks;
  if (ctas > 0x7fffffff / a.R) return cudaErrorNotSupported;
  auto bytes = [](int pad) { return sizeof(float) * (kRows * pad + 2 * kTile * (pad + 4) + kRows * kTile); };
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(attend_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes(kMaxPad)));
  });
  if (e != cudaSuccess) return e;
  // rows that can be read in fours
  const uintptr_t e4 = a.qkv_dtype == TREEWY_DTYPE_BF16 ? 8 : 16;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
  const int fours = all % e4 == 0 && a.cache.d % 4 == 0 && a.q_stride % 4 == 0 && a.k_stride % 4 == 0 && a.v_stride % 4 == 0 ? 1 : 0;
  return launch_after_smem(attend_scan_kernel, dim3(static_cast<unsigned>(ctas * a.R)), kThreads, bytes((a.cache.d + 3) & ~3), stream, a,
                           static_cast<int>(blocks), fours);
}

}  // namespace treewy
