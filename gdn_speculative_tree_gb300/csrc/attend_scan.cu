// attend_scan.cu -- attention over pages of e4m3 keys and values and the
// draft's own ones, in f32 on the CUDA cores (treewy_attend for f32 rows or
// outputs and for head sizes that the tensor-core kernel does not take).
//
// One pass over the tokens with the running maximum and sum of the softmax: a
// CTA holds 16 (node, query head) rows that share a key head, and takes 32
// tokens at a time, the context's and then the draft's, through one tile in
// shared memory (keys, then values).
#include "cache_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

constexpr int kRows = 16, kTile = 32, kThreads = 128;
constexpr unsigned kFull = 0xffffffffu;

__global__ void __launch_bounds__(kThreads) attend_scan_kernel(const treewy_attn a, int blocks) {
  after_previous();
  extern __shared__ float smem[];
  __shared__ int parent[kMaxNodes];
  __shared__ unsigned long long seen[kMaxNodes];
  __shared__ int page_of[2];
  const treewy_cache& c = a.cache;
  const int t = threadIdx.x, d = c.d, P = c.page_len, pitch = d + 1;
  const int block = static_cast<int>(blockIdx.x % blocks);
  const unsigned rest = blockIdx.x / blocks;
  const int h = static_cast<int>(rest % c.Hkv), r = static_cast<int>(rest / c.Hkv);
  const int G = a.Hq / c.Hkv;
  CacheRequest q = cache_request(c, a.node_offset, r, a.T, a.max_nodes, a.max_context);
  if (q.err == 0 && !load_parents(parent, a.parent, q.lo, q.N)) q.err = TREEWY_STATUS_BAD_TREE;
  if (q.err != 0) {
    if (block == 0 && h == 0 && t == 0) atomicOr(a.status + r, q.err);
    return;
  }
  const int row0 = block * kRows, live = min(kRows, q.N * G - row0);
  if (live <= 0) return;
  if (t < q.N) {  // the nodes that node t sees
    unsigned long long m = 0;
    for (int p = t; p >= 0; p = parent[p]) m |= 1ull << p;
    seen[t] = m;
  }
  float* qs = smem;                    // [kRows][d]
  float* tile = qs + kRows * d;        // [kTile][pitch]
  float* weight = tile + kTile * pitch;  // [kRows][kTile]
  const bool bf16 = a.qkv_dtype == TREEWY_DTYPE_BF16;
  for (int x = t; x < kRows * d; x += kThreads) {
    const int row = row0 + x / d;
    qs[x] = x / d < live ? load_qkv(a.q, (static_cast<int64_t>(q.lo) + row / G) * a.q_stride +
                                             (static_cast<int64_t>(h) * G + row % G) * d + x % d, bf16)
                         : 0.f;
  }
  const int row = t / 8, sub = t % 8;  // eight threads per row
  const int node = min(row0 + row, q.N * G - 1) / G;
  float acc[32], top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) acc[e] = 0.f;
  const int total = q.len + q.N;
  for (int t0 = 0; t0 < total; ) {
    // tokens of the context, or of the draft: a tile has one kind
    const bool context = t0 < q.len;
    const int n = min(kTile, (context ? q.len : total) - t0);
    __syncthreads();  // the tile and the weights are free
    if (context) {
      const int p0 = t0 / P;
      if (t < 2) {
        page_of[t] = -1;
        if (p0 + t <= (t0 + n - 1) / P) page_of[t] = __ldg(c.page_table + static_cast<int64_t>(r) * c.max_pages + p0 + t);
      }
      __syncthreads();
      bool bad = false;
      for (int i = 0; i <= (t0 + n - 1) / P - p0; ++i) bad |= page_of[i] < 0 || page_of[i] >= c.num_pages;
      if (bad) {
        if (block == 0 && h == 0 && t == 0) atomicOr(a.status + r, TREEWY_STATUS_BAD_PAGE);
        return;
      }
    }
    auto load = [&](bool values) {
      for (int x = t; x < n * d; x += kThreads) {
        const int j = x / d, col = x % d;
        float f;
        if (context) {
          const int at = t0 + j;
          const int64_t b = static_cast<int64_t>(page_of[at / P - t0 / P]) * c.Hkv + h;
          f = e4m3_to_float(__ldg(static_cast<const uint8_t*>(values ? c.v : c.k) + (b * P + at % P) * d + col)) *
              __ldg((values ? c.v_scale : c.k_scale) + b);
        } else {
          f = load_qkv(values ? a.v : a.k, (static_cast<int64_t>(q.lo) + t0 - q.len + j) * (values ? a.v_stride : a.k_stride) +
                                               static_cast<int64_t>(h) * d + col, bf16);
        }
        tile[j * pitch + col] = f;
      }
    };
    load(false);
    __syncthreads();
    float s[4], high = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = sub + 8 * e;
      s[e] = -INFINITY;
      if (j < n && (context || ((seen[node] >> (t0 - q.len + j)) & 1))) {
        float dot = 0.f;
        for (int x = 0; x < d; ++x) dot = fmaf(qs[row * d + x], tile[j * pitch + x], dot);
        s[e] = dot * a.scale;
      }
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
    for (int e = 0; e < 32; ++e) acc[e] *= keep;
    __syncthreads();
    load(true);
    __syncthreads();
    for (int j = 0; j < n; ++j) {
      const float w = weight[row * kTile + j];
      // what a node does not see adds nothing to it, whatever it is
      if (!context && !((seen[node] >> (t0 - q.len + j)) & 1)) continue;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const int col = sub + 8 * e;
        if (col < d) acc[e] = fmaf(w, tile[j * pitch + col], acc[e]);
      }
    }
    t0 += n;
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (row >= live) return;
  const int64_t out = ((static_cast<int64_t>(q.lo) + (row0 + row) / G) * a.Hq + static_cast<int64_t>(h) * G + (row0 + row) % G) * d;
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const int col = sub + 8 * e;
    if (col >= d) continue;
    const float y = acc[e] / sum;
    if (a.o_dtype == TREEWY_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.o)[out + col] = __float2bfloat16_rn(y);
    else static_cast<float*>(a.o)[out + col] = y;
  }
}

}  // namespace

cudaError_t launch_attend_scan(const treewy_attn& a, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(a.max_nodes) * (a.Hq / a.cache.Hkv) + kRows - 1) / kRows;
  const int64_t ctas = blocks * a.cache.Hkv;
  if (ctas > 0x7fffffff / a.R) return cudaErrorNotSupported;
  const int d = a.cache.d;
  const size_t bytes = sizeof(float) * (kRows * d + kTile * (d + 1) + kRows * kTile);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(attend_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                sizeof(float) * (kRows * 256 + kTile * 257 + kRows * kTile));
  });
  if (e != cudaSuccess) return e;
  return launch_after_smem(attend_scan_kernel, dim3(static_cast<unsigned>(ctas * a.R)), kThreads, bytes, stream, a,
                           static_cast<int>(blocks));
}

}  // namespace treewy
