// append.cu -- keys and values into pages of e4m3 codes (treewy_append): all
// rows of a request, or those on the path to its accepted node, behind the
// tokens that its cache holds.
//
// One CTA per (page that is written, head, keys or values): it finds the
// largest value of the page's new rows, from it the page's scale, and writes
// the codes.  Scales are powers of two, so that a code is the value with a
// shorter significand, and a scale that grows while a page fills only lowers
// the exponents of the codes that are there: nothing is rounded twice but what
// leaves e4m3's normal range.
#include "cache_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
  if constexpr (sizeof(T) == 2) return bf16_bits_to_float(x);
  else return x;
}

// Eight values of a row, in f32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(u[e] << 16);
      x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

// x in units of a scale, as e4m3; what is not finite becomes NaN.
struct Quantizer {
  float scale, inv;
  bool exact;  // inv is
  __device__ float unit(float x) const {
    const float y = exact ? x * inv : x / scale;
    return size_of(x) == fabsf(x) ? y : __uint_as_float(0x7fffffffu);
  }
  __device__ uint32_t pair(float a, float b) const { return e4m3x2(unit(a), unit(b)); }
};

template <typename T, int VEC>
__global__ void __launch_bounds__(256) append_kernel(const treewy_append_args a, int pages) {
  after_previous();
  __shared__ int parent[kMaxNodes], path[kMaxNodes], count;
  __shared__ float part[8];
  const treewy_cache& c = a.cache;
  const int t = threadIdx.x, P = c.page_len, d = c.d;
  // pages of one head are neighbours, then keys and values, heads, requests
  const int i = static_cast<int>(blockIdx.x % pages);
  unsigned rest = blockIdx.x / pages;
  const bool values = rest & 1;
  rest >>= 1;
  const int h = static_cast<int>(rest % c.Hkv), r = static_cast<int>(rest / c.Hkv);
  const bool first_cta = i == 0 && h == 0 && !values && t == 0;
  CacheRequest q = cache_request(c, a.node_offset, r, a.T, a.max_new, INT32_MAX);
  int m = q.N;  // rows that are taken
  if (a.accepted != nullptr && q.err == 0) {
    const int acc = __ldg(a.accepted + r);
    if (acc < -1 || acc >= q.N) q.err = TREEWY_STATUS_BAD_ACCEPTED;
    else if (!load_parents(parent, a.parent, q.lo, q.N)) q.err = TREEWY_STATUS_BAD_TREE;
    else {
      if (t == 0) {
        int n = 0;
        for (int p = acc; p >= 0; p = parent[p]) ++n;
        count = n;
        for (int p = acc; p >= 0; p = parent[p]) path[--n] = p;
      }
      __syncthreads();
      m = count;
    }
  }
  const int first = q.len / P;
  if (q.err == 0 && m > 0) {
    const int64_t after = static_cast<int64_t>(q.len) + m;
    bool bad = after > static_cast<int64_t>(c.max_pages) * P || after > INT32_MAX;
    if (!bad) {
      const int last = static_cast<int>((after - 1) / P);
      for (int p = first + t; p <= last; p += blockDim.x) {
        const int page = __ldg(c.page_table + static_cast<int64_t>(r) * c.max_pages + p);
        bad |= page < 0 || page >= c.num_pages;
      }
    }
    if (__syncthreads_or(bad)) q.err = TREEWY_STATUS_BAD_PAGE;
  }
  if (q.err != 0) {
    if (first_cta) atomicOr(a.status + r, q.err);
    return;
  }
  if (first_cta && a.new_length != nullptr) a.new_length[r] = q.len + m;
  const int64_t begin = static_cast<int64_t>(first + i) * P;  // the page's first token
  if (begin >= static_cast<int64_t>(q.len) + m) return;
  const int lo = max(0, static_cast<int>(q.len - begin));       // tokens that it holds already
  const int hi = static_cast<int>(min(static_cast<int64_t>(P), static_cast<int64_t>(q.len) + m - begin));
  const int j0 = static_cast<int>(begin + lo - q.len);            // the first new one
  const int page = __ldg(c.page_table + static_cast<int64_t>(r) * c.max_pages + first + i);
  const int64_t block = static_cast<int64_t>(page) * c.Hkv + h;
  uint8_t* codes = static_cast<uint8_t*>(values ? c.v : c.k) + block * P * d;
  float* scale = (values ? c.v_scale : c.k_scale) + block;
  const T* rows = static_cast<const T*>(values ? a.v : a.k) + static_cast<int64_t>(h) * d;
  const int64_t stride = values ? a.v_stride : a.k_stride;
  auto row_of = [&](int s) {  // of the page's row s
    const int j = j0 + s - lo;
    return rows + (static_cast<int64_t>(q.lo) + (a.accepted != nullptr ? path[j] : j)) * stride;
  };
  const int per = d / VEC, total = (hi - lo) * per;
  float top = 0.f;
  for (int x = t; x < total; x += blockDim.x) {
    const T* p = row_of(lo + x / per) + (x % per) * VEC;
    if constexpr (VEC == 8) {
      float f[8];
      load8(p, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, size_of(f[e]));
    } else {
      top = fmaxf(top, size_of(to_f32(__ldg(p))));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((t & 31) == 0) part[t >> 5] = top;
  const float was = lo > 0 ? *scale : 0.f;
  __syncthreads();  // and every thread has read the scale
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) top = fmaxf(top, part[w]);
  float now = was;
  if (lo == 0) now = scale_for(top);
  else if (!(top <= 448.f * was)) now = fmaxf(was, scale_for(top));
  if (t == 0) *scale = now;
  const Quantizer z{now, 1.f / now, (__float_as_uint(now) & 0x7fffffu) == 0};
  for (int x = t; x < total; x += blockDim.x) {
    const int s = lo + x / per, col = (x % per) * VEC;
    const T* p = row_of(s) + col;
    if constexpr (VEC == 8) {
      float f[8];
      load8(p, f);
      const uint2 w = make_uint2(z.pair(f[0], f[1]) | (z.pair(f[2], f[3]) << 16), z.pair(f[4], f[5]) | (z.pair(f[6], f[7]) << 16));
      *reinterpret_cast<uint2*>(codes + s * d + col) = w;
    } else {
      codes[s * d + col] = static_cast<uint8_t>(z.pair(to_f32(__ldg(p)), 0.f));
    }
  }
  if (now != was && lo > 0) {  // the scale has grown: the older tokens anew
    const float f = was / now;
    for (int x = t; x < lo * d; x += blockDim.x)
      codes[x] = static_cast<uint8_t>(e4m3x2(e4m3_to_float(codes[x]) * f, 0.f));
  }
}

}  // namespace

cudaError_t launch_append(const treewy_append_args& a, cudaStream_t stream) {
  const int P = a.cache.page_len;
  const int64_t pages = (static_cast<int64_t>(a.max_new) + P - 2) / P + 1;
  const int64_t ctas = pages * 2 * a.cache.Hkv;
  if (ctas > 0x7fffffff / a.R) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(ctas * a.R));
  const int size = a.kv_dtype == TREEWY_DTYPE_BF16 ? 2 : 4;
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                        static_cast<uintptr_t>(a.k_stride * size) | static_cast<uintptr_t>(a.v_stride * size) |
                        static_cast<uintptr_t>(a.cache.d * size);
  const bool wide = all % 16 == 0 && a.cache.d % 8 == 0;
  const int np = static_cast<int>(pages);
  if (size == 2)
    return wide ? launch_after(append_kernel<uint16_t, 8>, grid, 256, stream, a, np)
                : launch_after(append_kernel<uint16_t, 1>, grid, 256, stream, a, np);
  return wide ? launch_after(append_kernel<float, 8>, grid, 256, stream, a, np)
              : launch_after(append_kernel<float, 1>, grid, 256, stream, a, np);
}

}  // namespace treewy
