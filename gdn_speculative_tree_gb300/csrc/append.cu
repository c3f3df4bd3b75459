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
//
// Bound by HBM where there is much to do: 187 MB of prompts in 41.5 us
// (4.5 TB/s), and short of it by the two steps of every CTA, the loads and,
// behind a barrier, the writing; by the launch (4.3 us for 64 single tokens)
// where there is little.
#include "cache_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
  if constexpr (sizeof(T) == 2) return bf16_bits_to_float(x);
  else return x;
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

// Eight neighbouring values of a row, as they are stored.
template <typename T>
struct Piece {
  uint4 w[sizeof(T) / 2];
  __device__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) {
          x[2 * e] = __uint_as_float(u[e] << 16);
          x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
        } else {
          x[4 * i + e] = __uint_as_float(u[e]);
        }
      }
    }
  }
  // |values| as whole numbers, which order them: the largest so far of two in a word (bf16), or of one.
  __device__ uint32_t largest(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) m = __vmaxu2(m, u[e] & 0x7fff7fffu);
        else m = max(m, u[e] & 0x7fffffffu);
      }
    }
    return m;
  }
  __device__ float largest_finite() const {
    float x[8], top = 0.f;
    values(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, size_of(x[e]));
    return top;
  }
  __device__ uint2 codes(const Quantizer& z) const {
    float x[8];
    values(x);
    return make_uint2(z.pair(x[0], x[1]) | (z.pair(x[2], x[3]) << 16), z.pair(x[4], x[5]) | (z.pair(x[6], x[7]) << 16));
  }
  // The same where all are finite and 1 / scale is exact.
  __device__ uint2 codes(float inv) const {
    float x[8];
    values(x);
    return make_uint2(e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16),
                      e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16));
  }
};

// Four codes times f (2^-n), rounded again where they leave e4m3's normal range.
__device__ __forceinline__ uint32_t again(uint32_t w, float f) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = e4m3x2_to_f16x2((w >> (16 * i)) & 0xffffu);
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h));
    out |= e4m3x2(y.x * f, y.y * f) << (16 * i);
  }
  return out;
}

// HOLD: pieces of eight values that a thread keeps from the search for the
// largest to the writing, what is behind them is read twice; 0: one value at a
// time, read twice (odd sizes).
template <typename T, int HOLD>
// Two CTAs of 512 (64 registers a thread for bf16): 41.5 us for the prompts of pages of 64 tokens, 47.6 with 128 registers.
__global__ void __launch_bounds__(512, sizeof(T) == 2 ? 2 : 1) append_kernel(const treewy_append_args a, int pages) {
  after_previous();
  __shared__ int parent[kMaxNodes], path[kMaxNodes], count;
  __shared__ uint32_t part[16];
  const treewy_cache& c = a.cache;
  const int t = threadIdx.x, P = c.page_len, d = c.d, threads = blockDim.x;
  // heads are neighbours as they are in a row, then keys and values, pages, requests
  const int h = static_cast<int>(blockIdx.x % c.Hkv);
  unsigned rest = blockIdx.x / c.Hkv;
  const bool values = rest & 1;
  rest >>= 1;
  const int i = static_cast<int>(rest % pages), r = static_cast<int>(rest / pages);
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
  // what goes into this CTA's page
  const int first = q.len / P;
  const int64_t begin = (static_cast<int64_t>(first) + i) * P, after = static_cast<int64_t>(q.len) + m;
  const int lo = max(0, static_cast<int>(q.len - begin));  // tokens that it holds already
  const int hi = q.err == 0 && m > 0 && begin < after ? static_cast<int>(min(static_cast<int64_t>(P), after - begin)) : 0;  // and with the new ones
  const int j0 = static_cast<int>(begin + lo - q.len);       // the first of them
  const T* rows = static_cast<const T*>(values ? a.v : a.k) + static_cast<int64_t>(h) * d;
  const int64_t stride = values ? a.v_stride : a.k_stride;
  const int32_t* table = c.page_table + static_cast<int64_t>(r) * c.max_pages;
  auto row_of = [&](int row) {  // of the page
    const int j = j0 + row - lo;
    return rows + (static_cast<int64_t>(q.lo) + (a.accepted != nullptr ? path[j] : j)) * stride;
  };
  // a thread's pieces: its first row and column, and the way to the next ones
  const int per = HOLD > 0 ? d / 8 : d, row0 = t / per, col0 = t - row0 * per, down = threads / per, right = threads - down * per;
  Piece<T> x[HOLD > 0 ? HOLD : 1];
  if constexpr (HOLD > 0) {  // on their way while the pages are looked at
    int row = lo + row0, col = col0;
#pragma unroll
    for (int e = 0; e < HOLD; ++e) {
      if (row < hi) x[e].load(row_of(row) + 8 * col);
      row += down, col += right;
      if (col >= per) col -= per, ++row;
    }
  }
  if (q.err == 0 && m > 0) {
    bool bad = after > static_cast<int64_t>(c.max_pages) * P || after > INT32_MAX;
    if (!bad) {
      const int last = static_cast<int>((after - 1) / P);
      for (int p = first + t; p <= last; p += threads) {
        const int page = __ldg(table + p);
        bad |= page < 0 || page >= c.num_pages;
      }
    }
    if (__syncthreads_or(bad)) q.err = TREEWY_STATUS_BAD_PAGE;
  }
  if (q.err != 0) {
    if (first_cta) atomicOr(a.status + r, q.err);
    return;
  }
  if (first_cta && a.new_length != nullptr) a.new_length[r] = static_cast<int>(after);
  if (hi == 0) return;
  const int page = __ldg(table + first + i);
  const int64_t block = static_cast<int64_t>(page) * c.Hkv + h;
  uint8_t* codes = static_cast<uint8_t*>(values ? c.v : c.k) + block * P * d;
  float* scale = (values ? c.v_scale : c.k_scale) + block;
  const float was = lo > 0 ? *scale : 0.f;
  int row = 0, col = 0;
  auto step = [&] {
    row += down, col += right;
    if (col >= per) col -= per, ++row;
  };
  // f(piece, where it goes) for all of the thread's, those in the registers first
  auto pieces = [&](auto f) {
    row = lo + row0, col = col0;
    if constexpr (HOLD > 0) {
#pragma unroll
      for (int e = 0; e < HOLD; ++e) {
        if (row < hi) f(x[e], codes + row * d + 8 * col);
        step();
      }
#pragma unroll 1
      for (; row < hi; step()) {
        Piece<T> y;
        y.load(row_of(row) + 8 * col);
        f(y, codes + row * d + 8 * col);
      }
    }
  };
  auto over_cta = [&](uint32_t m, uint32_t* to) {  // the largest of a word of every thread
    m = __reduce_max_sync(0xffffffffu, m);
    if ((t & 31) == 0) to[t >> 5] = m;
    __syncthreads();
    for (int w = 0; w < threads >> 5; ++w) m = max(m, to[w]);
    return m;
  };
  float top;
  bool plain = false;  // all values are finite
  if constexpr (HOLD > 0) {
    uint32_t m = 0;
    pieces([&](const Piece<T>& y, uint8_t*) { m = y.largest(m); });
    if constexpr (sizeof(T) == 2) m = max(m & 0xffffu, m >> 16) << 16;
    m = over_cta(m, part);  // and every thread has read the scale
    plain = m < 0x7f800000u;
    top = __uint_as_float(m);
    if (!plain) {
      top = 0.f;
      pieces([&](const Piece<T>& y, uint8_t*) { top = fmaxf(top, y.largest_finite()); });
      __syncthreads();  // the words of the first search have been read
      top = __uint_as_float(over_cta(__float_as_uint(top), part));
    }
  } else {
    top = 0.f;
    for (row = lo + row0, col = col0; row < hi; step()) top = fmaxf(top, size_of(to_f32(__ldg(row_of(row) + col))));
    top = __uint_as_float(over_cta(__float_as_uint(top), part));
  }
  float now = was;
  if (lo == 0) now = scale_for(top);
  else if (!(top <= 448.f * was)) now = fmaxf(was, scale_for(top));
  if (t == 0) *scale = now;
  const Quantizer z{now, 1.f / now, (__float_as_uint(now) & 0x7fffffu) == 0};
  if constexpr (HOLD > 0) {
    if (plain && z.exact) pieces([&](const Piece<T>& y, uint8_t* at) { *reinterpret_cast<uint2*>(at) = y.codes(z.inv); });
    else pieces([&](const Piece<T>& y, uint8_t* at) { *reinterpret_cast<uint2*>(at) = y.codes(z); });
  } else {
    for (row = lo + row0, col = col0; row < hi; step())
      codes[row * d + col] = static_cast<uint8_t>(z.pair(to_f32(__ldg(row_of(row) + col)), 0.f));
  }
  if (now != was && lo > 0) {  // the scale has grown: the older tokens anew
    const float f = was / now;
    if constexpr (HOLD > 0) {
      for (int k = t; k < lo * d / 8; k += threads) {
        uint2* at = reinterpret_cast<uint2*>(codes) + k;
        const uint2 old = *at;
        *at = make_uint2(again(old.x, f), again(old.y, f));
      }
    } else {
      for (int k = t; k < lo * d; k += threads) codes[k] = static_cast<uint8_t>(e4m3x2(e4m3_to_float(codes[k]) * f, 0.f));
    }
  }
}

constexpr int kHold = 8;

template <typename T>
cudaError_t launch(const treewy_append_args& a, cudaStream_t stream) {
  const int P = a.cache.page_len;
  const int64_t pages = (static_cast<int64_t>(a.max_new) + P - 2) / P + 1;  // that max_new rows can touch
  const int64_t ctas = pages * 2 * a.cache.Hkv;
  if (ctas > 0x7fffffff / a.R) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(ctas * a.R));
  const int np = static_cast<int>(pages);
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                        static_cast<uintptr_t>(a.k_stride * sizeof(T)) | static_cast<uintptr_t>(a.v_stride * sizeof(T)) |
                        static_cast<uintptr_t>(a.cache.d * sizeof(T));
  if (all % 16 != 0 || a.cache.d % 8 != 0) return launch_after(append_kernel<T, 0>, grid, 256, stream, a, np);
  // paths are short whatever the trees' bound is
  const int rows = std::min(a.max_new, P), pieces = (a.accepted != nullptr ? std::min(rows, 8) : rows) * (a.cache.d / 8);
  // a single token's page: 640 requests 4.8 us, 6.7 with eight pieces a thread
  if (pieces <= 64) return launch_after(append_kernel<T, 1>, grid, 64, stream, a, np);
  // As few threads as hold the page: 16 prompts of 3500 to 4096 tokens with pages of 32 tokens, heads of 256, take 39 us with
  // 128 threads of eight pieces, 47 with 256 of four, 81 with 512 of two; pages of 128, whose second half 256 threads would
  // read twice, 45 us against 54; the paths of 256 trees 6.4 us with 64 threads, 7.7 with 128, 12.3 with 256.
  const unsigned threads = pieces <= 512 ? 64 : pieces <= 1024 ? 128 : pieces <= 2048 ? 256 : 512;
  return launch_after(append_kernel<T, kHold>, grid, threads, stream, a, np);
}

}  // namespace

cudaError_t launch_append(const treewy_append_args& a, cudaStream_t stream) {
  return a.kv_dtype == TREEWY_DTYPE_BF16 ? launch<uint16_t>(a, stream) : launch<float>(a, stream);
}

}  // namespace treewy
