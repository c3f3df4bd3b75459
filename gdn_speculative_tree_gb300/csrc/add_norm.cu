// add_norm.cu -- the residual's addition and the RMS norm of a row in one
// pass, with the normed row in its own type, in e4m3 with scales, or both
// (treewy_add_norm):
//
//   z = x + residual,  y = w z / sqrt(mean of z^2 + eps),
//   scale = (largest |y| of a group of columns) / 448,  y8 = y / scale.
//
// Bound by HBM: a row is read once, held in f32 by the threads that share it
// (eight neighbouring columns at a time, V times), and written from there:
// 940 MB in 149 us (6.3 TB/s, 0.93 of a copy); 4 us for 256 rows of 2048, the
// launch.
// Rows that this does not fit (odd widths, unaligned rows) are held in shared
// memory, element by element.
#include "cache_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct None {};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(u[e] << 16);
      x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      u[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
  }
}

struct Add {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// `op` over the row's TPR threads (a power of two), the same in all of them.
// part: a word for each of the CTA's warps, which no earlier reduction that a
// thread may still read used.
template <int TPR, typename Op>
__device__ __forceinline__ float reduce_row(float v, float* part, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(kFull, v, o));
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < TPR / 32; ++w) v = op(v, part[w]);
  }
  return v;
}

// A group's scale from its largest value, and what to multiply by: at least
// 2^-126, one over which is finite (zeros beside tiny values stay zeros).
__device__ __forceinline__ float2 scale_of(float top) {
  const float s = top > 0.f ? fmaxf(top / 448.f, 1.17549435e-38f) : 1.f;
  return make_float2(s, 1.f / s);
}

// CTAs that an SM shall hold (without a word on it the compiler takes more
// registers for some: 8,192 rows of 16384 then take 269 us for 180).
constexpr int ctas_of(int tpr, int v) { return tpr == 256 ? (v == 2 ? 6 : 5) : tpr == 512 ? 2 : tpr == 1024 ? 1 : v == 2 ? 12 : 16; }

// TPR threads to a row (32: four rows to a CTA; more: one), V pieces of eight
// columns to a thread.  Wide rows go to more threads rather than more pieces,
// as long as several CTAs fit an SM: 32,768 rows of 4096 take 149 us with 256
// threads of two pieces, 159 with 128 of four or 512 of one; of 8192, 304 us
// with 256 of four in 48 registers (324 in 61), 314 with 512 of two; 8,192 rows
// of 16384, 180 us with 512 of four, 233 with 1024 of two.
template <typename X, typename Z, int TPR, int V>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, ctas_of(TPR, V)) add_norm_kernel(const treewy_norm a) {
  after_previous();
  constexpr int kThreads = TPR < 128 ? 128 : TPR;
  constexpr bool kResidual = !std::is_same<Z, None>::value;
  __shared__ float part[2][32];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  if (TPR == 32 && row >= a.T) return;  // a whole warp
  const int n8 = a.n >> 3;
  const X* x = static_cast<const X*>(a.x) + row * a.x_stride;
  float z[V][8], sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = i * TPR + t;
    if (at < n8) {
      load8(x + 8 * at, z[i]);
      if constexpr (kResidual) {
        float f[8];
        load8(static_cast<const Z*>(a.residual) + row * a.residual_stride + 8 * at, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[i][e] += f[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = i * TPR + t;
    if constexpr (kResidual) {
      if (at < n8) store8(static_cast<Z*>(a.residual_out) + row * a.n + 8 * at, z[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(z[i][e], z[i][e], sum);
  }
  sum = reduce_row<TPR>(sum, part[0], Add());
  const float f = rsqrtf(sum / static_cast<float>(a.n) + a.eps);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = i * TPR + t;
    if (at < n8) {
      float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (a.weight != nullptr) load8(a.weight + 8 * at, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[i][e] *= f * w[e];
        top = fmaxf(top, fabsf(z[i][e]));
      }
      if (a.y != nullptr) store8(static_cast<X*>(a.y) + row * a.n + 8 * at, z[i]);
    }
  }
  if (a.y8 == nullptr) return;
  float2 s = make_float2(1.f, 1.f);
  if (a.group == 0) {
    top = reduce_row<TPR>(top, part[1], Max());
    s = scale_of(top);
    if (t == 0) a.y8_scale[row] = s.x;
  }
  const int lanes = a.group >> 3, groups = a.group != 0 ? (a.n + a.group - 1) / a.group : 1;  // a group's threads: 4, 8 or 16
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = i * TPR + t;
    if (lanes != 0) {
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(z[i][e]));
      for (int o = lanes >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      s = scale_of(m);
      if (at < n8 && at % lanes == 0) a.y8_scale[row * groups + at / lanes] = s.x;
    }
    if (at < n8) {
      uint32_t w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[e] = e4m3x2(z[i][4 * e] * s.y, z[i][4 * e + 1] * s.y) | (e4m3x2(z[i][4 * e + 2] * s.y, z[i][4 * e + 3] * s.y) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y8) + row * a.n + 8 * at) = make_uint2(w[0], w[1]);
    }
  }
}

template <typename T>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  if constexpr (sizeof(T) == 2) return bf16_bits_to_float(static_cast<const uint16_t*>(p)[at]);
  else return static_cast<const float*>(p)[at];
}
__device__ __forceinline__ void store1(void* p, int64_t at, float x, bool bf16) {
  if (bf16) static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(x);
  else static_cast<float*>(p)[at] = x;
}

constexpr int kPlainThreads = 256;

// A CTA per row, any width and alignment: the row in shared memory.  Bound by
// instructions, a value at a time: 16,000 rows of 4001 take 236 us (1.9 TB/s).
__global__ void __launch_bounds__(kPlainThreads) add_norm_plain_kernel(const treewy_norm a) {
  after_previous();
  extern __shared__ float z[];
  __shared__ float part[2][32];
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x, n = a.n;
  const bool xb = a.x_dtype == TREEWY_DTYPE_BF16, rb = a.residual_dtype == TREEWY_DTYPE_BF16;
  float sum = 0.f;
  for (int i = t; i < n; i += kPlainThreads) {
    const int64_t from = row * a.x_stride + i;  // plain loads: y may be x
    float v = xb ? load1<uint16_t>(a.x, from) : load1<float>(a.x, from);
    if (a.residual != nullptr) {
      const int64_t at = row * a.residual_stride + i;
      v += rb ? load1<uint16_t>(a.residual, at) : load1<float>(a.residual, at);
      store1(a.residual_out, row * n + i, v, rb);
    }
    z[i] = v;
    sum = fmaf(v, v, sum);
  }
  sum = reduce_row<kPlainThreads>(sum, part[0], Add());
  const float f = rsqrtf(sum / static_cast<float>(n) + a.eps);
  float top = 0.f;
  for (int i = t; i < n; i += kPlainThreads) {
    const float y = z[i] * (f * (a.weight != nullptr ? __ldg(a.weight + i) : 1.f));
    z[i] = y;
    top = fmaxf(top, fabsf(y));
    if (a.y != nullptr) store1(a.y, row * n + i, y, xb);
  }
  if (a.y8 == nullptr) return;
  uint8_t* y8 = static_cast<uint8_t*>(a.y8) + row * n;
  if (a.group == 0) {
    const float2 s = scale_of(reduce_row<kPlainThreads>(top, part[1], Max()));
    if (t == 0) a.y8_scale[row] = s.x;
    for (int i = t; i < n; i += kPlainThreads) y8[i] = static_cast<uint8_t>(e4m3x2(z[i] * s.y, 0.f));
    return;
  }
  __syncthreads();
  const int groups = (n + a.group - 1) / a.group;
  for (int g = t >> 5; g < groups; g += kPlainThreads / 32) {  // a warp per group
    const int hi = min(n, (g + 1) * a.group);
    float m = 0.f;
    for (int i = g * a.group + (t & 31); i < hi; i += 32) m = fmaxf(m, fabsf(z[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    const float2 s = scale_of(m);
    if ((t & 31) == 0) a.y8_scale[row * groups + g] = s.x;
    for (int i = g * a.group + (t & 31); i < hi; i += 32) y8[i] = static_cast<uint8_t>(e4m3x2(z[i] * s.y, 0.f));
  }
}

template <typename X, typename Z, int TPR, int V>
cudaError_t launch(const treewy_norm& a, cudaStream_t stream) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR;
  const int64_t ctas = (a.T + kThreads / TPR - 1) / (kThreads / TPR);
  return launch_after(add_norm_kernel<X, Z, TPR, V>, dim3(static_cast<unsigned>(ctas)), kThreads, stream, a);
}

template <typename X, typename Z>
cudaError_t by_width(const treewy_norm& a, cudaStream_t stream) {
  if (a.n <= 256) return launch<X, Z, 32, 1>(a, stream);
  if (a.n <= 1024) return launch<X, Z, 128, 1>(a, stream);
  if (a.n <= 2048) return launch<X, Z, 128, 2>(a, stream);
  if (a.n <= 4096) return launch<X, Z, 256, 2>(a, stream);
  if (a.n <= 8192) return launch<X, Z, 256, 4>(a, stream);
  if (a.n <= 16384) return launch<X, Z, 512, 4>(a, stream);
  return launch<X, Z, 1024, 4>(a, stream);
}

template <typename X>
cudaError_t by_residual(const treewy_norm& a, cudaStream_t stream) {
  if (a.residual == nullptr) return by_width<X, None>(a, stream);
  return a.residual_dtype == TREEWY_DTYPE_BF16 ? by_width<X, uint16_t>(a, stream) : by_width<X, float>(a, stream);
}

}  // namespace

cudaError_t launch_add_norm(const treewy_norm& a, cudaStream_t stream) {
  const int sx = a.x_dtype == TREEWY_DTYPE_BF16 ? 2 : 4, sr = a.residual_dtype == TREEWY_DTYPE_BF16 ? 2 : 4;
  uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.weight) | reinterpret_cast<uintptr_t>(a.y) |
                  static_cast<uintptr_t>(a.x_stride * sx);
  if (a.residual != nullptr)
    all |= reinterpret_cast<uintptr_t>(a.residual) | reinterpret_cast<uintptr_t>(a.residual_out) |
           static_cast<uintptr_t>(a.residual_stride * sr);
  if (a.n % 8 == 0 && all % 16 == 0 && reinterpret_cast<uintptr_t>(a.y8) % 8 == 0)
    return sx == 2 ? by_residual<uint16_t>(a, stream) : by_residual<float>(a, stream);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(add_norm_plain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 32768 * 4);
  });
  if (e != cudaSuccess) return e;
  return launch_after_smem(add_norm_plain_kernel, dim3(static_cast<unsigned>(a.T)), kPlainThreads,
                           static_cast<size_t>(a.n) * 4, stream, a);
}

}  // namespace treewy
