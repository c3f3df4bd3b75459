// qk_norm.cu -- norm, weight, scale and position rotation of every query and
// key head in one pass (treewy_qk_norm):
//
//   y = scale w x / sqrt(sum or mean of x^2 + eps),
//   (a, b) <- (a cos - b sin, b cos + a sin) for each rotated pair.
//
// Bound by HBM: every row is read once and written `repeat` times, and each
// lane keeps its eight elements in registers in between, f32 until the one
// rounding at the store.  A head's row is held by d / 8 neighbouring lanes
// (rounded up to a power of two), so that the sum of squares is a few shuffles
// and the other element of a rotated pair is one shuffle away or in the same
// lane.  Rows that this does not fit (odd sizes, unaligned rows, pairs that
// cross an eight at an odd place) go to one warp each, element by element.
#include "treewy_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

struct Row {
  const unsigned char* in;
  unsigned char* out;
  const float* w;
  float scale;
  int repeat;
  int64_t token;
};

// Row `head` of token t: the query heads come first.
__device__ __forceinline__ Row row_of(const treewy_qk& a, int64_t t, int head, int size) {
  Row r;
  r.token = t;
  if (head < a.Hq) {
    r.in = reinterpret_cast<const unsigned char*>(a.q) +
           (t * a.q_stride + static_cast<int64_t>(head) * a.d) * size;
    r.out = reinterpret_cast<unsigned char*>(a.q_out) +
            (t * a.Hq + head) * a.q_repeat * static_cast<int64_t>(a.d) * size;
    r.w = a.q_weight;
    r.scale = a.q_scale;
    r.repeat = a.q_repeat;
  } else {
    head -= a.Hq;
    r.in = reinterpret_cast<const unsigned char*>(a.k) +
           (t * a.k_stride + static_cast<int64_t>(head) * a.d) * size;
    r.out = reinterpret_cast<unsigned char*>(a.k_out) +
            (t * a.Hk + head) * a.k_repeat * static_cast<int64_t>(a.d) * size;
    r.w = a.k_weight;
    r.scale = a.k_scale;
    r.repeat = a.k_repeat;
  }
  return r;
}

// The rotation table's row of token t, or NULL with the status bit set.
__device__ __forceinline__ const float* table_row(const treewy_qk& a, int64_t t, bool report) {
  const int p = __ldg(a.position + t);
  if (p < 0 || p >= a.rope_rows) {
    if (report) atomicOr(a.status, TREEWY_STATUS_BAD_POSITION);
    return nullptr;
  }
  return a.rope + static_cast<int64_t>(p) * a.rope_dims;
}

__device__ __forceinline__ float inv_norm(const treewy_qk& a, float sum) {
  return 1.0f / sqrtf((a.norm == TREEWY_NORM_RMS ? sum / static_cast<float>(a.d) : sum) + a.eps);
}

// LANES lanes per row, eight elements each; UNROLL rows of a lane in flight.
template <typename T, int LANES, int UNROLL>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const treewy_qk a) {
  constexpr bool kBf16 = sizeof(T) == 2;
  constexpr int kGroups = kThreads / LANES;           // rows per pass of a CTA
  const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const int heads = a.Hq + a.Hk;
  const int64_t rows = a.T * heads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kGroups * UNROLL);
  const int64_t t_first = first / heads;
  const int h_first = static_cast<int>(first - t_first * heads);
  const int c0 = 8 * lane;
  const bool mine = c0 < a.d;

  float x[UNROLL][8];
  Row row[UNROLL];
  bool live[UNROLL];
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    const int local = i * kGroups + grp;
    live[i] = first + local < rows;
    const int at = h_first + (live[i] ? local : 0);
    row[i] = row_of(a, t_first + at / heads, at % heads, sizeof(T));
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
    if (live[i] && mine) {
      if constexpr (kBf16) {
        const uint4 u = *reinterpret_cast<const uint4*>(row[i].in + 2 * c0);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[i][2 * e] = __uint_as_float(w[e] << 16);
          x[i][2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(row[i].in + 4 * (c0 + e));
          x[i][e] = f.x; x[i][e + 1] = f.y; x[i][e + 2] = f.z; x[i][e + 3] = f.w;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(x[i][e], x[i][e], sum);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    const float f = row[i].scale * inv_norm(a, sum);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] *= f;
    if (row[i].w != nullptr && mine) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] *= __ldg(row[i].w + c0 + e);
    }
    if (a.rope_dims > 0) {
      const float* tab = live[i] ? table_row(a, row[i].token, lane == 0) : nullptr;
      if (tab == nullptr) live[i] = false;
      const int half = a.rope_dims / 2;
      if (a.interleaved) {
        if (tab != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            if (c0 + e < a.rope_dims) {
              const float c = __ldg(tab + (c0 + e) / 2), s = __ldg(tab + half + (c0 + e) / 2);
              const float u = x[i][e], v = x[i][e + 1];
              x[i][e] = u * c - v * s;
              x[i][e + 1] = v * c + u * s;
            }
          }
        }
      } else {
        // half is a multiple of 8: the pair's other eight are half / 8 lanes on
        const bool low = c0 < half, in = c0 < a.rope_dims;
        const int other = low ? lane + half / 8 : lane - half / 8;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(kFull, x[i][e], in ? other : lane, LANES);
        if (in && tab != nullptr) {
          const int j = low ? c0 : c0 - half;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float c = __ldg(tab + j + e), s = __ldg(tab + half + j + e);
            x[i][e] = low ? x[i][e] * c - y[e] * s : x[i][e] * c + y[e] * s;
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    if (!live[i] || !mine) continue;
    unsigned char* out = row[i].out + c0 * sizeof(T);
    if constexpr (kBf16) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[i][2 * e], x[i][2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&p);
      }
      for (int c = 0; c < row[i].repeat; ++c, out += a.d * sizeof(T))
        *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int c = 0; c < row[i].repeat; ++c, out += a.d * sizeof(T)) {
        *reinterpret_cast<float4*>(out) = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
        *reinterpret_cast<float4*>(out + 16) = make_float4(x[i][4], x[i][5], x[i][6], x[i][7]);
      }
    }
  }
}

// One warp per row, any size and alignment: the row passes through shared
// memory so that a pair's two elements may sit anywhere.
template <typename T>
__global__ void __launch_bounds__(kThreads) qk_norm_any_kernel(const treewy_qk a) {
  __shared__ float buf[kThreads / 32][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = a.Hq + a.Hk;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp;
  const int64_t t = at / heads;
  if (t >= a.T) return;  // a whole warp
  const Row row = row_of(a, t, static_cast<int>(at - t * heads), sizeof(T));
  const T* in = reinterpret_cast<const T*>(row.in);
  float* y = buf[warp];
  float sum = 0.f;
  for (int c = lane; c < a.d; c += 32) {
    const float x = static_cast<float>(in[c]);
    y[c] = x;
    sum = fmaf(x, x, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  const float f = row.scale * inv_norm(a, sum);
  for (int c = lane; c < a.d; c += 32) y[c] *= row.w != nullptr ? f * __ldg(row.w + c) : f;
  __syncwarp();
  if (a.rope_dims > 0) {
    const float* tab = table_row(a, t, lane == 0);
    if (tab == nullptr) return;
    const int half = a.rope_dims / 2;
    for (int i = lane; i < half; i += 32) {
      const int p = a.interleaved ? 2 * i : i, q = a.interleaved ? 2 * i + 1 : i + half;
      const float c = __ldg(tab + i), s = __ldg(tab + half + i);
      const float u = y[p], v = y[q];
      y[p] = u * c - v * s;
      y[q] = v * c + u * s;
    }
    __syncwarp();
  }
  T* out = reinterpret_cast<T*>(row.out);
  for (int c = 0; c < row.repeat; ++c)
    for (int e = lane; e < a.d; e += 32) out[c * a.d + e] = static_cast<T>(y[e]);
}

template <typename T, int LANES>
cudaError_t launch(const treewy_qk& a, int64_t rows, cudaStream_t stream) {
  constexpr int kUnroll = 4;
  constexpr int kRows = kThreads / LANES;
  const int64_t wide = (rows + kRows * kUnroll - 1) / (kRows * kUnroll);
  qk_norm_kernel<T, LANES, kUnroll><<<static_cast<unsigned>(wide), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const treewy_qk& a, cudaStream_t stream) {
  const int64_t rows = a.T * (a.Hq + a.Hk);
  auto on16 = [](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride * sizeof(T)) % 16 == 0;
  };
  bool wide = a.d % 8 == 0 && (a.interleaved || a.rope_dims % 16 == 0);
  if (a.Hq > 0) wide = wide && on16(a.q, a.q_stride) && on16(a.q_out, 0);
  if (a.Hk > 0) wide = wide && on16(a.k, a.k_stride) && on16(a.k_out, 0);
  if (!wide) {
    constexpr int kRows = kThreads / 32;
    qk_norm_any_kernel<T><<<static_cast<unsigned>((rows + kRows - 1) / kRows), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  if (a.d <= 64) return launch<T, 8>(a, rows, stream);
  if (a.d <= 128) return launch<T, 16>(a, rows, stream);
  return launch<T, 32>(a, rows, stream);
}

}  // namespace

cudaError_t launch_qk_norm(const treewy_qk& a, cudaStream_t stream) {
  return a.dtype == TREEWY_DTYPE_BF16 ? launch_typed<__nv_bfloat16>(a, stream)
                                      : launch_typed<float>(a, stream);
}

}  // namespace treewy
