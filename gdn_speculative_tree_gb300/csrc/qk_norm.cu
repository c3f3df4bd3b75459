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
// lane.  A warp takes several heads of one token and side (q or k), so that
// the weights and the token's cosines and sines are loaded once for all of
// them.  Where a pair's elements are not a multiple of eight apart (kOdd), the
// other one is loaded by itself.  Rows that this does not fit (odd sizes,
// unaligned rows) go to one warp each, element by element.
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

// The rotation table's row of position p, or NULL with the status bit set.
__device__ __forceinline__ const float* table_row(const treewy_qk& a, int p, bool report) {
  if (p < 0 || p >= a.rope_rows) {
    if (report) atomicOr(a.status, TREEWY_STATUS_BAD_POSITION);
    return nullptr;
  }
  return a.rope + static_cast<int64_t>(p) * a.rope_dims;
}

// 1 / sqrt: the hardware's reciprocal root, right to two units of f32's last
// place, against the 2^-9 or 2^-24 of the outputs' rounding.  mean: 1 / d for
// the RMS norm, 1 for L2.
__device__ __forceinline__ float inv_norm(float sum, float mean, float eps) {
  return rsqrtf(fmaf(sum, mean, eps));
}

// Eight elements of a row as they are stored.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
    const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(T) == 2) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      } else {
        x[4 * i + e] = __uint_as_float(w[e]);
      }
    }
  }
}
__device__ __forceinline__ void load8_f32(const float* p, float (&x)[8]) {
  const float4 f = *reinterpret_cast<const float4*>(p), g = *reinterpret_cast<const float4*>(p + 4);
  x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  x[4] = g.x; x[5] = g.y; x[6] = g.z; x[7] = g.w;
}

// From element c of a rotated pair to the other one.
__device__ __forceinline__ int pair_step(const treewy_qk& a, int c) {
  if (a.interleaved) return (c & 1) ? -1 : 1;
  return c < a.rope_dims / 2 ? a.rope_dims / 2 : -(a.rope_dims / 2);
}

// Many rows outgrow L2: they pass through it as a stream.
template <bool STREAM>
__device__ __forceinline__ uint4 get(const void* p) {
  const uint4* q = static_cast<const uint4*>(p);
  return STREAM ? __ldcs(q) : *q;
}
template <bool STREAM, typename V>
__device__ __forceinline__ void put(void* p, V x) {
  if (STREAM) __stcs(static_cast<V*>(p), x);
  else *static_cast<V*>(p) = x;
}

// LANES lanes per head, eight elements each; a warp takes UNROLL passes of
// 32 / LANES heads of one token's q or k, all loaded before the first is used.
// PAIRS: the two elements of a pair are half / 8 lanes apart, neighbours, or at
// any distance with the rotation ending anywhere.
enum Pairs { kLanes, kNeighbours, kOdd };
template <typename T, int LANES, int UNROLL, int THREADS, Pairs PAIRS>
__global__ void __launch_bounds__(THREADS, 896 / THREADS)
    qk_norm_kernel(const treewy_qk a, int q_units, int units, float mean) {
  after_previous();
  constexpr bool ODD = PAIRS == kOdd, NEXT = PAIRS == kNeighbours, kStream = UNROLL > 2;
  constexpr int kPass = 32 / LANES;                   // heads per pass
  const int lane = threadIdx.x % LANES, grp = (threadIdx.x & 31) / LANES;
  const int c0 = 8 * lane;
  const bool mine = c0 < a.d;
  // half is a multiple of 8 (but where ODD): a pair's other eight are half / 8 lanes on
  const int half = a.rope_dims / 2;
  const bool in_rope = c0 < a.rope_dims, low = c0 < half;
  const int other = in_rope ? (low ? lane + half / 8 : lane - half / 8) : lane;
  // a warp's first token and part, and the way to its next ones
  const unsigned at = blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5), warps = gridDim.x * (THREADS / 32);
  int64_t t = at / static_cast<unsigned>(units);
  int part = static_cast<int>(at % static_cast<unsigned>(units));
  const int hop = static_cast<int>(warps / units), step = static_cast<int>(warps % units);
  for (; t < a.T; t += hop + (part + step >= units), part = part + step - (part + step >= units ? units : 0)) {
    const int position = a.rope_dims > 0 ? __ldg(a.position + t) : 0;
    const bool isq = part < q_units;
    const int heads = isq ? a.Hq : a.Hk, repeat = isq ? a.q_repeat : a.k_repeat;
    const int h0 = (isq ? part : part - q_units) * (UNROLL * kPass) + grp;
    const unsigned char* in =
        reinterpret_cast<const unsigned char*>(isq ? a.q : a.k) +
        (t * (isq ? a.q_stride : a.k_stride) + static_cast<int64_t>(h0) * a.d + c0) * static_cast<int64_t>(sizeof(T));
    const int step = kPass * a.d * static_cast<int>(sizeof(T));
    Raw8<T> raw[UNROLL];
    T far[ODD ? UNROLL : 1][8];                       // ODD: the pairs' other elements
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      if constexpr (ODD) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          far[i][e] = static_cast<T>(0.f);
          if (h0 + i * kPass < heads && c0 + e < a.rope_dims)
            far[i][e] = reinterpret_cast<const T*>(in + static_cast<int64_t>(i) * step)[pair_step(a, c0 + e) + e];
        }
      }
#pragma unroll
      for (int k = 0; k < static_cast<int>(sizeof(T) / 2); ++k) {
        raw[i].w[k] = make_uint4(0u, 0u, 0u, 0u);
        if (h0 + i * kPass < heads && mine)
          raw[i].w[k] = get<kStream>(in + static_cast<int64_t>(i) * step + 16 * k);
      }
    }
    const float* tab = nullptr;                       // looked up while the rows are on their way
    if (a.rope_dims > 0) {
      tab = table_row(a, position, part == 0 && (threadIdx.x & 31) == 0);
      if (tab == nullptr) continue;                   // a whole warp
    }
    // y = f (x wc + x' ws) with x' the pair's other element (ws = 0: no pair)
    float wc[8], ws[8];
    const float* weight = isq ? a.q_weight : a.k_weight;
    const float scale = isq ? a.q_scale : a.k_scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) wc[e] = scale, ws[e] = 0.f;
    if constexpr (ODD) {
      float cs[8], sn[8], v[8];                       // all on their way before the first is used
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + e, by = pair_step(a, c), i = a.interleaved ? c / 2 : by > 0 ? c : c - half;
        const bool pair = c < a.rope_dims;
        cs[e] = pair ? tab[i] : 1.f;
        sn[e] = pair ? tab[half + i] : 0.f;
        v[e] = pair && weight != nullptr ? weight[c + by] : 1.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        wc[e] *= cs[e];
        ws[e] = scale * (pair_step(a, c0 + e) > 0 ? -sn[e] : sn[e]) * v[e];
      }
    } else if (in_rope) {
      float cs[8], sn[8], v[8];
      if constexpr (NEXT) {
        const float4 c = *reinterpret_cast<const float4*>(tab + c0 / 2);
        const float4 s = *reinterpret_cast<const float4*>(tab + half + c0 / 2);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          cs[e] = cc[e / 2];
          sn[e] = (e & 1) ? ss[e / 2] : -ss[e / 2];
        }
      } else {
        load8_f32(tab + (low ? c0 : c0 - half), cs);
        load8_f32(tab + half + (low ? c0 : c0 - half), sn);
        if (low) {
#pragma unroll
          for (int e = 0; e < 8; ++e) sn[e] = -sn[e];
        }
      }
      if (weight != nullptr) load8_f32(weight + (NEXT ? c0 : 8 * other), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        wc[e] *= cs[e];
        ws[e] = scale * sn[e] * (weight != nullptr ? v[NEXT ? e ^ 1 : e] : 1.f);
      }
    }
    if (weight != nullptr && mine) {
      float v[8];
      load8_f32(weight + c0, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) wc[e] *= v[e];
    }
    unsigned char* out = reinterpret_cast<unsigned char*>(isq ? a.q_out : a.k_out) +
                         ((t * heads + h0) * repeat * static_cast<int64_t>(a.d) + c0) * static_cast<int64_t>(sizeof(T));
    const int copy = a.d * static_cast<int>(sizeof(T));
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      if (i > 0 && h0 - grp + i * kPass >= heads) break;  // a whole warp
      float x[8];
      unpack8<T>(raw[i], x);
      float2 sums = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 8; e += 2) sums = fma2(make_float2(x[e], x[e + 1]), make_float2(x[e], x[e + 1]), sums);
      float sum = sums.x + sums.y;
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      const float f = inv_norm(sum, mean, a.eps);
      float y[8];
      if constexpr (ODD) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = static_cast<float>(far[i][e]);
      } else if (a.rope_dims > 0) {
        Raw8<T> pair = raw[i];
        if (!NEXT) {
#pragma unroll
          for (int k = 0; k < static_cast<int>(sizeof(T) / 2); ++k) {
            pair.w[k].x = __shfl_sync(kFull, pair.w[k].x, other, LANES);
            pair.w[k].y = __shfl_sync(kFull, pair.w[k].y, other, LANES);
            pair.w[k].z = __shfl_sync(kFull, pair.w[k].z, other, LANES);
            pair.w[k].w = __shfl_sync(kFull, pair.w[k].w, other, LANES);
          }
        }
        float z[8];
        unpack8<T>(pair, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = NEXT ? z[e ^ 1] : z[e];
      }
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float2 z = mul2(make_float2(x[e], x[e + 1]), make_float2(wc[e], wc[e + 1]));
        if (ODD || a.rope_dims > 0) z = fma2(make_float2(y[e], y[e + 1]), make_float2(ws[e], ws[e + 1]), z);
        z = mul2(z, make_float2(f, f));
        x[e] = z.x;
        x[e + 1] = z.y;
      }
      if (h0 + i * kPass < heads && mine) {
        unsigned char* o = out + static_cast<int64_t>(i) * step * repeat;
        if constexpr (sizeof(T) == 2) {
          uint32_t p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            p[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          const uint4 w = make_uint4(p[0], p[1], p[2], p[3]);
          put<kStream>(o, w);
          for (int c = 1; c < repeat; ++c) put<kStream>(o += copy, w);
        } else {
          for (int c = 0; c < repeat; ++c, o += copy) {
            put<kStream>(o, make_float4(x[0], x[1], x[2], x[3]));
            put<kStream>(o + 16, make_float4(x[4], x[5], x[6], x[7]));
          }
        }
      }
    }
  }
}

// One warp per row, any size and alignment: the row passes through shared
// memory so that a pair's two elements may sit anywhere.
template <typename T>
__global__ void __launch_bounds__(kThreads) qk_norm_any_kernel(const treewy_qk a) {
  after_previous();
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
  const float f = row.scale * inv_norm(sum, a.norm == TREEWY_NORM_RMS ? 1.0f / static_cast<float>(a.d) : 1.f, a.eps);
  for (int c = lane; c < a.d; c += 32) y[c] *= row.w != nullptr ? f * __ldg(row.w + c) : f;
  __syncwarp();
  if (a.rope_dims > 0) {
    const float* tab = table_row(a, __ldg(a.position + t), lane == 0);
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

template <typename T, int LANES, int UNROLL, int THREADS, Pairs PAIRS>
cudaError_t launch_passes(const treewy_qk& a, cudaStream_t stream) {
  constexpr int kHeads = UNROLL * 32 / LANES;
  const int q_units = (a.Hq + kHeads - 1) / kHeads, units = q_units + (a.Hk + kHeads - 1) / kHeads;
  // as many warps as the GPU holds (a CTA costs about a nanosecond of the whole
  // GPU's time to start), each with every so many-th token and part
  const int64_t ctas = (a.T * units + THREADS / 32 - 1) / (THREADS / 32);
  const dim3 grid(static_cast<unsigned>(min(ctas, int64_t(152 * 896 / THREADS))));
  const float mean = a.norm == TREEWY_NORM_RMS ? 1.0f / static_cast<float>(a.d) : 1.f;
  return launch_after(qk_norm_kernel<T, LANES, UNROLL, THREADS, PAIRS>, grid, THREADS, stream, a, q_units, units, mean);
}

template <typename T, int LANES>
cudaError_t launch(const treewy_qk& a, cudaStream_t stream) {
  // Many rows: as many heads per warp as its registers hold, and a warp per
  // CTA, a token's parts one after the other (32768 tokens of 18 bf16 heads of
  // 256: 102 us, 6.0 TB/s; 106 us with a CTA per token and part, 118 us without
  // the streaming hints, 128 us with all tokens' first parts first).  Few: the
  // rows spread over more warps (256 tokens of 32 heads of 128: 2.3 us).  Odd
  // pairs: one shape for both (8001 tokens of 24 bf16 heads of 80, 20 of them
  // rotated: 40 us, 67 us element by element).
  constexpr int kMany = sizeof(T) == 2 ? 8 : 4;
  if (a.rope_dims % (a.interleaved ? 8 : 16) != 0) return launch_passes<T, LANES, 4, 32, kOdd>(a, stream);
  const bool many = a.T * (a.Hq + a.Hk) >= int64_t(152) * 64 * (32 / LANES);
  if (a.interleaved)
    return many ? launch_passes<T, LANES, kMany, 32, kNeighbours>(a, stream)
                : launch_passes<T, LANES, 2, 64, kNeighbours>(a, stream);
  return many ? launch_passes<T, LANES, kMany, 32, kLanes>(a, stream) : launch_passes<T, LANES, 2, 64, kLanes>(a, stream);
}

template <typename T>
cudaError_t launch_typed(const treewy_qk& a, cudaStream_t stream) {
  const int64_t rows = a.T * (a.Hq + a.Hk);
  auto on16 = [](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride * sizeof(T)) % 16 == 0;
  };
  bool wide = a.d % 8 == 0 &&
              reinterpret_cast<uintptr_t>(a.rope) % 16 == 0 && reinterpret_cast<uintptr_t>(a.q_weight) % 16 == 0 &&
              reinterpret_cast<uintptr_t>(a.k_weight) % 16 == 0;
  if (a.Hq > 0) wide = wide && on16(a.q, a.q_stride) && on16(a.q_out, 0);
  if (a.Hk > 0) wide = wide && on16(a.k, a.k_stride) && on16(a.k_out, 0);
  if (!wide) {
    constexpr int kRows = kThreads / 32;
    return launch_after(qk_norm_any_kernel<T>, dim3(static_cast<unsigned>((rows + kRows - 1) / kRows)), kThreads, stream, a);
  }
  if (a.d <= 64) return launch<T, 8>(a, stream);
  if (a.d <= 128) return launch<T, 16>(a, stream);
  return launch<T, 32>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm(const treewy_qk& a, cudaStream_t stream) {
  return a.dtype == TREEWY_DTYPE_BF16 ? launch_typed<__nv_bfloat16>(a, stream)
                                      : launch_typed<float>(a, stream);
}

}  // namespace treewy
