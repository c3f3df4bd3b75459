// cache_device.cuh -- what the kernels of treewy_attend and treewy_append share.
#pragma once
#include <cuda_fp8.h>

#include "treewy_device.cuh"

namespace treewy {

// One request's rows and context, and the status bits that refuse it.
struct CacheRequest {
  int lo, N, len, err;
};
__device__ __forceinline__ CacheRequest cache_request(const treewy_cache& c, const int32_t* offset, int r, int64_t T, int max_rows,
                                                      int64_t max_len) {
  CacheRequest q;
  q.lo = __ldg(offset + r);
  const int hi = __ldg(offset + r + 1);
  q.len = __ldg(c.length + r);
  const int64_t n = static_cast<int64_t>(hi) - q.lo;
  q.err = 0;
  if (q.lo < 0 || hi > T) q.err |= TREEWY_STATUS_BAD_TREE;
  if (n < 0 || n > max_rows) q.err |= TREEWY_STATUS_TOO_MANY_NODES;
  if (q.len < 0 || q.len > max_len || q.len > static_cast<int64_t>(c.max_pages) * c.page_len) q.err |= TREEWY_STATUS_BAD_PAGE;
  q.N = q.err != 0 ? 0 : static_cast<int>(n);
  return q;
}

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// Two f32 to e4m3, rounded to nearest, beyond 448 to 448 (NaN stays NaN); x0 in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float x0, float x1) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}
// The two values of an e4m3 pair, as f16 (exactly).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
  return r;
}

// The least e, -40 at least, with x <= 448 * 2^e for a finite x >= 0 (448 is
// 1.75 * 2^8), as 2^e.
__device__ __forceinline__ float scale_for(float x) {
  const uint32_t b = __float_as_uint(x);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -40) + 127) << 23);
}

// |x| for a page's largest value: what is not finite does not count.
__device__ __forceinline__ float size_of(float x) {
  const float a = fabsf(x);
  return a <= 3.4028234664e38f ? a : 0.f;
}

// Parents of N nodes in shared memory: every one in [-1, n).  All threads call
// it, at least N of them; chains where `parent` is NULL.
__device__ __forceinline__ bool load_parents(int* to, const int32_t* parent, int lo, int N) {
  bool bad = false;
  const int t = threadIdx.x;
  if (t < N) {
    const int p = parent != nullptr ? __ldg(parent + lo + t) : t - 1;
    bad = p < -1 || p >= t;
    to[t] = bad ? -1 : p;
  }
  return !__syncthreads_or(bad);
}

}  // namespace treewy
