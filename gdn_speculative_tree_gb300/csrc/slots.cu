// slots.cu -- moves between slots of the state pools of all layers
// (treewy_copy_slots): block dst[i] <- block src[i], or zeros.
//
// Bound by HBM: each CTA copies one piece of one move in one layer, every
// 16-byte word of it in flight at once.  A CTA first looks through the whole
// list for a move that meets its own (two words per move from L2), so that
// which moves are made does not depend on the order in which CTAs run, and no
// move reads what another one writes.
#include "treewy_device.cuh"
#include "treewy_internal.h"

namespace treewy {
namespace {

constexpr int kThreads = 256;
constexpr int kWords = 8;  // words of a thread per piece

template <typename W>
__global__ void __launch_bounds__(kThreads)
    copy_slots_kernel(const treewy_slots a, int64_t words, int pieces, int64_t layer_stride) {
  after_previous();
  // pieces of one block are neighbours, then layers, then moves
  const int piece = static_cast<int>(blockIdx.x % pieces);
  const unsigned rest = blockIdx.x / pieces;
  const int layer = static_cast<int>(rest % a.layers), i = static_cast<int>(rest / a.layers);
  const int s = __ldg(a.src + i), d = __ldg(a.dst + i);
  bool clash = false;
  if (s != d) {
    for (int j = threadIdx.x; j < a.n; j += kThreads) {
      const int sj = __ldg(a.src + j), dj = __ldg(a.dst + j);
      // another move's destination; one that leaves its block as it is writes nothing
      clash |= j != i && sj != dj && (dj == d || (dj == s && s >= 0));
    }
  }
  clash = __syncthreads_or(clash);
  const bool range = s < -1 || s >= a.num_slots || d < 0 || d >= a.num_slots;
  if (clash || range) {
    if (piece == 0 && layer == 0 && threadIdx.x == 0)
      atomicOr(a.status + i, (clash ? TREEWY_STATUS_SLOT_CLASH : 0) | (range ? TREEWY_STATUS_BAD_SLOT : 0));
    return;
  }
  if (s == d) return;
  unsigned char* pool = reinterpret_cast<unsigned char*>(a.state) + layer * layer_stride;
  const W* from = reinterpret_cast<const W*>(pool + (s < 0 ? 0 : s) * a.slot_bytes);
  W* to = reinterpret_cast<W*>(pool + d * a.slot_bytes);
  const int64_t w0 = static_cast<int64_t>(piece) * (kThreads * kWords) + threadIdx.x;
  W x[kWords];
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    const int64_t w = w0 + k * kThreads;
    x[k] = W{};
    if (s >= 0 && w < words) x[k] = from[w];
  }
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    const int64_t w = w0 + k * kThreads;
    if (w < words) to[w] = x[k];
  }
}

template <typename W>
cudaError_t launch(const treewy_slots& a, int64_t layer_stride, cudaStream_t stream) {
  const int64_t words = a.slot_bytes / static_cast<int64_t>(sizeof(W));
  const int64_t pieces = (words + kThreads * kWords - 1) / (kThreads * kWords);
  const int64_t copies = static_cast<int64_t>(a.layers) * a.n;
  if (pieces > 0x7fffffff / copies) return cudaErrorNotSupported;
  return launch_after(copy_slots_kernel<W>, dim3(static_cast<unsigned>(pieces * copies)), kThreads, stream, a, words,
                      static_cast<int>(pieces), layer_stride);
}

}  // namespace

cudaError_t launch_copy_slots(const treewy_slots& a, cudaStream_t stream) {
  const int64_t stride = a.layer_stride != 0 ? a.layer_stride : a.num_slots * a.slot_bytes;
  const uint64_t all = reinterpret_cast<uintptr_t>(a.state) | static_cast<uint64_t>(a.slot_bytes) |
                       static_cast<uint64_t>(stride);
  if (all % 16 == 0) return launch<uint4>(a, stride, stream);
  if (all % 4 == 0) return launch<uint32_t>(a, stride, stream);
  return launch<uint8_t>(a, stride, stream);
}

}  // namespace treewy
