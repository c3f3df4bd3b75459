// serving_device.cuh -- what the kernels of treewy_extend share.
#pragma once
#include "treewy.h"

namespace treewy {

constexpr int kRanked = 128;  // sequences that are put in order

// The sequence of the CTAs that come idx-th: the longest first, so that a long
// one does not begin when the others are done (13 sequences of 1 to 2500 tokens
// in order of their number: 328 us, 263 us so).  Every CTA finds it for itself
// from all lengths, in less than half a microsecond for 128; more sequences
// keep their order.  All threads of the CTA call it, at least kRanked of them.
__device__ __forceinline__ int longest_first(const treewy_seqs& a, int idx) {
  __shared__ int len[kRanked];
  __shared__ int found;
  if (a.R == 1 || a.R > kRanked) return idx;
  const int t = threadIdx.x;
  int mine = 0;
  if (t < a.R) {
    // any order will do for offsets that are wrong: they are refused by number
    mine = static_cast<int>(static_cast<unsigned>(__ldg(a.seq_offset + t + 1)) -
                            static_cast<unsigned>(__ldg(a.seq_offset + t)));
    len[t] = mine;
  }
  __syncthreads();
  if (t < a.R) {
    int before = 0;
    for (int i = 0; i < a.R; ++i) before += len[i] > mine || (len[i] == mine && i < t);
    if (before == idx) found = t;
  }
  __syncthreads();
  return found;
}

}  // namespace treewy
