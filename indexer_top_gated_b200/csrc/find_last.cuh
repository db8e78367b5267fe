// find_last.cuh - block-wide search in a monotone sequence, for kernels whose CTAs look up the
// sequence that owns their rows.
#pragma once

#include "common.cuh"

namespace dsa {

// The last b in [0, n) with le(b), where le holds for 0 and for a prefix.  Every thread of the
// CTA calls it.  A short sequence is read in rounds of THREADS loads that do not wait for one
// another (64 sequences: one round against six dependent loads), a long one bisected.
template <int THREADS, typename F>
DSA_DEV int find_last(int n, F le) {
  int b = 0;
  if (n <= 4 * THREADS) {
    for (int i = 1; i < n; i += THREADS) {
      const int at = i + (int)threadIdx.x;
      b += __syncthreads_count(at < n && le(at));
    }
    return b;
  }
  int hi = n - 1;
  while (b < hi) {
    const int mid = (b + hi + 1) >> 1;
    if (le(mid)) b = mid;
    else hi = mid - 1;
  }
  return b;
}

}  // namespace dsa
