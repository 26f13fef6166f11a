// ranges.cuh -- document table -> the interval of keys that each row attends to.
//
// Several documents (samples, requests) packed into one sequence: row i of the
// document [s, e) with a prefix of p rows attends to
//   document       [s, e)
//   prefix causal  [s, max(s + p, i + 1))   the prefix in full, causal behind it
//   prefix block   [s, s + p) for i < s + p, else [s, e): the prefix does not
//                  look at the rest, so its K and V do not depend on the rest
// and rows in no document to nothing.  One thread per row, binary search over
// the starts; launch-bound at every size (8 bytes written per row; 14,098 rows 2.8 us).
#pragma once

#include "common.cuh"

namespace h3 {

__global__ void __launch_bounds__(256) key_ranges_kernel(const int32_t* __restrict__ starts,
                                                         const int32_t* __restrict__ prefix, int n_docs, int n_rows,
                                                         int mode, int2* __restrict__ ranges, int err_slot) {
  begin_after_predecessor(starts, prefix);
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long tid = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  // a table that does not ascend inside [0, n_rows] is an input fault; its rows
  // still get intervals inside [0, n_rows)
  for (long long d = tid; d <= n_docs; d += step) {
    const int s = starts[d];
    if (s < 0 || s > n_rows || (d < n_docs && starts[d + 1] < s)) raise_error(err_slot, DEVERR_INPUT);
    if (d < n_docs && prefix != nullptr && prefix[d] < 0) raise_error(err_slot, DEVERR_INPUT);
  }
  for (long long i = tid; i < n_rows; i += step) {
    const int r = static_cast<int>(i);
    int lo = 0, hi = n_docs;               // documents that end at or before r
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid + 1] <= r) lo = mid + 1; else hi = mid;
    }
    int2 out = make_int2(0, 0);
    if (lo < n_docs && starts[lo] <= r) {
      const int s = max(starts[lo], 0), e = min(starts[lo + 1], n_rows);
      const int p = prefix != nullptr && mode != H3_MASK_DOCUMENT ? s + min(max(prefix[lo], 0), e - s) : s;
      out.x = s;
      out.y = mode == H3_MASK_PREFIX_CAUSAL ? max(p, r + 1) : mode == H3_MASK_PREFIX_BLOCK && r < p ? p : e;
    }
    ranges[i] = out;
  }
}

}  // namespace h3
