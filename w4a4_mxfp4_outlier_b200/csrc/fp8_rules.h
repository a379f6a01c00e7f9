// Size rules of the 8-bit product that need no CUDA types.
#pragma once

#include <cstdint>

namespace w4a4 {

// Few-token kernel: into how many ranges K is split, one for each CTA of a
// cluster: as many as let all clusters run at once.  fits[c]: how many clusters of
// c CTAs the device holds (B200, c = 2, 3, 4, 6, 8: 148, 90, 66, 44, 30).  That is
// fewer than its CTA slots divided by c, since a cluster lives inside one group of
// SMs.  linear(), us, clusters by the slots alone and by this rule: 1 token, 5120 ->
// 4608, 36 tiles, clusters of 8 12.6, of 6 9.8; 5120 -> 6144, 48 tiles, clusters
// of 6 14.9, of 4 10.9; 48 tokens, 5120 -> 12288, 96 tiles, of 3 24.3, of 2 19.9.
constexpr int kFewSplits[] = {2, 3, 4, 6, 8};
constexpr int kFewMaxSplit = 8;
inline int fp8_few_split(int64_t tiles, int nkb, const int* fits) {
  int split = 1;
  for (const int c : kFewSplits)
    if (tiles <= fits[c] && c <= nkb) split = c;
  return split;
}

// Clusters that fit where `per_sm` CTAs run on an SM, from the number that the
// occupancy query gives and the CTAs per SM that it counted.  (For kernels that
// allocate tensor memory it counts one, though two run at once.)
inline int fp8_clusters_that_fit(int queried, int counted_per_sm, int per_sm) {
  return counted_per_sm > 0 ? queried * per_sm / counted_per_sm : 0;
}

}  // namespace w4a4
