// dsa_paged_split.h - how the rows of the dense paged attention are shared out among the CTAs: plain
// integers, for the device and for host code.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define DSA_SPLIT_FN __host__ __device__ __forceinline__
#else
#define DSA_SPLIT_FN inline
#endif

namespace dsa {
namespace paged {

constexpr int kMaxCtas = 192;  // the join's lists (its threads look at 256 CTAs)

// First cost of CTA c's share, floor(c * total / G): G is at most kMaxCtas < 2^8, total below 2^31.
DSA_SPLIT_FN int share(int c, int total, int G) {
  const uint32_t q = (uint32_t)total / (uint32_t)G, r = (uint32_t)total - q * (uint32_t)G;
  return (int)((uint32_t)c * q + (uint32_t)c * r / (uint32_t)G);
}

// Whether a record of the split can be one that join block `block` has to work on: a row of the call (the
// block's own when there are at most G rows), the CTAs that start and finish it, the split's cost. After
// a wait that ran out the scheduler leaves without writing the rest of the records, and the
// workspace may hold anything there.
DSA_SPLIT_FN bool record_valid(int row, int first, int last, int total, int64_t nrows, int G, int block) {
  return row >= 0 && row < nrows && (nrows > G || row == block) && first >= 0 && first <= last && last < G && total > 0;
}

}  // namespace paged
}  // namespace dsa
