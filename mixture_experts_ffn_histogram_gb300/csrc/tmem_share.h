// When kernels of two streams share an SM.  tcgen05.alloc waits, without a
// limit, until its columns are free.  A CTA whose cluster needs columns on two
// SMs may hold them on one and wait on the other, and two such clusters that
// hold what the other waits for would wait for ever.  So kernels of clusters
// take so much shared memory that CTAs which fit an SM together never ask for
// more than its 512 columns.  (A CTA without a cluster ends by itself and
// frees its columns.)
#pragma once

#include <stddef.h>

namespace moe {

constexpr size_t kSmSmem = 228 * 1024;   // of an SM, for all of its blocks
constexpr size_t kBlockSmem = 1024;      // what the system takes for each block
constexpr int kSmTmemCols = 512;

// Dynamic shared memory that a kernel of CTA pairs with all 512 columns takes
// at least; each such kernel asserts it, and a cluster's CTA of any other
// kernel asserts that it does not fit beside so much.
constexpr size_t kLeastPairSmem = 185 * 1024;

constexpr bool fits_beside_pair(size_t dynamic_bytes) {
  return dynamic_bytes + kLeastPairSmem + 2 * kBlockSmem <= kSmSmem;
}

}  // namespace moe
