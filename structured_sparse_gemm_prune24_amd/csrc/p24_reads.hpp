// Where the GEMM kernels' direct-to-LDS buffer loads read: the parts of their
// addresses that may lie past a matrix (host and device).
//
// A raw buffer load drops the lanes whose vector offset lies past the resource.
// The scalar offset is no sure part of that check: it is described as left out of
// it, or as taken off the size first, which wraps once it is the larger.  So a
// row or token that may lie past the matrix goes into the vector offset, where
// it alone decides; whole blocks of rows, which are uniform, stop at the last
// one (their results are not stored); and the scalar offset otherwise only
// advances along K, inside every row.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define P24_HD __host__ __device__ __forceinline__
#else
#define P24_HD inline
#endif

namespace p24 {

P24_HD int last_of(int i, int count) { return i < count ? i : count - 1; }

// bf16 products.  A: 1 KiB load q of a K step is block q % asteps of row block q / asteps,
// of which the matrix has `row_blocks` from the tile's first on, `row_steps` blocks each.
P24_HD uint32_t a_scalar(int q, int asteps, int64_t row_steps, int row_blocks) {
  return (uint32_t)((last_of(q / asteps, row_blocks) * row_steps + q % asteps) * 1024);
}
// Metadata: load `group` of the `groups` from the tile's first on, `pairs` KiB each.
P24_HD uint32_t meta_scalar(int group, int64_t pairs, int groups) {
  return (uint32_t)(last_of(group, groups) * pairs * 1024);
}
// X^T (N x K): load q of a tile fills LDS rows 8 q on, row' = 8 q + lane / 8 with n = row' ^ (q & 1)
// and chunk (lane & 7) ^ (n & 7).  `rows`: from load q to load q + more, `more` even.
P24_HD uint32_t xt_vector(int lane, int q, int64_t ldx) {
  const int n = 8 * q + ((lane >> 3) ^ (q & 1)), c = (lane & 7) ^ (n & 7);
  return (uint32_t)((n * ldx + 8 * c) * 2);
}
P24_HD uint32_t xt_rows(int more, int64_t ldx) { return (uint32_t)(8 * more * ldx * 2); }

}  // namespace p24
