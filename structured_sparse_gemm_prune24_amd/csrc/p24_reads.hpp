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

}  // namespace p24
