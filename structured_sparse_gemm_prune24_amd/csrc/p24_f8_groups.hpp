// Tiles of BN rows over the ranges of rows that belong to the experts of a grouped product.
//
// `offsets` lies on the device: the launch knows an upper bound of the tiles only, and each block finds
// its own.  Lane l of a wave holds expert 64 chunk + l's range; an inclusive sum over the lanes gives
// the tiles up to it.  Ranges are clipped to [0, rows], so that no offset leads outside the output.
#pragma once

#include "p24_device.hpp"

namespace p24 {

struct F8Groups {
  const int* offsets;   // experts + 1
  const int* tokens;    // row of X of each row of Y, or nullptr: the same row
  int experts, rows;    // rows of Y
  int x_rows;           // rows of X
};

template <int BN>
struct F8GroupSearch {
  const F8Groups g;
  const int lane;
  int chunk = -1;          // experts 64 chunk on are held
  uint32_t before = 0;     // tiles ahead of them
  uint32_t held = 0;       // tiles of theirs
  uint32_t upto = 0;       // this lane's: tiles up to its expert, itself included
  int lo = 0, n = 0;       // its rows

  __device__ __forceinline__ F8GroupSearch(const F8Groups& groups) : g(groups), lane(threadIdx.x & 63) {}

  __device__ __forceinline__ void range(int c, int& first, int& count) const {
    const int e = 64 * c + lane;
    const int a = e < g.experts ? g.offsets[e] : 0, b = e < g.experts ? g.offsets[e + 1] : 0;
    first = min(max(a, 0), g.rows);
    count = max(min(b, g.rows) - first, 0);
  }
  static __device__ __forceinline__ uint32_t tiles_of(int rows) { return ((uint32_t)rows + BN - 1) / BN; }

  // tiles of all experts
  __device__ __forceinline__ uint32_t total() const {
    uint32_t sum = 0;
    for (int c = 0; 64 * c < g.experts; ++c) {
      int first, count;
      range(c, first, count);
      sum += tiles_of(count);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    return __builtin_amdgcn_readfirstlane(sum);
  }
  // The expert of tile t, its first row and rows, and its first tile.  t does not fall from call to call;
  // false past the last tile.
  __device__ __forceinline__ bool find(uint32_t t, int& expert, int& first, int& count, uint32_t& first_tile) {
    while (t >= before + held) {
      if (64 * (chunk + 1) >= g.experts) return false;
      before += held;
      ++chunk;
      range(chunk, lo, n);
      upto = tiles_of(n);
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t other = __shfl_up(upto, o);
        upto += lane >= o ? other : 0;
      }
      held = __builtin_amdgcn_readlane(upto, 63);
    }
    const int l = __builtin_ctzll(__ballot(before + upto > t));
    expert = 64 * chunk + l;
    first = __builtin_amdgcn_readlane(lo, l);
    count = __builtin_amdgcn_readlane(n, l);
    first_tile = before + __builtin_amdgcn_readlane(upto, l) - tiles_of(count);
    return true;
  }
};

}  // namespace p24
