// Tiles of BN rows over the ranges of rows that belong to the experts of a grouped product.
//
// `offsets` lies on the device: the launch knows an upper bound of the tiles only, and each block finds
// its own.  Lane l of a wave holds expert 64 chunk + l's range; an inclusive sum over the lanes gives
// the tiles up to it.  Ranges are clipped to [0, rows], so that no offset leads outside the output, and offsets
// that fall have no tiles: their ranges could overlap, and the tiles be more than the launch and the walk allow for.
#pragma once

#include "p24_places.hpp"
#ifdef __HIP__
#include "p24_device.hpp"
#endif

namespace p24 {

struct F8Groups {
  const int* offsets;   // experts + 1
  const int* tokens;    // row of X of each row of Y, or nullptr: the same row
  int experts, rows;    // rows of Y
  int x_rows;           // rows of X
};

// Most tiles of bn rows that `rows` rows of `experts` experts can take: every expert with rows has one part tile at most.
P24_HD int64_t f8_most_tiles(int64_t rows, int64_t experts, int bn) {
  const int64_t live = experts < rows ? experts : rows;
  return (rows - live) / bn + live;
}

// A tile: row block bm and rows bn BN on of an expert's `count` rows from `first` on.
struct F8GroupTile {
  int expert, first, count;
  uint32_t bm, bn;
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

  // false where the offsets fall
  __device__ __forceinline__ bool range(int c, int& first, int& count) const {
    const int e = 64 * c + lane;
    const int a = e < g.experts ? g.offsets[e] : 0, b = e < g.experts ? g.offsets[e + 1] : 0;
    first = min(max(a, 0), g.rows);
    count = max(min(b, g.rows), first) - first;      // (a difference of any two ints would wrap)
    return a <= b;
  }
  static __device__ __forceinline__ uint32_t tiles_of(int rows) { return ((uint32_t)rows + BN - 1) / BN; }

  // tiles of all experts; 0 if the offsets fall
  __device__ __forceinline__ uint32_t total() const {
    uint32_t sum = 0;
    bool rise = true;
    for (int c = 0; 64 * c < g.experts; ++c) {
      int first, count;
      rise &= range(c, first, count);
      sum += tiles_of(count);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    return __ballot(!rise) ? 0 : __builtin_amdgcn_readfirstlane(sum);
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
  // Tile i of `tiles`, total() times the nbm row blocks.  A block asks for i, i + grid, ...: the grid is a multiple of the
  // XCDs' number or holds all tiles, so that xcd_remap's numbers do not fall.
  __device__ __forceinline__ bool tile(uint32_t i, uint32_t tiles, uint32_t nbm, F8GroupTile& t) {
    const uint32_t b = xcd_remap(i, tiles);
    uint32_t first_tile;
    if (!find(b / nbm, t.expert, t.first, t.count, first_tile)) return false;   // (never: b < tiles)
    f8_place(b - first_tile * nbm, nbm, tiles_of(t.count), t.bm, t.bn);
    return true;
  }
};

}  // namespace p24
