// The grouped product's walk over tiles on the CPU (test infrastructure): p24_f8_groups.hpp as it is, its wave
// instructions emulated by 64 fibers that meet at each of them.
#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <vector>

namespace model {

struct Wave {
  ucontext_t scheduler, lanes[64];
  std::vector<char> stacks = std::vector<char>(64 * 65536);
  uint64_t slots[2][64];
  int turn[64], lane = 0;
  void (*body)(void*);
  void* arg;
} wave;

// The lanes' values once all of them have come here.
const uint64_t* exchange(uint64_t v) {
  const int l = wave.lane, side = wave.turn[l]++ & 1;
  wave.slots[side][l] = v;
  swapcontext(&wave.lanes[l], &wave.scheduler);
  return wave.slots[side];
}

void run_lane() { wave.body(wave.arg); }

// Runs body(arg) on 64 lanes; false if they do not meet at the same instructions.
bool run(void (*body)(void*), void* arg, const bool* done) {
  wave.body = body;
  wave.arg = arg;
  for (int l = 0; l < 64; ++l) {
    getcontext(&wave.lanes[l]);
    wave.lanes[l].uc_stack = {wave.stacks.data() + l * 65536, 0, 65536};
    wave.lanes[l].uc_link = &wave.scheduler;
    wave.turn[l] = 0;
    makecontext(&wave.lanes[l], run_lane, 0);
  }
  for (;;) {
    int ended = 0;
    for (wave.lane = 0; wave.lane < 64; ++wave.lane) {
      if (!done[wave.lane]) swapcontext(&wave.scheduler, &wave.lanes[wave.lane]);
      ended += done[wave.lane];
    }
    if (ended == 64) return true;
    if (ended) return false;
  }
}

struct Index {
  struct X {
    operator unsigned() const { return (unsigned)wave.lane; }
  } x;
} thread;

}  // namespace model

#define __device__
#define __forceinline__ inline
#define threadIdx model::thread
#define __shfl_xor(v, o) ((decltype(v))model::exchange((uint64_t)(v))[model::wave.lane ^ (o)])
#define __shfl_up(v, o) ((decltype(v))model::exchange((uint64_t)(v))[model::wave.lane < (o) ? model::wave.lane : model::wave.lane - (o)])
#define __builtin_amdgcn_readlane(v, l) ((decltype(v))model::exchange((uint64_t)(v))[l])
#define __builtin_amdgcn_readfirstlane(v) ((decltype(v))model::exchange((uint64_t)(v))[0])
inline uint64_t model_ballot(bool p) {
  const uint64_t* v = model::exchange(p);
  uint64_t mask = 0;
  for (int l = 0; l < 64; ++l) mask |= v[l] << l;
  return mask;
}
#define __ballot model_ballot
using std::max;
using std::min;

#include "../../structured_sparse_gemm_prune24_amd/csrc/p24_f8_groups.hpp"

namespace {

using namespace p24;

struct Walk {
  F8Groups groups;
  uint32_t block, grid, nbm;
  int* cover;       // of a row: how often its nbm row blocks are computed
  long bad, steps;
  bool done[64];
};

// A block of k_gemm_f8_grouped, its tiles looked at and not computed.
template <int BN>
void walk(void* arg) {
  Walk& w = *(Walk*)arg;
  const int lane = model::wave.lane;
  F8GroupSearch<BN> search(w.groups);
  const uint32_t tiles = search.total() * w.nbm;
  F8GroupTile t;
  long steps = 0;
  for (uint32_t i = w.block; i < tiles; i += w.grid) {
    if (++steps > 100000) break;
    const bool found = search.tile(i, tiles, w.nbm, t);
    if (lane) continue;
    ++w.steps;
    const bool inside = found && t.expert >= 0 && t.expert < w.groups.experts && t.first >= 0 && t.count > 0 &&
                        (int64_t)t.first + t.count <= w.groups.rows && t.bm < w.nbm &&
                        t.bn < F8GroupSearch<BN>::tiles_of(t.count);
    if (!inside) {
      ++w.bad;
      continue;
    }
    for (int r = (int)t.bn * BN; r < std::min(((int)t.bn + 1) * BN, t.count); ++r) ++w.cover[t.first + r];
  }
  w.done[lane] = true;
}

template <int BN>
long walk_all(Walk w, int fit) {
  const int64_t most = f8_most_tiles(w.groups.rows, w.groups.experts, BN) * w.nbm;
  w.grid = (uint32_t)std::min<int64_t>(most, fit);
  for (w.block = 0; w.block < w.grid; ++w.block) {
    std::fill(w.done, w.done + 64, false);
    if (!model::run(walk<BN>, &w, w.done)) return -1;
  }
  // the launch's bound of the tiles holds
  return w.bad + (w.steps > most ? w.steps - most : 0);
}

}  // namespace

// A block of k_f8_tokens_grouped: tile w.block of 32 rows.
void few(void* arg) {
  Walk& w = *(Walk*)arg;
  F8GroupSearch<32> search(w.groups);
  int expert, first, count;
  uint32_t first_tile;
  const bool found = search.find(w.block, expert, first, count, first_tile);
  if (model::wave.lane == 0 && found) {
    const bool inside = expert >= 0 && expert < w.groups.experts && first >= 0 && count > 0 && (int64_t)first + count <= w.groups.rows &&
                        first_tile <= w.block && w.block - first_tile < F8GroupSearch<32>::tiles_of(count);
    if (!inside) ++w.bad;
    else
      for (int r = (int)(w.block - first_tile) * 32; r < std::min((int)(w.block - first_tile + 1) * 32, count); ++r) ++w.cover[first + r];
  }
  w.done[model::wave.lane] = true;
}

// Tiles outside the experts, the rows or the row blocks, and tiles past the launch's bound, over all blocks of a launch of
// at most `fit` blocks (a multiple of 8).
extern "C" long group_walk(int bn, const int* offsets, int experts, int rows, int nbm, int fit, int* cover) {
  Walk w{};
  w.groups.offsets = offsets;
  w.groups.experts = experts;
  w.groups.rows = rows;
  w.groups.x_rows = rows;
  w.nbm = (uint32_t)nbm;
  w.cover = cover;
  switch (bn) {
    case 32: return walk_all<32>(w, fit);
    case 64: return walk_all<64>(w, fit);
    case 192: return walk_all<192>(w, fit);
    case 256: return walk_all<256>(w, fit);
  }
  return -1;
}

// The same of the kernel for few rows, whose grid holds every tile that there could be (one row block).
extern "C" long group_few(const int* offsets, int experts, int rows, int* cover) {
  Walk w{};
  w.groups.offsets = offsets;
  w.groups.experts = experts;
  w.groups.rows = rows;
  w.cover = cover;
  const int64_t most = f8_most_tiles(rows, experts, 32);
  for (w.block = 0; w.block < most; ++w.block) {
    std::fill(w.done, w.done + 64, false);
    if (!model::run(few, &w, w.done)) return -1;
  }
  return w.bad;
}
