// spmm24_f8_grouped: the 8-bit 2:4 product of experts with ragged numbers of rows, on the tiles of
// p24_f8_gemm.hpp.
//
// How many tiles there are is known on the device only.  Blocks of the block tiles walk over them
// (as many as fit the chip at once, tile b, b + grid, ...), so that an upper bound of the tiles
// costs nothing; a tile belongs to one expert, whose part of the operands it takes as a product of
// its own.  The kernel for few rows has a block for every tile that there could be.
#include <cmath>
#include <cstdlib>
#include <cstring>

#include "../../include/prune24_experts.h"
#include "p24_api_internal.hpp"
#include "p24_f8_cost.hpp"
#include "p24_f8_gemm.hpp"

namespace p24 {

struct F8GroupedArgs {
  F8Args a;          // of expert 0 and all rows
  F8Groups groups;
  int64_t w_bytes;   // of an expert's weight
};

// The part of one expert: rows first on, `count` of them.
template <typename OutT>
__device__ __forceinline__ F8Args f8_part(const F8GroupedArgs& g, int expert, int first, int count, F8RowMap& rows) {
  F8Args a = g.a;
  a.W += expert * g.w_bytes;
  a.w_scale += (int64_t)expert * a.M;
  if (a.bias) a.bias += (int64_t)expert * a.M;
  a.Y = (OutT*)a.Y + first * a.ldy;
  a.N = count;
  a.residual = nullptr;
  a.res_dma = 0;
  rows.last = (uint32_t)g.groups.x_rows - 1;
  rows.tokens = g.groups.tokens;
  if (rows.tokens) {
    rows.tokens += first;
  } else {
    a.X += first * a.ldx;
    a.x_scale += first;
  }
  return a;
}

template <int W, typename OutT>
__global__ __launch_bounds__(W * 64) void k_f8_tokens_grouped(const F8GroupedArgs g) {
  int expert, first, count;
  uint32_t first_tile;
  F8GroupSearch<32> search(g.groups);
  if (!search.find(blockIdx.y, expert, first, count, first_tile)) return;
  F8RowMap rows;
  const F8Args a = f8_part<OutT>(g, expert, first, count, rows);
  f8_tokens_tile<W, OutT, true>(a, (int)(blockIdx.y - first_tile) * 32, rows);
}

template <int BM, int BN, int WGM, int WGN, int LW, int KG, typename OutT>
__global__ __launch_bounds__(WGM * WGN * KG * 64) void k_gemm_f8_grouped(const F8GroupedArgs g) {
  using C = F8Tile<BM, BN, WGM, WGN, LW, KG>;
  constexpr bool CHAIN = f8_chained<BM, BN, WGM, WGN, LW, KG, OutT>();
  __shared__ __attribute__((aligned(1024)))
  uint8_t lds[f8_lds_bytes<BM, BN, WGM, WGN, LW, KG, OutT>() + (CHAIN ? F8Chain<C>::TOKENS : 0)];
  F8GroupSearch<BN> search(g.groups);
  const uint32_t nbm = g.a.nbm, tiles = search.total() * nbm;
  F8Chain<C> chain;
  F8GroupTile tile;
  uint32_t i = blockIdx.x;
  if (i >= tiles || !search.tile(i, tiles, nbm, tile)) return;
  for (;;) {
    i += gridDim.x;
    F8GroupTile next = tile;
    const bool more = i < tiles && search.tile(i, tiles, nbm, next);
    F8RowMap rows;
    const F8Args a = f8_part<OutT>(g, tile.expert, tile.first, tile.count, rows);
    if constexpr (CHAIN) {
      F8RowMap next_rows;
      const F8Args n = f8_part<OutT>(g, next.expert, next.first, next.count, next_rows);
      chain.more = more;
      chain.W = n.W;
      chain.X = n.X;
      chain.tokens = next_rows.tokens;
      chain.N = n.N;
      chain.m0 = (int)next.bm * BM;
      chain.n0 = (int)next.bn * BN;
    }
    f8_block_tile<BM, BN, WGM, WGN, LW, KG, OutT, true, CHAIN>(a, lds, (int)tile.bm * BM, (int)tile.bn * BN, rows, &chain);
    if (!more) return;
    tile = next;
    // the next tile's loads go where this one's epilogue reads
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
}

static int64_t f8_most_tiles(const F8GroupedArgs& g, int bn) { return f8_most_tiles(g.groups.rows, g.groups.experts, bn); }

template <int W, typename OutT>
static p24_status launch_tokens_grouped(const F8GroupedArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)((g.a.M + 31) / 32), (unsigned)f8_most_tiles(g, 32));
  hipLaunchKernelGGL((k_f8_tokens_grouped<W, OutT>), grid, dim3(W * 64), 0, st, g);
  return launch_status();
}

template <int BM, int BN, int WGM, int WGN, int LW, int KG, typename OutT>
static p24_status launch_tile_grouped(F8GroupedArgs g, hipStream_t st) {
  g.a.nbm = (g.a.M + BM - 1) / BM;
  const int64_t most = f8_most_tiles(g, BN) * g.a.nbm;
  if (most >= (1ll << 31)) return P24_ERR_UNSUPPORTED;
  // blocks that fit the 256 CUs at once; a multiple of the 8 XCDs
  constexpr int LDS = f8_lds_bytes<BM, BN, WGM, WGN, LW, KG, OutT>();
  const int64_t fit = 256 * (160 * 1024 / LDS < 4 ? 160 * 1024 / LDS : 4);
  hipLaunchKernelGGL((k_gemm_f8_grouped<BM, BN, WGM, WGN, LW, KG, OutT>), dim3((unsigned)(most < fit ? most : fit)),
                     dim3(WGM * WGN * KG * 64), 0, st, g);
  return launch_status();
}

// Which kernel.  Where the rows lie is not known here: the experts' numbers of rows are taken as
// exponentially distributed, so that an expert with a rows on average has 1 / (1 - exp(-BN / a)) tiles of BN rows.
// With that many blocks the kernel of the fewest microseconds by forecast wins (p24_f8_cost.hpp).  Over 60 shapes drawn
// at random (1 to 8192 tokens of 2 to 128 experts) it is 3.1 % behind the fastest, fp32 outputs 1.7 % (geometric means), a
// tenth of the shapes 8 and 4 %, the worst 21 % for both.
// Measured, us (T tokens of k experts, of E with M x K; bf16 unless said), * the one that is taken:
//   4096 of 8, 64 of 4096 x 2048   256x256 227*, 256x192 247, 256x128 273, 128x128 317, 64x64 499
//   2048 of 8, 128 of 2048 x 2048  256x256 104*, 256x128 109, 128x128 113, 256x192 121, 64x64 162
//   512 of 2, 8 of 4096 x 4096     256x128 23.4, 256x192 26.2, 128x128 28.0*, 64x32 38.4; fp32 256x128 38.5, 128x128 41.7*
//   1571 of 2, 7 of 1000 x 1088    128x128 10.1, 128x64 10.6*, 64x64 12.4; fp32 128x128 14.1*, 128x64 14.7, 64x64 16.4
//   64 of 4, 32 of 4096 x 4096     128x64 58.5, 64x32 59.6*, 64x64 63.7, tokens 72; fp32 64x32 63.1*, 128x64 63.0
//   1 of 8, 128 of 2048 x 4096     tokens 8.4*, 64x64 12.8, 64x32 13.1
//
// What bounds the largest (measured inside the kernel, 256x256 of the first line): a tile takes 21.5 us, 15 of them its
// 16 steps, 4.4 its epilogue, 1.8 the start of the next.  A step of 0.94 us takes 0.85 without the multiplies, 0.65
// without the loads, 0.86 with half of its rows dead and 0.89 with every weight in the L2: its bytes and its hits do not
// set it, which leaves the loads' latency, two steps of them in flight and one barrier a step.
enum F8GroupedKernel { G_TOKENS, G_64x32, G_64x64, G_128x64, G_128x128, G_256x128, G_256x192, G_256x256, G_KERNELS };

constexpr TileCost GROUPED_BF16[G_KERNELS] = {
    {32, 32, 4.02, 0.066, 0.46, 0.137},  {64, 32, 5.83, 0.237, 0.66, 0.138},   {64, 64, 5.85, 0.221, 0.93, 0.160},
    {128, 64, 5.84, 0.232, 1.75, 0.283}, {128, 128, 6.35, 0.269, 2.33, 0.369}, {256, 128, 11.4, 0.322, 5.73, 0.748},
    {256, 192, 12.6, 0.428, 6.70, 0.858}, {256, 256, 12.2, 0.574, 6.95, 0.944},
};
// (the widened operands of an fp32 output do not fit the registers of the two widest)
constexpr TileCost GROUPED_F32[G_256x192] = {
    {32, 32, 4.21, 0.088, 0.49, 0.145},  {64, 32, 5.86, 0.471, 0.85, 0.165},   {64, 64, 5.85, 0.441, 1.27, 0.220},
    {128, 64, 6.05, 0.440, 2.20, 0.390}, {128, 128, 6.39, 0.451, 3.61, 0.511}, {256, 128, 7.27, 0.831, 7.15, 1.02},
};

static F8GroupedKernel choose_grouped(const F8GroupedArgs& g, bool exact) {
  // the kernel for few rows has a block for every tile that there could be: as many as a grid holds in y
  const F8GroupedKernel first = f8_most_tiles(g, 32) <= 65535 ? G_TOKENS : G_64x32;
  if (const char* e = getenv("P24_F8_TILE")) {
    static const char* const names[G_KERNELS] = {"tokens", "64x32", "64x64", "128x64", "128x128", "256x128", "256x192", "256x256"};
    for (int i = 0; i < G_KERNELS; ++i)
      if (strcmp(e, names[i]) == 0) return exact && i > G_256x128 ? G_256x128 : i < first ? first : (F8GroupedKernel)i;
  }
  const TileCost* costs = exact ? GROUPED_F32 : GROUPED_BF16;
  const double rows = g.groups.rows, experts = g.groups.experts;
  const double live = experts * -expm1(-rows / experts), mean = rows / live;    // experts with rows, theirs on average
  int best = first;
  double least = 0;
  for (int i = first; i < (exact ? G_256x192 : G_KERNELS); ++i) {
    const TileCost& c = costs[i];
    const double us = c.us(live / -expm1(-c.bn / mean) * ((g.a.M + c.bm - 1) / c.bm), g.a.K);
    if (i == first || us < least) {
      least = us;
      best = i;
    }
  }
  return (F8GroupedKernel)best;
}

template <typename OutT>
static p24_status launch_grouped(const F8GroupedArgs& g, hipStream_t st) {
  constexpr bool EXACT = sizeof(OutT) == 4;
  switch (choose_grouped(g, EXACT)) {
    case G_256x256:
      if constexpr (!EXACT) return launch_tile_grouped<256, 256, 2, 4, 8, 1, OutT>(g, st);
    case G_256x192:
      if constexpr (!EXACT) return launch_tile_grouped<256, 192, 4, 2, 4, 1, OutT>(g, st);
    case G_256x128: return launch_tile_grouped<256, 128, 4, 2, 4, 1, OutT>(g, st);
    case G_128x128: return launch_tile_grouped<128, 128, 2, 4, 4, 1, OutT>(g, st);
    case G_128x64: return launch_tile_grouped<128, 64, 2, 2, 4, 1, OutT>(g, st);
    case G_64x64: return launch_tile_grouped<64, 64, 2, 2, 4, 1, OutT>(g, st);
    case G_64x32: return launch_tile_grouped<64, 32, 2, 1, 2, 1, OutT>(g, st);
    default: break;
  }
  if (g.a.K >= 2048 && ((int64_t)g.a.M + 31) / 32 * f8_most_tiles(g, 32) <= 256) return launch_tokens_grouped<16, OutT>(g, st);
  if (g.a.K >= 1024) return launch_tokens_grouped<8, OutT>(g, st);
  return launch_tokens_grouped<4, OutT>(g, st);
}

}  // namespace p24

using namespace p24;

extern "C" P24_API p24_status spmm24_f8_grouped(const void* data, const float* w_scale, int64_t E, int64_t M, int64_t K,
                                                const void* X, int64_t ldx, const float* x_scale, int64_t x_rows,
                                                const int32_t* offsets, const int32_t* tokens, int64_t rows, void* Y,
                                                int32_t y_dtype, int64_t ldy, const float* bias, int32_t act,
                                                void* stream) {
  if (y_dtype != P24_F32 && y_dtype != P24_BF16) return P24_ERR_DTYPE;
  if (!f8_act_known(act)) return P24_ERR_UNSUPPORTED;
  if (E < 1 || M < 0 || K < 0 || rows < 0 || x_rows < 0 || M > INT32_MAX || K > INT32_MAX || rows > INT32_MAX ||
      x_rows > INT32_MAX)
    return P24_ERR_SHAPE;
  if (ldx < K || ldy < M) return P24_ERR_SHAPE;
  if (E > P24_EXPERTS_MAX || K % 64) return P24_ERR_UNSUPPORTED;
  if (M == 0 || rows == 0) return P24_OK;
  if (x_rows == 0 || (!tokens && x_rows != rows)) return P24_ERR_SHAPE;
  if (x_rows == 1) ldx = K;   // a single row has no stride of its own
  if (K == 0 || K >= (1 << 24) || M >= (1 << 24) || rows > 65535 * 32 || (uint64_t)ldx * 512 >= (1ull << 32)) return P24_ERR_UNSUPPORTED;
  if (tokens && (ldx >= (1ll << 32) / x_rows)) return P24_ERR_UNSUPPORTED;
  if (!data || !w_scale || !X || !x_scale || !Y || !offsets) return P24_ERR_NULL;
  const size_t ye = y_dtype == P24_F32 ? 4 : 2;
  if (!aligned(data, 16) || !aligned(X, 16) || ldx % 16 || !aligned(Y, ye) || !aligned(w_scale, 4) || !aligned(x_scale, 4) ||
      !aligned(offsets, 4) || (tokens && !aligned(tokens, 4)) || (bias && !aligned(bias, 4)))
    return P24_ERR_ALIGN;
  F8GroupedArgs g{};
  g.a.W = (const uint8_t*)data;
  g.a.w_scale = w_scale;
  g.a.X = (const uint8_t*)X;
  g.a.x_scale = x_scale;
  g.a.Y = Y;
  g.a.bias = bias;
  g.a.ldx = ldx;
  g.a.ldy = ldy;
  g.a.M = (int)M;
  g.a.N = (int)rows;
  g.a.K = (int)K;
  g.a.act = act;
  // an expert's rows start anywhere: whole lines if every row is
  g.a.stream = aligned(Y, 128) && ldy * (int64_t)ye % 128 == 0 && (uint64_t)ldy * 1024 < (1ull << 32);
  g.groups.offsets = offsets;
  g.groups.tokens = tokens;
  g.groups.experts = (int)E;
  g.groups.rows = (int)rows;
  g.groups.x_rows = (int)x_rows;
  g.w_bytes = (int64_t)prune24_f8_bytes(M, K);
  if (y_dtype == P24_F32) return launch_grouped<float>(g, (hipStream_t)stream);
  return launch_grouped<uint16_t>(g, (hipStream_t)stream);
}
