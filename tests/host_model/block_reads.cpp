// The direct-to-LDS loads of the block-scaled product and of the grouped one, lane by lane on the CPU
// (test infrastructure): how many of them could read past the matrix that they belong to.
#include <algorithm>
#include <cstdint>

#include "../../structured_sparse_gemm_prune24_amd/csrc/p24_f8_tile.hpp"
#include "../../structured_sparse_gemm_prune24_amd/csrc/p24_f8b_tile.hpp"

namespace {

using namespace p24;

// As in reads.cpp: a load is dropped for certain if its vector offset alone lies past the resource and the
// scalar offset does not; any other must be whole and inside.
bool bad(uint64_t vector, uint64_t scalar, uint64_t width, uint64_t bytes, uint64_t end) {
  if (bytes > end || vector + scalar + width > UINT32_MAX) return true;
  if (vector >= bytes) return scalar > bytes;
  return vector + scalar + width > bytes;
}

template <int BM, int BN, int WGM, int WGN, int LW, int NST, int KG>
long block_tile(int64_t M, int64_t N, int64_t K, int64_t ld, int64_t ldxs) {
  using C = F8BTile<BM, BN, WGM, WGN, LW, NST, KG>;
  const F8BSteps steps((int)K);
  const int blocks = (int)((K + 127) / 128), row_blocks = (int)((M + 127) / 128);
  if (steps.count != blocks) return 1;
  if (KG > 1 && steps.count < KG) return 0;          // not launched
  long n_bad = 0;
  // every block of K is one step's, a part of one the first
  for (int b = 0; b < blocks; ++b) {
    int found = 0;
    for (int s = 0; s < steps.count; ++s) found += steps.block(s) == b;
    n_bad += found != 1;
  }
  if (steps.rest) n_bad += steps.block(0) != blocks - 1;
  for (int64_t m0 = 0; m0 < M; m0 += BM)
    for (int64_t n0 = 0; n0 < N; n0 += BN) {
      const int mr = (int)std::min<int64_t>(M - m0, BM), nr = (int)std::min<int64_t>(N - n0, BN);
      const int rb = std::min(row_blocks - (int)(m0 / 128), C::ROW_BLOCKS);
      const uint64_t x_end = (N - 1 - n0) * ld + K, w_end = (M - 1 - m0) * ld + K;
      const uint64_t sx_end = ((blocks - 1) * ldxs + N - n0) * 4, sw_end = (uint64_t)(row_blocks - m0 / 128) * blocks * 4;
      const uint64_t sx_bytes = ((blocks - 1) * ldxs + nr) * 4, sw_bytes = (uint64_t)rb * blocks * 4;
      for (int wave = 0; wave < LW; ++wave)
        for (int lane = 0; lane < 64; ++lane) {
          const F8BReads<LW> x(lane, wave, ld, steps), w(lane, wave, ld, steps);
          for (int kg = 0; kg < KG; ++kg) {
            const int first = steps.count * kg / KG, count = steps.count * (kg + 1) / KG - first;
            for (int it = 0; it < count + NST; ++it) {
              const int s = first + last_of(it, count), b = steps.block(s);
              for (int q = 0; q < C::X_DMA; ++q)
                n_bad += bad(x.vector(q, s == 0), F8BReads<LW>::scalar(b), 16, F8BReads<LW>::bytes(nr, ld, (int)K), x_end);
              for (int q = 0; q < C::W_DMA; ++q)
                n_bad += bad(w.vector(q, s == 0), F8BReads<LW>::scalar(b), 16, F8BReads<LW>::bytes(mr, ld, (int)K), w_end);
              for (int q = 0; q < C::S_DMA; ++q) {
                const int n = F8BScaleReads<C>::number(wave, q);
                n_bad += n < 0 || n >= C::SCALE_LOADS;
                const uint64_t at = F8BScaleReads<C>::vector(lane, n, nr, rb, blocks), on = F8BScaleReads<C>::scalar(n, b, ldxs);
                n_bad += F8BScaleReads<C>::tokens(n) ? bad(at, on, 4, sx_bytes, sx_end) || at >= sx_bytes
                                                     : bad(at, on, 4, sw_bytes, sw_end) || at >= sw_bytes;
              }
            }
          }
        }
    }
  return n_bad;
}

template <int BM, int BN, int WGM, int WGN, int LW>
long grouped_tile(int64_t rows, int64_t x_rows, int64_t K, int64_t ldx) {
  using C = F8Tile<BM, BN, WGM, WGN, LW, 1>;
  const int nk = (int)(f8_steps(K) / 2);
  const uint64_t end = (x_rows - 1) * ldx + K;
  long n_bad = 0;
  for (int64_t n0 = 0; n0 < rows; n0 += BN) {
    const int n_rows = (int)std::min<int64_t>(rows - n0, BN);
    for (int wave = 0; wave < LW; ++wave)
      for (int lane = 0; lane < 64; ++lane)
        for (int q = 0; q < C::X_DMA; ++q) {
          const int r = std::min(F8XReads<C>::row(lane, wave, q), n_rows - 1);
          if (n0 + r >= rows) ++n_bad;                       // its index is read there
          const int chunk = F8XReads<C>::chunk(lane, wave);
          if (chunk != ((lane & 7) ^ (F8XReads<C>::row(lane, wave, q) & 7))) ++n_bad;
          for (int64_t token : {(int64_t)0, std::min<int64_t>(n0 + r, x_rows - 1), x_rows - 1})
            for (int g = 0; g < nk; ++g) {
              const uint64_t v = (uint64_t)token * ldx + chunk * 16 - (g == nk - 1 ? F8XReads<C>::back(chunk, (int)K) : 0);
              n_bad += bad(v, F8XReads<C>::scalar(g), 16, F8XReads<C>::bytes((int)x_rows, ldx, (int)K), end);
            }
        }
  }
  return n_bad;
}

}  // namespace

// The block tiles that gemm_f8_block launches.
extern "C" long block_bad_reads(int tile, int64_t M, int64_t N, int64_t K, int64_t ld, int64_t ldxs) {
  switch (tile) {
    case 0: return block_tile<64, 32, 1, 2, 2, 3, 1>(M, N, K, ld, ldxs);
    case 1: return block_tile<64, 32, 1, 2, 2, 3, 2>(M, N, K, ld, ldxs);
    case 2: return block_tile<64, 64, 1, 4, 4, 3, 1>(M, N, K, ld, ldxs);
    case 3: return block_tile<64, 64, 1, 4, 4, 4, 2>(M, N, K, ld, ldxs);
    case 4: return block_tile<128, 64, 2, 2, 4, 3, 1>(M, N, K, ld, ldxs);
    case 5: return block_tile<128, 64, 2, 2, 4, 3, 2>(M, N, K, ld, ldxs);
    case 6: return block_tile<128, 128, 2, 2, 4, 2, 1>(M, N, K, ld, ldxs);
    case 7: return block_tile<256, 128, 4, 2, 8, 3, 1>(M, N, K, ld, ldxs);
    case 8: return block_tile<256, 256, 2, 4, 8, 2, 1>(M, N, K, ld, ldxs);
  }
  return -1;
}

// The tiles that spmm24_f8_grouped launches, one expert of `rows` rows.
extern "C" long grouped_bad_reads(int tile, int64_t rows, int64_t x_rows, int64_t K, int64_t ldx) {
  switch (tile) {
    case 0: return grouped_tile<64, 32, 2, 1, 2>(rows, x_rows, K, ldx);
    case 1: return grouped_tile<64, 64, 2, 2, 4>(rows, x_rows, K, ldx);
    case 2: return grouped_tile<128, 64, 2, 2, 4>(rows, x_rows, K, ldx);
    case 3: return grouped_tile<128, 128, 2, 4, 4>(rows, x_rows, K, ldx);
    case 4: return grouped_tile<256, 128, 4, 2, 4>(rows, x_rows, K, ldx);
    case 5: return grouped_tile<256, 192, 4, 2, 4>(rows, x_rows, K, ldx);
    case 6: return grouped_tile<256, 256, 2, 4, 8>(rows, x_rows, K, ldx);
  }
  return -1;
}
