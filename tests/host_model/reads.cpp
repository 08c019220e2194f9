// The direct-to-LDS loads of the GEMM kernels, lane by lane on the CPU (test infrastructure): how
// many of them could read past the matrix that they belong to.
#include <algorithm>
#include <cstdint>

#include "../../structured_sparse_gemm_prune24_amd/csrc/p24_f8_tile.hpp"

namespace {

using namespace p24;

// A load of `width` bytes at vector + scalar through a resource of `bytes`, over memory that ends at
// `end`.  It is dropped for certain if the vector offset alone lies past the resource and the scalar
// offset does not (size minus scalar offset would wrap); any other must be whole and inside.
bool bad(uint64_t vector, uint64_t scalar, uint64_t width, uint64_t bytes, uint64_t end) {
  if (bytes > end || vector + scalar + width > UINT32_MAX) return true;
  if (vector >= bytes) return scalar > bytes;
  return vector + scalar + width > bytes;
}

template <int BM, int BN, int WGM, int WGN, int LW, int KG>
long f8_tile(int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldr) {
  using C = F8Tile<BM, BN, WGM, WGN, LW, KG>;
  const int64_t steps = f8_steps(K), nk = steps / 2;
  long n_bad = 0;
  for (int64_t m0 = 0; m0 < M; m0 += BM)
    for (int64_t n0 = 0; n0 < N; n0 += BN) {
      const int rows = (int)std::min<int64_t>(N - n0, BN);
      const uint64_t x_end = (N - 1 - n0) * ldx + K, r_end = ((N - 1 - n0) * ldr + M - m0) * 2;
      const uint64_t w_end = (f8_groups(M) - m0 / 128) * steps * F8_PIECE;
      const F8WReads<C> w((int)m0, (int)M, (int)K);
      for (int wave = 0; wave < LW; ++wave)
        for (int lane = 0; lane < 64; ++lane) {
          const F8XReads<C> x(lane, wave, ldx, (int)K);
          const F8RReads<C> res(lane, wave, ldr);
          for (int64_t g = 0; g < nk; ++g) {
            for (int q = 0; q < C::X_DMA; ++q)
              n_bad += bad(x.vector(x.rows(q), g == nk - 1), x.scalar((int)g), 16, x.bytes(rows, ldx, (int)K), x_end);
            for (int j = 0; j < C::A_DMA; ++j)
              n_bad += bad(w.vector(lane, j, wave), w.scalar(j, wave) + g * 2 * F8_PIECE, 16, w.bytes(), w_end);
          }
          if (M % 8 == 0 && ldr % 8 == 0)
            for (int q = 0; q < C::RDMA; ++q)
              for (int r0 = 0; r0 < C::GWAVES; r0 += C::RPS) {
                const int l = q * LW + wave, r = r0 + l / C::RL;
                if (r < C::GWAVES)
                  n_bad += bad(res.vector(res.uniform(l, r, WGN)), 0, 16, res.bytes(rows, ldr, (int)(M - m0)), r_end);
              }
        }
    }
  return n_bad;
}

}  // namespace

// The bf16 products' loads for any tile: BM rows, BN columns, LW loading waves, whole row groups or a
// part of one, sparse (asteps 2) or dense (4).
extern "C" long bf16_bad_reads(int BM, int BN, int LW, int asteps, int64_t M, int64_t N, int64_t K, int64_t ldx) {
  const int64_t S = asteps == 2 ? K / 32 : K / 16, T = K / 64;
  const int RB = BM / 32, MG = RB % 4 ? RB / 4 + 1 : RB / 4;
  const int nrb = (int)((M + 31) / 32), ngroups = (int)((M + 127) / 128);
  long n_bad = 0;
  for (int64_t m0 = 0; m0 < M; m0 += BM) {
    const int rb0 = (int)(m0 / 32), rbs = std::min(nrb - rb0, RB), groups = std::min(ngroups - rb0 / 4, MG);
    for (int lane = 0; lane < 64; ++lane)
      for (int64_t g = 0; g < K / 64; ++g) {
        for (int q = 0; q < RB * asteps; ++q)
          n_bad += bad(lane * 16, g * asteps * 1024 + a_scalar(q, asteps, S, rbs), 16, rbs * S * 1024, (nrb - rb0) * S * 1024);
        for (int w = 0; asteps == 2 && w < MG; ++w)
          n_bad += bad(lane * 16, g * 1024 + meta_scalar(w, T, groups), 16, groups * T * 1024, (ngroups - rb0 / 4) * T * 1024);
      }
  }
  for (int64_t n0 = 0; n0 < N; n0 += BN) {
    const int64_t rows = std::min<int64_t>(N - n0, BN), end = (N - n0) * ldx * 2;
    for (int lane = 0; lane < 64; ++lane)
      for (int64_t g = 0; g < K / 64; ++g)
        for (int q = 0; q < BN / 8; ++q)
          n_bad += bad(xt_vector(lane, q % LW, ldx) + xt_rows(q / LW * LW, ldx), g * 128, 16, rows * ldx * 2, end);
  }
  return n_bad;
}

// The block tiles that spmm24_f8 launches, by place in its order.
extern "C" long f8_bad_reads(int tile, int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldr) {
  switch (tile) {
    case 0: return f8_tile<64, 32, 2, 1, 2, 1>(M, N, K, ldx, ldr);
    case 1: return f8_tile<64, 32, 2, 1, 2, 4>(M, N, K, ldx, ldr);
    case 2: return f8_tile<64, 64, 2, 2, 4, 1>(M, N, K, ldx, ldr);
    case 3: return f8_tile<64, 64, 2, 2, 4, 2>(M, N, K, ldx, ldr);
    case 4: return f8_tile<64, 64, 1, 2, 2, 4>(M, N, K, ldx, ldr);
    case 5: return f8_tile<128, 64, 2, 2, 4, 1>(M, N, K, ldx, ldr);
    case 6: return f8_tile<128, 64, 2, 2, 4, 2>(M, N, K, ldx, ldr);
    case 7: return f8_tile<128, 128, 2, 4, 4, 1>(M, N, K, ldx, ldr);
    case 8: return f8_tile<256, 128, 4, 2, 4, 1>(M, N, K, ldx, ldr);
    case 9: return f8_tile<256, 192, 4, 2, 4, 1>(M, N, K, ldx, ldr);
    case 10: return f8_tile<256, 256, 2, 4, 4, 1>(M, N, K, ldx, ldr);
  }
  return -1;
}
