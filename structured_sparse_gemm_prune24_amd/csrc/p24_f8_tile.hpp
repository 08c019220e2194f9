// The 8-bit product's block tiles and the places that their direct-to-LDS loads
// read (host and device).
#pragma once

#include "p24_reads.hpp"

namespace p24 {

// The layout of compressed 8-bit weights (include/prune24_f8.h).
constexpr int F8_PIECE = 5120;                // one row group's 64-k block: 4 x 1 KiB values, 4 x 256 B positions
P24_HD int64_t f8_groups(int64_t M) { return (M + 127) / 128; }
P24_HD int64_t f8_steps(int64_t K) { return 2 * ((K + 127) / 128); }

// BM rows x BN tokens per block on WGM x WGN waves; K goes by 128 values (two
// 64-k blocks) a step.  With KG > 1 there are KG such groups of waves, each with
// its own stages and its own part of K.
template <int BM, int BN, int WGM, int WGN, int LW_, int KG>
struct F8Tile {
  static constexpr int GWAVES = WGM * WGN;                 // waves of a group
  static constexpr int WTM = BM / WGM, WTN = BN / WGN;     // wave tile
  static constexpr int TM = WTM / 32, TN = WTN / 32;       // its 32 x 32 tiles
  static constexpr int LW = LW_;                           // waves of a group that load
  // stage: [X: BN rows of 128 B | per row group: two 64-k blocks of (row blocks' values, 1 KiB of positions)],
  // with half a row group [.. | two row blocks' values of either 64-k block | 512 B of positions of each]
  static constexpr int GROUPS = BM >= 128 ? BM / 128 : 1;
  static constexpr int RBG = BM >= 128 ? 4 : BM / 32;      // row blocks used of a group
  static constexpr int UNITS = RBG == 4 ? 10 : 2 * RBG + 1;   // 1 KiB loads of a group's step
  static constexpr int BLOCK = RBG == 4 ? 5120 : RBG * 1024;  // from one 64-k block's values to the next's
  static constexpr int P_FIRST = RBG == 4 ? 4096 : 2 * BLOCK, P_NEXT = RBG == 4 ? BLOCK : 512;   // the same of positions
  static constexpr int X_BYTES = BN * 128, A_BYTES = GROUPS * UNITS * 1024;
  static constexpr int STAGE = X_BYTES + A_BYTES;
  static constexpr int NSTAGE = 3 * KG * STAGE <= 160 * 1024 ? 3 : 2;
  static constexpr int X_DMA = BN / 8 / LW;                // 1 KiB loads per loading wave and step
  static constexpr int A_LOADS = A_BYTES / 1024;
  // A remainder of one load is left to one wave; of two, the other two waves repeat
  // a load, which is cheaper than uneven counts (4096 x 2304 x 768 in 128 x 128: 13.9 us, 14.9).
  static constexpr int A_DMA = (A_LOADS + LW - 1) / LW;
  static constexpr int A_LAST = A_LOADS % LW == 1 ? 1 : 0;   // waves that issue the last one (0: all)
  static constexpr int DMA = X_DMA + A_DMA;
  static_assert(BM % (32 * WGM) == 0 && BN % (32 * WGN) == 0, "whole 32 x 32 tiles per wave");
  static_assert((BN / 8) % LW == 0 && LW % 2 == 0 && LW <= GWAVES, "even X loads");
  static_assert(BM % 128 == 0 || BM == 64, "whole row groups, or half of one");
  static_assert(NSTAGE * KG * STAGE <= 160 * 1024, "LDS");
  static_assert(NSTAGE * DMA < 64, "vmcnt range");
  // epilogue by slices (fp32 outputs, split K): each wave turns one 32-token slice at a time through LDS
  static constexpr int PITCH = WTM + 4;                    // floats per token
  static_assert(GWAVES * 32 * PITCH * 4 <= NSTAGE * STAGE, "the slices fit the stages' LDS");
  // epilogue in place (bf16 outputs): each wave's output tile as bf16, RPS of them in a stage
  static constexpr int REGION = WTM * WTN * 2, RL = REGION / 1024;   // bytes, and 1 KiB loads of its residual
  static constexpr int RPS = STAGE / REGION < GWAVES ? STAGE / REGION : GWAVES;
  static constexpr int RDMA = RPS * RL / LW;               // residual loads per loading wave and stage
  static constexpr int CH = WTM / 8;                       // 16 B chunks per token of a region
  static constexpr int X_SCALES = BN < 64 ? 64 : BN;
  static constexpr int SCALES = (2 * BM + X_SCALES) * 4;   // weight scales, bias, token scales
  static_assert(RPS >= 1 && (RPS * RL) % LW == 0 && RDMA <= DMA, "residual loads take the place of a step's loads");
  static_assert((GWAVES + RPS - 1) / RPS <= NSTAGE, "the regions fit the stages");
};

// X: load q of loading wave w brings 8 tokens x 128 B of a step, tokens 8 (q LW + w) on.
// LDS slot of (token n, 16 B chunk c) = (n ^ ((n >> 3) & 1)) * 8 + (c ^ (n & 7)): sixteen
// consecutive tokens at one chunk fall on sixteen bank groups.  LW is even: every load of
// a wave keeps its tokens' parity.  Tokens past the tile's `rows` lie past the resource.
// In the last step of an odd count of 64-k blocks chunks 4..7 repeat chunks
// 0..3: they meet the weights' zero padding.
template <class C>
struct F8XReads {
  uint32_t voff, tail, jump;
  P24_HD F8XReads(int lane, int wave, int64_t ldx, int K) {
    const int row = 8 * wave + ((lane >> 3) ^ (wave & 1)), chunk = (lane & 7) ^ (row & 7);
    voff = (uint32_t)(row * ldx + 16 * chunk);
    tail = voff - ((K & 64) && chunk >= 4 ? 64 : 0);
    jump = (uint32_t)(8 * C::LW * ldx);
  }
  static P24_HD uint32_t bytes(int rows, int64_t ldx, int K) { return (uint32_t)((rows - 1) * ldx + K); }
  P24_HD uint32_t rows(int q) const { return q * jump; }     // from load 0's tokens to load q's
  P24_HD uint32_t vector(uint32_t rows, bool last) const { return (last ? tail : voff) + rows; }
  static P24_HD uint32_t scalar(int step) { return (uint32_t)step * 128; }
};

// Weights: load j of loading wave w is unit u of a row group of the tile: the
// pieces of its two 64-k blocks in order, or of half a group two row blocks' values of
// each, then the positions, 512 B of either.
template <class C>
struct F8WReads {
  int groups;             // of the tile's row groups, those inside the weight
  uint32_t steps;         // f8_steps(K)
  uint32_t first_rb;      // half a group: its first row block
  P24_HD F8WReads(int m0, int M, int K) {
    groups = (int)f8_groups(M) - m0 / 128;
    groups = groups < C::GROUPS ? groups : C::GROUPS;
    steps = (uint32_t)f8_steps(K);
    first_rb = (uint32_t)(m0 / 32) % 4;
  }
  P24_HD uint32_t bytes() const { return (uint32_t)groups * steps * F8_PIECE; }
  static P24_HD int unit(int j, int wave) { return last_of(j * C::LW + wave, C::A_LOADS); }
  static P24_HD bool positions(int j, int wave) { return C::RBG < 4 && (j * C::LW + wave) % C::UNITS == 2 * C::RBG; }
  static P24_HD uint32_t vector(int lane, int j, int wave) {
    return positions(j, wave) ? (uint32_t)(lane / 32) * F8_PIECE + (uint32_t)(lane % 32) * 16 : (uint32_t)lane * 16;
  }
  // of the first step; each further one is 2 F8_PIECE on
  P24_HD uint32_t scalar(int j, int wave) const {
    const int q = unit(j, wave), u = q % C::UNITS;
    if (C::RBG == 4) return (uint32_t)last_of(q / C::UNITS, groups) * steps * F8_PIECE + u * 1024;
    return u == 2 * C::RBG ? 4096 + first_rb * 256 : (u / C::RBG) * F8_PIECE + (first_rb + u % C::RBG) * 1024;
  }
};

// The residual (bf16, rows of whole aligned 16 B chunks): load l of a stage, by wave l % LW, is
// tokens (l % RL) * 64 / CH on of region r, wave r's output tile; chunk c of a region's token t
// goes to place c ^ (t % CH).  All of a wave's loads have the same t % CH in a lane: one
// offset of its own and a uniform rest.
template <class C>
struct F8RReads {
  static_assert(C::LW * (64 / C::CH) % C::CH == 0 && (C::RL % C::LW == 0 || C::LW % C::RL == 0), "one t % CH a lane");
  uint32_t voff, row_bytes;
  int wave;
  P24_HD F8RReads(int lane, int wave_, int64_t ldr) : row_bytes((uint32_t)ldr * 2), wave(wave_) {
    const int t = (wave % C::RL) * (64 / C::CH) + lane / C::CH, chunk = (lane % C::CH) ^ (t % C::CH);
    voff = (uint32_t)t * row_bytes + 16 * chunk;
  }
  static P24_HD uint32_t bytes(int rows, int64_t ldr, int features) { return (uint32_t)((rows - 1) * ldr + features) * 2; }
  P24_HD uint32_t uniform(int l, int region, int WGN) const {
    const int t = (region % WGN) * C::WTN + (l % C::RL - wave % C::RL) * (64 / C::CH);
    return (uint32_t)t * row_bytes + (uint32_t)((region / WGN) * C::WTM) * 2;
  }
  P24_HD uint32_t vector(uint32_t uniform) const { return voff + uniform; }
};

}  // namespace p24
