// The block-scaled 8-bit product's tiles and the places that their direct-to-LDS loads read (host and
// device).
#pragma once

#include "p24_reads.hpp"

namespace p24 {

// BM rows x BN tokens per block on WGM x WGN waves, of which the first LW load; K by 128 values (one block of
// scales) a step, NST steps in LDS.  With KG > 1 there are KG such groups of waves, each with its own stages and
// its own part of K.
template <int BM, int BN, int WGM, int WGN, int LW_, int NST, int KG>
struct F8BTile {
  static constexpr int WAVES = WGM * WGN, LW = LW_;        // of a group
  static constexpr int WTM = BM / WGM, WTN = BN / WGN;     // wave tile
  static constexpr int TM = WTM / 16, TN = WTN / 16;       // its 16 x 16 tiles
  static constexpr int PAIRS = TM / 2;                     // rows go by 32
  // a step's scales: 64 tokens a load, then one of the row blocks
  static constexpr int TOKEN_LOADS = (BN + 63) / 64, SCALE_LOADS = TOKEN_LOADS + 1;
  static constexpr int ROW_BLOCKS = BM >= 128 ? BM / 128 : 1;
  // stage: [X: BN rows of 128 B | W: BM rows of 128 B | scales: 256 B a load]
  static constexpr int X_BYTES = BN * 128, W_BYTES = BM * 128;
  static constexpr int STAGE = X_BYTES + W_BYTES + (SCALE_LOADS * 256 + 1023) / 1024 * 1024;
  // loads per loading wave and step (where the scales' do not come out even, the last one is repeated)
  static constexpr int X_DMA = BN / 8 / LW, W_DMA = BM / 8 / LW, S_DMA = (SCALE_LOADS + LW - 1) / LW;
  static constexpr int DMA = X_DMA + W_DMA + S_DMA;
  // epilogue: each wave turns 16 tokens at a time through LDS
  static constexpr int PITCH = WTM + 4;                    // floats per token
  static_assert(LW % 2 == 0 && LW <= WAVES && BN % (8 * LW) == 0 && BM % (8 * LW) == 0, "even loads");
  static_assert(PAIRS >= 2 && TM % 2 == 0 && TN >= 1, "rows go by pairs of tiles, two pairs at least");
  static_assert(WTM <= 128 && 128 % WTM == 0, "a wave's rows lie in one block of scales");
  static_assert(KG * NST * STAGE <= 160 * 1024 && WAVES * 16 * PITCH * 4 <= NST * STAGE, "LDS");
  static_assert(NST * DMA < 64, "vmcnt range");
};

// Where K's steps lie.  A part of a block goes first: its missing chunks are cleared in LDS before the first use.
struct F8BSteps {
  int count, rest;      // steps; values of the part (0: none)
  P24_HD explicit F8BSteps(int K) : count((K + 127) / 128), rest(K % 128) {}
  P24_HD int block(int step) const {          // steps past the end repeat the last
    const int s = last_of(step, count);
    return rest == 0 ? s : s == 0 ? count - 1 : s - 1;
  }
};

// X or W: load q of loading wave w brings 8 rows x 128 B of a step, rows 8 (q LW + w) on.
// LDS slot of (row n, 16 B chunk c) = (n ^ ((n >> 3) & 1)) * 8 + (c ^ (n & 7)): sixteen
// consecutive rows at one chunk fall on sixteen bank groups.  LW is even: every load of
// a wave keeps its rows' parity.  Rows past the tile's `rows` lie past the resource.
// In a part of a block the chunks past K read chunk 0.
template <int LW>
struct F8BReads {
  uint32_t voff, back, jump;
  static P24_HD int row(int lane, int wave, int q) { return 8 * (q * LW + wave) + ((lane >> 3) ^ (wave & 1)); }
  static P24_HD int chunk(int lane, int wave) { return (lane & 7) ^ (row(lane, wave, 0) & 7); }
  P24_HD F8BReads(int lane, int wave, int64_t ld, const F8BSteps& steps) {
    const int c = chunk(lane, wave);
    voff = (uint32_t)(row(lane, wave, 0) * ld + 16 * c);
    back = steps.rest && 16 * c >= steps.rest ? (uint32_t)(16 * c) : 0;
    jump = (uint32_t)(8 * LW * ld);
  }
  static P24_HD uint32_t bytes(int rows, int64_t ld, int K) { return (uint32_t)((rows - 1) * ld + K); }
  P24_HD uint32_t vector(int q, bool part) const { return voff + q * jump - (part ? back : 0); }
  static P24_HD uint32_t scalar(int block) { return (uint32_t)block * 128; }
};

// A step's scales: load q of loading wave w is number q LW + w, 4 B a lane; lanes past the tile repeat its last
// token or row block.
template <class C>
struct F8BScaleReads {
  static P24_HD int number(int wave, int q) { return last_of(q * C::LW + wave, C::SCALE_LOADS); }
  static P24_HD bool tokens(int number) { return number < C::TOKEN_LOADS; }
  static P24_HD uint32_t vector(int lane, int number, int n_tokens, int row_blocks, int blocks) {
    return 4 * (uint32_t)(tokens(number) ? last_of(64 * number + lane, n_tokens) : last_of(lane, row_blocks) * blocks);
  }
  static P24_HD uint32_t scalar(int number, int block, int64_t ldxs) {
    return (uint32_t)block * (tokens(number) ? (uint32_t)ldxs * 4 : 4);
  }
};

}  // namespace p24
