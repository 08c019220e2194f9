// The block-scaled 8-bit product's tiles and the places that their direct-to-LDS loads read (host and
// device).
#pragma once

#include "p24_reads.hpp"

namespace p24 {

// BM rows x BN tokens per block on WGM x WGN waves, K by 128 values (one block of scales) a step, NST
// steps in LDS.
template <int BM, int BN, int WGM, int WGN, int NST>
struct F8BTile {
  static constexpr int WAVES = WGM * WGN;
  static constexpr int WTM = BM / WGM, WTN = BN / WGN;     // wave tile
  static constexpr int TM = WTM / 16, TN = WTN / 16;       // its 16 x 16 tiles
  static constexpr int PAIRS = TM / 2;                     // rows go by 32
  // stage: [X: BN rows of 128 B | W: BM rows of 128 B | scales: 256 B per wave]
  static constexpr int X_BYTES = BN * 128, W_BYTES = BM * 128, SCALES = WAVES * 256;
  static constexpr int STAGE = X_BYTES + W_BYTES + SCALES;
  static constexpr int X_DMA = BN / 8 / WAVES, W_DMA = BM / 8 / WAVES, DMA = X_DMA + W_DMA + 1;   // loads per wave and step
  // a step's scales: wave w < TOKEN_LOADS loads those of tokens 64 w on, the others those of the row blocks
  static constexpr int TOKEN_LOADS = (BN + 63) / 64;
  static constexpr int ROW_BLOCKS = BM >= 128 ? BM / 128 : 1;
  // epilogue: each wave turns 16 tokens at a time through LDS
  static constexpr int PITCH = WTM + 4;                    // floats per token
  static_assert(WAVES % 2 == 0 && TOKEN_LOADS < WAVES, "a wave is left for the row blocks' scales");
  static_assert(BN % (8 * WAVES) == 0 && BM % (8 * WAVES) == 0, "even loads");
  static_assert(PAIRS >= 2 && TM % 2 == 0 && TN >= 1, "rows go by pairs of tiles, two pairs at least");
  static_assert(WTM <= 128 && 128 % WTM == 0, "a wave's rows lie in one block of scales");
  static_assert(NST * STAGE <= 160 * 1024 && WAVES * 16 * PITCH * 4 <= NST * STAGE, "LDS");
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

// X or W: load q of wave w brings 8 rows x 128 B of a step, rows 8 (q WAVES + w) on.
// LDS slot of (row n, 16 B chunk c) = (n ^ ((n >> 3) & 1)) * 8 + (c ^ (n & 7)): sixteen
// consecutive rows at one chunk fall on sixteen bank groups.  WAVES is even: every load of
// a wave keeps its rows' parity.  Rows past the tile's `rows` lie past the resource.
// In a part of a block the chunks past K read chunk 0.
template <int WAVES>
struct F8BReads {
  uint32_t voff, back, jump;
  static P24_HD int row(int lane, int wave, int q) { return 8 * (q * WAVES + wave) + ((lane >> 3) ^ (wave & 1)); }
  static P24_HD int chunk(int lane, int wave) { return (lane & 7) ^ (row(lane, wave, 0) & 7); }
  P24_HD F8BReads(int lane, int wave, int64_t ld, const F8BSteps& steps) {
    const int c = chunk(lane, wave);
    voff = (uint32_t)(row(lane, wave, 0) * ld + 16 * c);
    back = steps.rest && 16 * c >= steps.rest ? (uint32_t)(16 * c) : 0;
    jump = (uint32_t)(8 * WAVES * ld);
  }
  static P24_HD uint32_t bytes(int rows, int64_t ld, int K) { return (uint32_t)((rows - 1) * ld + K); }
  P24_HD uint32_t vector(int q, bool part) const { return voff + q * jump - (part ? back : 0); }
  static P24_HD uint32_t scalar(int block) { return (uint32_t)block * 128; }
};

// A step's scales, 4 B a lane; lanes past the tile repeat its last token or row block.
template <class C>
struct F8BScaleReads {
  uint32_t voff, step;      // of block 0; from block to block
  P24_HD F8BScaleReads(int lane, int wave, int tokens, int row_blocks, int64_t ldxs, int blocks) {
    if (wave < C::TOKEN_LOADS) {
      voff = (uint32_t)last_of(64 * wave + lane, tokens) * 4;
      step = (uint32_t)ldxs * 4;
    } else {
      voff = (uint32_t)(last_of(lane, row_blocks) * blocks) * 4;
      step = 4;
    }
  }
  P24_HD uint32_t scalar(int block) const { return (uint32_t)block * step; }
};

}  // namespace p24
