// Which tile a block takes (host and device).
#pragma once

#include "p24_reads.hpp"

namespace p24 {

// XCD-aware block order.  Workgroups are handed to the 8 XCDs round-robin, so
// block b runs on XCD b % 8.  Renumbering so that each XCD receives one
// contiguous range of logical tiles keeps neighbouring tiles (which share rows
// of W and columns of X) in the same XCD's L2.
P24_HD uint32_t xcd_remap(uint32_t b, uint32_t nblocks) {
  constexpr uint32_t NXCD = 8;
  const uint32_t per = nblocks / NXCD;          // full rounds
  const uint32_t full = per * NXCD;
  if (b >= full) return b;                      // the ragged last round keeps its ids
  return (b % NXCD) * per + (b / NXCD);
}

// Row block and token tile of block b of nbm x nbn: groups of eight row blocks.
P24_HD void f8_place(uint32_t b, uint32_t nbm, uint32_t nbn, uint32_t& bm, uint32_t& bn) {
  constexpr uint32_t GROUP = 8;
  const uint32_t group_size = GROUP * nbn;
  const uint32_t first_m = (b / group_size) * GROUP;
  const uint32_t gsz = nbm - first_m < GROUP ? nbm - first_m : GROUP;
  bm = first_m + (b % group_size) % gsz;
  bn = (b % group_size) / gsz;
}

}  // namespace p24
