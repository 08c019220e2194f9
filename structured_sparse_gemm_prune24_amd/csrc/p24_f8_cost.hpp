// How long a kernel of the 8-bit products takes, for the choice between them (host).
#pragma once

#include <cmath>

namespace p24 {

// A tile of bm rows x bn tokens over K = 128 steps.  One block alone takes alone + alone_step * steps us: launch,
// first loads and epilogue, and a step's waits.  With many blocks a round of 256 takes many + many_step * steps: the CUs'
// throughput, several blocks to a CU where they fit.  The time is the larger of the two, joined smoothly.  The four numbers
// of a kernel are a least-squares fit (of the logarithm) to its times over shapes drawn at random; a
// forecast is 10-15 % off, up to 30 % at a shape (the rules' comments have measured ones): it is for the order of the
// kernels.
struct TileCost {
  int bm, bn;
  double alone, alone_step, many, many_step;
  double us(double blocks, int64_t K) const {
    const double steps = (double)((K + 127) / 128);
    const double a = alone + alone_step * steps, m = blocks / 256 * (many + many_step * steps);
    return std::sqrt(std::sqrt(a * a * a * a + m * m * m * m));
  }
};

}  // namespace p24
