// spmm24_f8: which kernel of p24_f8_gemm.hpp runs a product, its launch and the entry point.
#include <cstdlib>
#include <cstring>

#include "p24_api_internal.hpp"
#include "p24_f8_gemm.hpp"

namespace p24 {

template <int W, typename OutT>
static p24_status launch_tokens(const F8Args& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.M + 31) / 32), (unsigned)((a.N + 31) / 32));
  hipLaunchKernelGGL((k_f8_tokens<W, OutT>), grid, dim3(W * 64), 0, st, a);
  return launch_status();
}

template <int BM, int BN, int WGM, int WGN, int LW, int KG, typename OutT>
static p24_status launch_tile(F8Args a, hipStream_t st) {
  a.nbm = (a.M + BM - 1) / BM;
  a.nbn = (a.N + BN - 1) / BN;
  if ((int64_t)a.nbm * a.nbn * (WGM * WGN * KG * 64) > UINT32_MAX) return P24_ERR_UNSUPPORTED;   // a grid's threads
  hipLaunchKernelGGL((k_gemm_f8<BM, BN, WGM, WGN, LW, KG, OutT>), dim3((unsigned)(a.nbm * a.nbn)),
                     dim3(WGM * WGN * KG * 64), 0, st, a);
  return launch_status();
}

// Which kernel.  A block tile's loads per multiply shrink with its size, but a
// launch needs enough blocks for 256 CUs: the largest tile that still gives about
// 144 of them wins.  Between 256 x 256 and 256 x 192 the rounds of blocks decide,
// full ones included (2048 x 1024 with 6144 tokens, 256 blocks of 256 x 192 13.4,
// 192 of 256 x 256 14.5; 4096 x 2048 with 6144 tokens, 512 blocks 33.5, 384 36.5).
// Measured, us, M x K with N tokens:
//   8192 x 8192, 8192   256x256 264, 256x128 358, 128x128 421
//   2304 x 768, 4096    256x192 11.8 (198 blocks), 256x256 13.2 (144), 128x128 14.3
//   2880 x 7232, 6098   256x192 91.7 (384 blocks), 256x256 109.7 (288)
//   1288 x 4416, 3231   256x128 24.4 (156 blocks), 256x192 29.3 (102), 128x128 31.8
//   768 x 768, 4096     128x128 6.3 (192 blocks), 256x128 7.7, 64x64 7.1
//   4096 x 4096, 512    128x64 11.4 (256 blocks), 128x128 14.3, 64x64 13.4
//   4096 x 4096, 256    64x64 9.0 (256 blocks), 128x64 10.6
// Where one round of blocks covers the CUs at most, a block has its CU to itself:
// two or four groups of waves then split K inside it, which keeps more loads in
// flight (64x64 in the last line 10.9 -> 9.2; 64x32 on 4096 x 4096 with 128 tokens
// 9.8 -> 7.7).  A group needs a few steps of its own to be worth its part in the
// sum: K >= 1024.
// A tile's steps wait for memory and for each other; the kernel without shared
// operands does neither, but reads the tokens once per 32 rows.  It wins where
// that is little: at most 128 tiles of 32 x 32 (4096 x 4096, one token 4.9, 64x32
// 6.2; 1024 x 8192, one token 5.7, 8.5), at most 640 with a short K (4096 x 512, 128
// tokens 3.8, 4.0; 1000 x 1024, 400 tokens 4.8, 5.0; but 8192 x 1024, 128 tokens 7.6,
// 64x64 4.9), and with few tokens (16384 x 4096, one token 8.8, 64x64 9.6; but 24
// tokens 11.5, 64x32 10.2).
// Over 260 shapes drawn at random the choice was 1.6 % behind the fastest of the
// eight kernels (geometric mean).
enum class F8Kernel { TOKENS, T64x32, T64x64, T128x64, T128x128, T256x128, T256x192, T256x256 };

static int64_t f8_blocks(const F8Args& a, int bm, int bn) {
  return ((a.M + (int64_t)bm - 1) / bm) * ((a.N + (int64_t)bn - 1) / bn);
}

static F8Kernel choose_f8(const F8Args& a, bool exact) {
  if (const char* e = getenv("P24_F8_TILE")) {
    auto is = [&](const char* name) { return strcmp(e, name) == 0; };
    if (is("tokens")) return F8Kernel::TOKENS;
    if (is("64x32")) return F8Kernel::T64x32;
    if (is("64x64")) return F8Kernel::T64x64;
    if (is("128x64")) return F8Kernel::T128x64;
    if (is("128x128")) return F8Kernel::T128x128;
    if (is("256x128") || (exact && (is("256x192") || is("256x256")))) return F8Kernel::T256x128;
    if (is("256x192")) return F8Kernel::T256x192;
    if (is("256x256")) return F8Kernel::T256x256;
  }
  const int64_t tiles = f8_blocks(a, 32, 32);
  if (a.N <= 8 || tiles <= 128 || (tiles <= 640 && a.K <= 1408)) return F8Kernel::TOKENS;
  const int64_t n128 = f8_blocks(a, 256, 128);
  // the widened operands of an fp32 output do not fit the registers of the two widest
  if (!exact) {
    const int64_t n256 = f8_blocks(a, 256, 256), n192 = f8_blocks(a, 256, 192);
    const int64_t t256 = (n256 + 255) / 256 * 4, t192 = (n192 + 255) / 256 * 3;
    if (n192 >= 160 && t192 < t256) return F8Kernel::T256x192;
    if (n256 >= 144) return F8Kernel::T256x256;
  }
  if ((n128 >= 144 && n128 <= 256) || n128 >= 768) return F8Kernel::T256x128;
  if (f8_blocks(a, 128, 128) >= 144) return F8Kernel::T128x128;
  if (f8_blocks(a, 128, 64) >= 144) return F8Kernel::T128x64;
  if (f8_blocks(a, 64, 64) >= 128) return F8Kernel::T64x64;
  return F8Kernel::T64x32;
}

template <typename OutT>
static p24_status launch_f8(const F8Args& a, hipStream_t st) {
  constexpr bool EXACT = sizeof(OutT) == 4;
  const bool long_k = a.K >= 1024;
  switch (choose_f8(a, EXACT)) {
    case F8Kernel::T256x256:
      if constexpr (!EXACT) return launch_tile<256, 256, 2, 4, 4, 1, OutT>(a, st);
    case F8Kernel::T256x192:
      if constexpr (!EXACT) return launch_tile<256, 192, 4, 2, 4, 1, OutT>(a, st);
    case F8Kernel::T256x128: return launch_tile<256, 128, 4, 2, 4, 1, OutT>(a, st);
    case F8Kernel::T128x128: return launch_tile<128, 128, 2, 4, 4, 1, OutT>(a, st);
    case F8Kernel::T128x64:
      if (long_k && f8_blocks(a, 128, 64) <= 256) return launch_tile<128, 64, 2, 2, 4, 2, OutT>(a, st);
      return launch_tile<128, 64, 2, 2, 4, 1, OutT>(a, st);
    case F8Kernel::T64x64:
      if (long_k && f8_blocks(a, 64, 64) <= 256) {
        // widening is the larger part of an fp32 output's work: taller wave tiles
        // widen each operand for more multiplies (1000 x 4032 with 517 tokens 13.3 -> 11.9)
        if constexpr (EXACT) return launch_tile<64, 64, 1, 2, 2, 4, OutT>(a, st);
        else return launch_tile<64, 64, 2, 2, 4, 2, OutT>(a, st);
      }
      return launch_tile<64, 64, 2, 2, 4, 1, OutT>(a, st);
    case F8Kernel::T64x32:
      if (long_k) return launch_tile<64, 32, 2, 1, 2, 4, OutT>(a, st);
      return launch_tile<64, 32, 2, 1, 2, 1, OutT>(a, st);
    case F8Kernel::TOKENS: break;
  }
  // waves that split K: 4.9, 5.1 and 6.2 us with 16, 8 and 4 (4096 x 4096, one token);
  // 10.5, 8.8 and 9.4 (16384 x 4096); 4.8, 3.5 and 3.4 (500 x 256, 700 tokens)
  if (a.K >= 2048 && f8_blocks(a, 32, 32) <= 256) return launch_tokens<16, OutT>(a, st);
  if (a.K >= 1024) return launch_tokens<8, OutT>(a, st);
  return launch_tokens<4, OutT>(a, st);
}

}  // namespace p24

using namespace p24;

extern "C" P24_API p24_status spmm24_f8(const void* data, const float* w_scale, int64_t M, int64_t K, const void* X,
                                        int64_t ldx, const float* x_scale, int64_t N, void* Y, int32_t y_dtype,
                                        int64_t ldy, const float* bias, int32_t act, const void* residual, int64_t ldr,
                                        void* stream) {
  if (y_dtype != P24_F32 && y_dtype != P24_BF16) return P24_ERR_DTYPE;
  if (!f8_act_known(act)) return P24_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return P24_ERR_SHAPE;
  if (ldx < K || ldy < M || (residual && ldr < M)) return P24_ERR_SHAPE;
  if (K % 64) return P24_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return P24_OK;
  if (N == 1) ldx = K;   // a single token has no stride of its own
  if (K == 0 || K >= (1 << 24) || M >= (1 << 24) || N > 65535 * 32 || (uint64_t)ldx * 512 >= (1ull << 32)) return P24_ERR_UNSUPPORTED;
  if (!data || !w_scale || !X || !x_scale || !Y) return P24_ERR_NULL;
  const size_t ye = y_dtype == P24_F32 ? 4 : 2;
  if (!aligned(data, 16) || !aligned(X, 16) || ldx % 16 || !aligned(Y, ye) || (residual && !aligned(residual, ye)) ||
      !aligned(w_scale, 4) || !aligned(x_scale, 4) || (bias && !aligned(bias, 4)))
    return P24_ERR_ALIGN;
  F8Args a{};
  a.W = (const uint8_t*)data;
  a.w_scale = w_scale;
  a.X = (const uint8_t*)X;
  a.x_scale = x_scale;
  a.Y = Y;
  a.bias = bias;
  a.residual = residual;
  a.ldx = ldx;
  a.ldy = ldy;
  a.ldr = ldr;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.act = act;
  a.stream = aligned(Y, 128) && ldy * (int64_t)ye % 128 == 0 && (uint64_t)ldy * 1024 < (1ull << 32);
  a.res_dma = residual && aligned(residual, 16) && ldr % 8 == 0 && M % 8 == 0 && (uint64_t)ldr * 1024 < (1ull << 32);
  if (y_dtype == P24_F32) return launch_f8<float>(a, (hipStream_t)stream);
  return launch_f8<uint16_t>(a, (hipStream_t)stream);
}
