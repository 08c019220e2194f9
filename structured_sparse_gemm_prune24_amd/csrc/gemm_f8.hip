// Y = act(sw sx W X^T + bias) + residual for 8-bit 2:4-sparse weights W (M x K)
// and 8-bit activations X (N x K), tokens x features out, on the sparse 8-bit
// MFMA (v_smfmac_f32_32x32x64_fp8_fp8: 32 rows x 32 tokens x 64 k, half of the
// k kept).
//
// Operands of one instruction: lane L holds row L % 32's 16 kept values of
// k 32 (L / 32) + [0, 32) with their 16 positions in one word (the order they
// are stored in), and token L % 32's 32 values of k 16 (L / 32) + [0, 16) and
// 32 + 16 (L / 32) + [0, 16).  The result: token L % 32, rows
// 8 (i / 4) + 4 (L / 32) + i % 4, i = 0..15: four consecutive features of one
// token at a time, which is the output's own order.
#include <cstdlib>
#include <string>
#include <type_traits>

#include "p24_api_internal.hpp"
#include "p24_f8.hpp"

namespace p24 {

struct F8Args {
  const uint8_t* W;
  const float* w_scale;
  const uint8_t* X;
  const float* x_scale;
  void* Y;
  const float* bias;
  const void* residual;
  int64_t ldx, ldy, ldr;
  int M, N, K;
  int act;
  int nbm, nbn;   // grid of block tiles
};

// Four consecutive features m .. m+3 of token n from the fp32 sums: scales,
// bias, activation, residual, one rounding.
template <typename OutT>
__device__ __forceinline__ void finish4(const F8Args& a, int n, int m, f32x4 sum) {
  const float sx = a.x_scale[n];
  OutT* y = (OutT*)a.Y + (int64_t)n * a.ldy + m;
  const OutT* r = a.residual ? (const OutT*)a.residual + (int64_t)n * a.ldr + m : nullptr;
  float z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[i] = sum[i] * sx;
    if (m + i < a.M) z[i] = fmaf(z[i], a.w_scale[m + i], a.bias ? a.bias[m + i] : 0.0f);
  }
  f8_act(z, a.act);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (m + i >= a.M) break;
    if constexpr (sizeof(OutT) == 2) {
      if (r) z[i] += __uint_as_float((uint32_t)r[i] << 16);
      y[i] = (uint16_t)pack_bf16(z[i], 0.0f);
    } else {
      if (r) z[i] += r[i];
      y[i] = z[i];
    }
  }
}

// Eight e4m3 values widened to bf16 (exact).
__device__ __forceinline__ bf16x8 widen8(uint32_t v0, uint32_t v1) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v0, 1.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v0, 1.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v1, 1.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v1, 1.0f, true);
  return (bf16x8){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// One 64-k block of a 32 x 32 tile.  On the bf16 unit instruction j takes stored
// values 8 j .. 8 j + 7 of each lane, which are k 16 j + [0, 16) of lanes 0..31 and
// 32 + 16 j + [0, 16) of lanes 32..63; its token operand is then, in lane L,
// k 16 j + 8 (L / 32) + [0, 8) and the same 32 further on.  `x` points at the
// block's first k of this lane's token.
template <bool EXACT>
__device__ __forceinline__ f32x16 block_product(i32x4 a, int pos, const uint8_t* x, int half, f32x16 acc) {
  if constexpr (EXACT) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const u32x2 lo = *reinterpret_cast<const u32x2*>(x + 16 * j + 8 * half);
      const u32x2 hi = *reinterpret_cast<const u32x2*>(x + 32 + 16 * j + 8 * half);
      const bf16x16 b = __builtin_shufflevector(widen8(lo[0], lo[1]), widen8(hi[0], hi[1]), 0, 1, 2, 3, 4, 5, 6, 7, 8,
                                                9, 10, 11, 12, 13, 14, 15);
      const bf16x8 av = widen8((uint32_t)a[2 * j], (uint32_t)a[2 * j + 1]);
      acc = j == 0 ? __builtin_amdgcn_smfmac_f32_32x32x32_bf16(av, b, acc, pos, 0, 0)
                   : __builtin_amdgcn_smfmac_f32_32x32x32_bf16(av, b, acc, pos, 0, 1);
    }
    return acc;
  } else {
    const i32x4 b0 = *reinterpret_cast<const i32x4*>(x + 16 * half);
    const i32x4 b1 = *reinterpret_cast<const i32x4*>(x + 32 + 16 * half);
    const i32x8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(a, b, acc, pos, 0, 0);
  }
}

// A 32-row x 32-token tile per block; its W waves split K, every wave taking
// 64-k blocks w, w + W, ..., and the partial tiles meet in LDS, summed in wave
// order.  Nothing is shared between the waves before that, so each streams its
// part of the weights at its own pace.
template <int W, typename OutT>
__global__ __launch_bounds__(W * 64) void k_f8_tokens(const F8Args args) {
  constexpr int PITCH = 36;   // floats per token: 32 rows, padded so that the 16-byte writes spread over the banks
  __shared__ __attribute__((aligned(16))) float part[W][32 * PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rb = blockIdx.x;
  const int n0 = blockIdx.y * 32;
  const int64_t steps = f8_steps(args.K);
  const int n = min(n0 + (lane & 31), args.N - 1);
  const uint8_t* x = args.X + n * args.ldx;
  const uint8_t* group = args.W + (rb / 4) * steps * F8_PIECE;
  const uint32_t v_off = (rb % 4) * 1024 + lane * 16, p_off = 4096 + (rb % 4) * 256 + lane * 4;
  f32x16 acc = {};
  for (int s = wave; s < args.K / 64; s += W) {
    const uint8_t* piece = group + (int64_t)s * F8_PIECE;
    const i32x4 a = *reinterpret_cast<const i32x4*>(piece + v_off);
    const int pos = *reinterpret_cast<const int*>(piece + p_off);
    acc = block_product<sizeof(OutT) == 4>(a, pos, x + (int64_t)s * 64, lane >> 5, acc);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<f32x4*>(&part[wave][(lane & 31) * PITCH + 8 * q + 4 * (lane >> 5)]) =
        (f32x4){acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
  __syncthreads();
  for (int q = threadIdx.x; q < 256; q += W * 64) {
    const int tn = q / 8, tm = (q % 8) * 4;
    f32x4 z = {};
#pragma unroll
    for (int w = 0; w < W; ++w) z += *reinterpret_cast<const f32x4*>(&part[w][tn * PITCH + tm]);
    if (n0 + tn < args.N) finish4<OutT>(args, n0 + tn, rb * 32 + tm, z);
  }
}

// ---------------------------------------------------------------------------
// Block tiles for many tokens
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void lds_void;

// BM rows x BN tokens per block on WGM x WGN waves; K goes by 128 values (two
// 64-k blocks) a step.  With KG > 1 there are KG such groups of waves, each with
// its own stages and its own part of K.
template <int BM, int BN, int WGM, int WGN, int LW_, int KG>
struct F8Tile {
  static constexpr int GWAVES = WGM * WGN;                 // waves of a group
  static constexpr int WTM = BM / WGM, WTN = BN / WGN;     // wave tile
  static constexpr int TM = WTM / 32, TN = WTN / 32;       // its 32 x 32 tiles
  static constexpr int LW = LW_;                           // waves of a group that load
  // stage: [X: BN rows of 128 B | per row group: two 64-k blocks of (row blocks' values, 1 KiB of positions)]
  static constexpr int GROUPS = BM >= 128 ? BM / 128 : 1;
  static constexpr int RBG = BM >= 128 ? 4 : BM / 32;      // row blocks used of a group
  static constexpr int BLOCK = (RBG + 1) * 1024;           // one 64-k block of a group in LDS
  static constexpr int X_BYTES = BN * 128, A_BYTES = GROUPS * 2 * BLOCK;
  static constexpr int STAGE = X_BYTES + A_BYTES;
  static constexpr int NSTAGE = 3 * KG * STAGE <= 160 * 1024 ? 3 : 2;
  static constexpr int X_DMA = BN / 8 / LW;                // 1 KiB loads per loading wave and step
  static constexpr int A_LOADS = A_BYTES / 1024;
  static constexpr int A_DMA = (A_LOADS + LW - 1) / LW;    // the last ones may repeat a load
  static constexpr int DMA = X_DMA + A_DMA;
  static_assert(BM % (32 * WGM) == 0 && BN % (32 * WGN) == 0, "whole 32 x 32 tiles per wave");
  static_assert((BN / 8) % LW == 0 && LW % 2 == 0 && LW <= GWAVES, "even X loads");
  static_assert(BM % 128 == 0 || BM == 64 || BM == 32, "whole row groups, or an aligned part of one");
  static_assert(NSTAGE * KG * STAGE <= 160 * 1024, "LDS");
  static_assert(NSTAGE * DMA < 64, "vmcnt range");
  // epilogue: each wave turns one 32-token slice at a time through LDS
  static constexpr int PITCH = WTM + 4;                    // floats per token
  static_assert(GWAVES * 32 * PITCH * 4 <= NSTAGE * STAGE, "the slices fit the stages' LDS");
};

template <int I, int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<I + 1, N>(f);
  }
}

// LDS reads are inline assembly, waited for by lgkmcnt: the compiler would hold
// each one back until every direct-to-LDS load has landed.
template <int OFF>
__device__ __forceinline__ i32x4 lds_b128(uint32_t addr) {
  i32x4 v;
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ u32x2 lds_b64(uint32_t addr) {
  u32x2 v;
  asm volatile("ds_read_b64 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ int lds_b32(uint32_t addr) {
  int v;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
  return v;
}

// The fragments of one 64-k block in a wave: weights, positions, tokens.
template <int TM, int TN, bool EXACT>
struct F8Frags {
  static constexpr int PIECES = EXACT ? 4 : 2;             // LDS reads per token fragment
  typedef typename std::conditional<EXACT, u32x2, i32x4>::type Piece;
  i32x4 a[TM];
  int pos[TM];
  Piece b[TN][PIECES];
  // ties every register to the wait: no use moves above it
  __device__ __forceinline__ void tie() {
#pragma unroll
    for (int i = 0; i < TM; ++i) asm volatile("" : "+v"(a[i]), "+v"(pos[i]));
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < PIECES; ++q) asm volatile("" : "+v"(b[j][q]));
  }
  __device__ __forceinline__ void wait() {
    tie();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    tie();
  }
};

// Buffer over [base, base + bytes): loads past it return zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t f8_rsrc(const uint8_t* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, (int)bytes, 0x00020000);
}
// 16 bytes per lane from voff + soff straight to LDS, lane l at dst + 16 l.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, voff, soff, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int BM, int BN, int WGM, int WGN, int LW, int KG, typename OutT>
__global__ __launch_bounds__(WGM * WGN * KG * 64) void k_gemm_f8(const F8Args args) {
  using C = F8Tile<BM, BN, WGM, WGN, LW, KG>;
  constexpr bool EXACT = sizeof(OutT) == 4;
  constexpr int TM = C::TM, TN = C::TN, NSTAGE = C::NSTAGE;
  typedef F8Frags<TM, TN, EXACT> Frags;
  __shared__ __attribute__((aligned(1024))) uint8_t lds_all[KG * NSTAGE * C::STAGE];

  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG == 1 ? 0 : wave_id / C::GWAVES, wave = KG == 1 ? wave_id : wave_id % C::GWAVES;
  const int wm = wave / WGN, wn = wave % WGN;
  uint8_t* lds = lds_all + kg * (NSTAGE * C::STAGE);     // this group's stages

  // block -> tile: each XCD a contiguous range, in groups of eight row blocks
  const uint32_t b = xcd_remap(blockIdx.x, (uint32_t)args.nbm * args.nbn);
  constexpr uint32_t GROUP = 8;
  const uint32_t group_size = GROUP * args.nbn;
  const uint32_t first_m = (b / group_size) * GROUP;
  const uint32_t gsz = min((uint32_t)args.nbm - first_m, GROUP);
  const int m0 = (int)(first_m + (b % group_size) % gsz) * BM;
  const int n0 = (int)((b % group_size) / gsz) * BN;

  const int64_t ldx = args.ldx;
  const uint32_t steps = (uint32_t)f8_steps(args.K);
  const int nk = (int)(steps / 2);
  // this group's steps: k_first .. k_first + count - 1; the groups' counts differ by one at most
  const int k_first = (int)((int64_t)nk * kg / KG), count = (int)((int64_t)nk * (kg + 1) / KG) - k_first;
  const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_void*)lds;

  // X: load q of the tile brings 8 tokens x 128 B.  LDS slot of (token n, 16 B
  // chunk c) = (n ^ ((n >> 3) & 1)) * 8 + (c ^ (n & 7)): sixteen consecutive tokens at
  // one chunk fall on sixteen bank groups.  Tokens past N lie past the resource.
  // In the last step of an odd count of 64-k blocks chunks 4..7 repeat chunks
  // 0..3: they meet the weights' zero padding.
  const int n_rows = min(args.N - n0, BN);
  const __amdgpu_buffer_rsrc_t x_rsrc =
      f8_rsrc(args.X + (int64_t)n0 * ldx, (uint32_t)((int64_t)(n_rows - 1) * ldx + args.K));
  const int x_row = 8 * wave + ((lane >> 3) ^ (wave & 1));      // q = wave; the other loads keep its parity
  const int x_chunk = (lane & 7) ^ (x_row & 7);
  const uint32_t x_voff = (uint32_t)(x_row * ldx + 16 * x_chunk);
  const uint32_t x_tail = x_voff - ((args.K & 64) && x_chunk >= 4 ? 64 : 0);
  const uint32_t x_jump = (uint32_t)(8 * C::LW * ldx);
  // weights: load q is block q % (RBG + 1) of 64-k block (q / (RBG + 1)) % 2 of row group q / (2 (RBG + 1))
  const int g0 = m0 / 128;
  const int g_count = min((int)f8_groups(args.M) - g0, C::GROUPS);
  const __amdgpu_buffer_rsrc_t a_rsrc =
      f8_rsrc(args.W + (int64_t)g0 * steps * F8_PIECE, (uint32_t)g_count * steps * F8_PIECE);
  const uint32_t a_voff = (uint32_t)lane * 16;
  uint32_t a_soff[C::A_DMA], a_dst[C::A_DMA];
#pragma unroll
  for (int j = 0; j < C::A_DMA; ++j) {
    const int q = min(j * C::LW + wave, C::A_LOADS - 1);
    const int grp = q / (2 * (C::RBG + 1)), u = q % (2 * (C::RBG + 1));
    const int s = u / (C::RBG + 1), v = u % (C::RBG + 1);
    const int part = v == C::RBG ? 4 : (m0 / 32) % 4 + v;     // positions after the values
    a_soff[j] = ((uint32_t)grp * steps + s) * F8_PIECE + part * 1024;
    a_dst[j] = C::X_BYTES + q * 1024;
  }
  const bool loader = wave < C::LW;

  // load Q of a loading wave for the group's step `it` (its last one past the end) into the stage at byte st
  auto issue = [&](auto Q, int it, uint32_t st) {
    constexpr int q = decltype(Q)::value;
    uint8_t* stage = lds + st;
    const int g = k_first + min(it, count - 1);
    if constexpr (q < C::X_DMA) {
      const uint32_t voff = g == nk - 1 ? x_tail : x_voff;
      load_to_lds(x_rsrc, stage + (q * C::LW + wave) * 1024, voff, (uint32_t)g * 128 + q * x_jump);
    } else {
      constexpr int j = q - C::X_DMA;
      load_to_lds(a_rsrc, stage + a_dst[j], a_voff, (uint32_t)g * (2 * F8_PIECE) + a_soff[j]);
    }
  };

  // LDS read addresses
  const int nl = lane & 31;
  const uint32_t b_row = (uint32_t)(wn * C::WTN + (nl ^ ((nl >> 3) & 1))) * 128;
  uint32_t b_addr[2][Frags::PIECES];     // of stage 0, per 64-k block
#pragma unroll
  for (int ss = 0; ss < 2; ++ss)
#pragma unroll
    for (int q = 0; q < Frags::PIECES; ++q) {
      // piece q: 16 B chunk 2 q + h of the block's four, or 8 B half h of chunk q
      const int c = 4 * ss + (EXACT ? q : 2 * q + h);
      b_addr[ss][q] = lds_base + b_row + (uint32_t)((c ^ (nl & 7)) * 16) + (EXACT ? 8 * h : 0);
    }
  // row blocks wm * TM .. of the tile: group wm * TM / RBG (a wave's rows lie in one group, or are whole groups)
  const uint32_t a_group = lds_base + C::X_BYTES + (uint32_t)(wm * TM / C::RBG) * (2 * C::BLOCK);
  const uint32_t a_addr = a_group + (uint32_t)(wm * TM % C::RBG) * 1024 + lane * 16;
  const uint32_t p_addr = a_group + C::RBG * 1024 + (uint32_t)((m0 / 32 + wm * TM) % 4) * 256 + lane * 4;
  static_assert(TM <= C::RBG ? C::RBG % TM == 0 : TM % C::RBG == 0, "a wave's row blocks and row groups nest");

  // read r of the TM + TM + TN * PIECES of 64-k block SS of the stage at byte `st`
  constexpr int NR = 2 * TM + TN * Frags::PIECES;
  auto read_one = [&](auto SS, auto R, uint32_t st, Frags& f) {
    constexpr int ss = decltype(SS)::value, r = decltype(R)::value;
    if constexpr (r < TM) {
      constexpr int off = (r / C::RBG) * 2 * C::BLOCK + ss * C::BLOCK + (r % C::RBG) * 256;
      f.pos[r] = lds_b32<off>(p_addr + st);
    } else if constexpr (r < 2 * TM) {
      constexpr int i = r - TM;
      constexpr int off = (i / C::RBG) * 2 * C::BLOCK + ss * C::BLOCK + (i % C::RBG) * 1024;
      f.a[i] = lds_b128<off>(a_addr + st);
    } else {
      constexpr int j = (r - 2 * TM) / Frags::PIECES, q = (r - 2 * TM) % Frags::PIECES;
      if constexpr (EXACT) f.b[j][q] = lds_b64<j * 4096>(b_addr[ss][q] + st);
      else f.b[j][q] = lds_b128<j * 4096>(b_addr[ss][q] + st);
    }
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = (f32x16){};

  // The multiplies of one 64-k block, with the reads of the next one (block RSS
  // of the stage at byte rst) spread over their first three quarters and, where
  // LD, this wave's loads of step g into the stage at byte lst, one after each
  // multiply.
  auto block = [&](auto LD, const Frags& f, Frags& next, auto RSS, uint32_t rst, int g, uint32_t lst) {
    constexpr int NM = TM * TN, SPREAD = NM * 3 / 4 > 0 ? NM * 3 / 4 : 1;
    static_for<0, NM>([&](auto K) {
      constexpr int k = decltype(K)::value, i = k / TN, j = k % TN;
      if constexpr (EXACT) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const bf16x8 av = widen8((uint32_t)f.a[i][2 * u], (uint32_t)f.a[i][2 * u + 1]);
          const bf16x16 bv =
              __builtin_shufflevector(widen8(f.b[j][u][0], f.b[j][u][1]), widen8(f.b[j][2 + u][0], f.b[j][2 + u][1]), 0,
                                      1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
          acc[i][j] = u == 0 ? __builtin_amdgcn_smfmac_f32_32x32x32_bf16(av, bv, acc[i][j], f.pos[i], 0, 0)
                             : __builtin_amdgcn_smfmac_f32_32x32x32_bf16(av, bv, acc[i][j], f.pos[i], 0, 1);
        }
      } else {
        const i32x8 bv = __builtin_shufflevector(f.b[j][0], f.b[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
        acc[i][j] = __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(f.a[i], bv, acc[i][j], f.pos[i], 0, 0);
      }
      if constexpr (decltype(LD)::value && k < C::DMA) issue(K, g, lst);
      constexpr int lo = k < SPREAD ? NR * k / SPREAD : NR, hi = k < SPREAD ? NR * (k + 1) / SPREAD : NR;
      static_for<lo, hi>([&](auto R) { read_one(RSS, R, rst, next); });
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (decltype(LD)::value)
      static_for<NM < C::DMA ? NM : C::DMA, C::DMA>([&](auto Q) { issue(Q, g, lst); });
  };

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
#pragma unroll
  for (int g = 0; g < NSTAGE; ++g)
    if (loader) static_for<0, C::DMA>([&](auto Q) { issue(Q, g, g * C::STAGE); });
  wait_loads<(NSTAGE - 1) * C::DMA>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frags f0, f1;
  static_for<0, NR>([&](auto R) { read_one(I0{}, R, 0, f0); });
  f0.wait();

  // Step `it` lives in stage it % NSTAGE.  The barrier between its two 64-k
  // blocks says that every wave has read the stage (its reads were waited for)
  // and that step it + 1 has landed (every loading wave waited for its part):
  // the stage is then refilled with step it + NSTAGE.  Steps past the end load
  // the last one again, into stages that are not read.
  auto body = [&](auto LD, int it, uint32_t st) {
    const uint32_t nx = st == (NSTAGE - 1) * C::STAGE ? 0 : st + C::STAGE;
    block(std::false_type{}, f0, f1, I1{}, st, 0, 0);
    f1.wait();
    if constexpr (decltype(LD)::value) wait_loads<(NSTAGE - 2) * C::DMA>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    block(LD, f1, f0, I0{}, nx, it + NSTAGE, st);
    f0.wait();
    return nx;
  };
  auto loop = [&](auto LD) {
    const int common = nk / KG;
    uint32_t st = 0;
    for (int it = 0; it < common; ++it) st = body(LD, it, st);
    if (KG > 1 && nk % KG) {
      if (count > common) body(LD, common, st);
      else __builtin_amdgcn_s_barrier();        // the other groups' last step
    }
  };
  if (loader) loop(std::true_type{});
  else loop(std::false_type{});

  // Epilogue: slices of 32 tokens through LDS, so that a lane holds eight
  // consecutive features of a token for the residual, the rounding and the
  // store.  A lane's features are the same for every token.
  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  constexpr int LPT = C::WTM / 8, TPI = 64 / LPT;      // lanes per token, tokens per pass
  constexpr int U = KG > 1 ? 1 : 32 / TPI < 4 ? 32 / TPI : 4;        // tokens of a lane in flight at once
  constexpr int PARTS = C::GWAVES * 32 * C::PITCH;      // floats of one group's slices
  float* part = reinterpret_cast<float*>(lds_all) + wave * 32 * C::PITCH;
  const int m = m0 + wm * C::WTM + 8 * (lane % LPT);
  auto finish = [&](auto FULL) {
    constexpr bool full = decltype(FULL)::value;   // the whole tile lies inside the output
    const int left = full ? 8 : args.M - m;
    float ws[8], bs[8], sx[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = n0 + wn * C::WTN + 32 * j + nl;
      sx[j] = args.x_scale[full ? n : min(n, args.N - 1)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) bs[i] = 0.0f;
    load8(args.w_scale + m, left, ws);
    if (args.bias) load8(args.bias + m, left, bs);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if (KG > 1 && j > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          *reinterpret_cast<f32x4*>(part + kg * PARTS + nl * C::PITCH + 32 * i + 8 * q + 4 * h) = v * sx[j];
        }
      if (KG > 1) __syncthreads();
#pragma unroll 1
      for (int t0 = kg * U; t0 < 32 / TPI; t0 += U * KG) {      // the groups share the slice's tokens
        const int tn = t0 * TPI + lane / LPT;
        const int n = n0 + wn * C::WTN + 32 * j + tn;
        float z[8 * U];
#pragma unroll
        for (int t = 0; t < U; ++t) {
          const float* row = part + (tn + t * TPI) * C::PITCH + 8 * (lane % LPT);
          f32x4 lo = *reinterpret_cast<const f32x4*>(row), hi = *reinterpret_cast<const f32x4*>(row + 4);
#pragma unroll
          for (int g = 1; g < KG; ++g) {
            lo += *reinterpret_cast<const f32x4*>(row + g * PARTS);
            hi += *reinterpret_cast<const f32x4*>(row + g * PARTS + 4);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) z[8 * t + i] = fmaf(i < 4 ? lo[i] : hi[i - 4], ws[i], bs[i]);
        }
        f8_act(z, args.act);
        if (args.residual) {
          float r[U][8];
#pragma unroll
          for (int t = 0; t < U; ++t)
            load8((const OutT*)args.residual + (int64_t)(n + t * TPI) * args.ldr + m,
                  full || n + t * TPI < args.N ? left : 0, r[t]);
#pragma unroll
          for (int t = 0; t < U; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) z[8 * t + i] += r[t][i];
        }
#pragma unroll
        for (int t = 0; t < U; ++t) {
          if (!full && n + t * TPI >= args.N) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = z[8 * t + i];
          store8<true>((OutT*)args.Y + (int64_t)(n + t * TPI) * args.ldy + m, left, v);
        }
      }
    }
  };
  if (m0 + BM <= args.M && n0 + BN <= args.N) finish(std::true_type{});
  else finish(std::false_type{});
}

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
  hipLaunchKernelGGL((k_gemm_f8<BM, BN, WGM, WGN, LW, KG, OutT>), dim3((unsigned)(a.nbm * a.nbn)),
                     dim3(WGM * WGN * KG * 64), 0, st, a);
  return launch_status();
}

// Which kernel.  A block tile's loads per multiply shrink with its size, but a
// launch needs enough blocks for 256 CUs: the largest tile that still gives about
// five eighths of them wins (144 blocks for 256 x 256, whose loads are the
// fewest).  Measured, us, M x K with N tokens:
//   8192 x 8192, 8192   256x256 264, 256x128 358, 128x128 421
//   2304 x 768, 4096    256x256 12.6 (144 blocks), 128x128 14.0
//   8192 x 4096, 1024   256x128 24.1 (256 blocks), 128x128 28.5, 256x256 28.2
//   768 x 768, 4096     128x128 6.3 (192 blocks), 256x128 7.7, 64x64 7.3
//   4096 x 4096, 512    128x64 12.4 (256 blocks), 128x128 14.2, 64x64 13.6
//   4096 x 4096, 256    64x64 10.9 (256 blocks), 128x64 11.7
// Where one round of blocks covers the CUs at most, a block has its CU to itself:
// two or four groups of waves then split K inside it, which keeps more loads in
// flight (64x64 in the last line 10.9 -> 9.2; 1000 x 4032 with 517 tokens, fp32,
// 16.7 -> 12.2; 64x32 on 4096 x 4096 with 128 tokens 9.8 -> 7.7).  A group needs a
// few steps of its own to be worth its part in the sum: K >= 1024.
// At 128 tiles of 32 x 32 or fewer, no tile that shares operands in LDS fills the
// chip, and the kernel without them is faster: 16 waves on each (4096 x 4096, one
// token: 5.3, 64x32 6.5), 4 where K is under 1024.
enum class F8Kernel { TOKENS, T64x32, T64x64, T128x64, T128x128, T256x128, T256x256 };

static int64_t f8_blocks(const F8Args& a, int bm, int bn) {
  return ((a.M + (int64_t)bm - 1) / bm) * ((a.N + (int64_t)bn - 1) / bn);
}

static F8Kernel choose_f8(const F8Args& a, bool exact) {
  if (const char* e = getenv("P24_F8_TILE")) {
    const std::string t(e);
    if (t == "tokens") return F8Kernel::TOKENS;
    if (t == "64x32") return F8Kernel::T64x32;
    if (t == "64x64") return F8Kernel::T64x64;
    if (t == "128x64") return F8Kernel::T128x64;
    if (t == "128x128") return F8Kernel::T128x128;
    if (t == "256x128" || (t == "256x256" && exact)) return F8Kernel::T256x128;
    if (t == "256x256") return F8Kernel::T256x256;
  }
  // the widened operands of an fp32 output do not fit the registers of 256 x 256
  if (!exact && f8_blocks(a, 256, 256) >= 144) return F8Kernel::T256x256;
  if (f8_blocks(a, 256, 128) >= 160) return F8Kernel::T256x128;
  if (f8_blocks(a, 128, 128) >= 160) return F8Kernel::T128x128;
  if (f8_blocks(a, 128, 64) >= 160) return F8Kernel::T128x64;
  if (f8_blocks(a, 64, 64) >= 144) return F8Kernel::T64x64;
  return f8_blocks(a, 32, 32) > 128 ? F8Kernel::T64x32 : F8Kernel::TOKENS;
}

template <typename OutT>
static p24_status launch_f8(const F8Args& a, hipStream_t st) {
  constexpr bool EXACT = sizeof(OutT) == 4;
  const bool long_k = a.K >= 1024;
  switch (choose_f8(a, EXACT)) {
    case F8Kernel::T256x256:
      if constexpr (!EXACT) return launch_tile<256, 256, 2, 4, 4, 1, OutT>(a, st);
    case F8Kernel::T256x128: return launch_tile<256, 128, 4, 2, 4, 1, OutT>(a, st);
    case F8Kernel::T128x128: return launch_tile<128, 128, 2, 4, 4, 1, OutT>(a, st);
    case F8Kernel::T128x64:
      if (long_k && f8_blocks(a, 128, 64) <= 256) return launch_tile<128, 64, 2, 2, 4, 2, OutT>(a, st);
      return launch_tile<128, 64, 2, 2, 4, 1, OutT>(a, st);
    case F8Kernel::T64x64:
      if (long_k && f8_blocks(a, 64, 64) <= 256) return launch_tile<64, 64, 2, 2, 4, 2, OutT>(a, st);
      return launch_tile<64, 64, 2, 2, 4, 1, OutT>(a, st);
    case F8Kernel::T64x32:
      if (long_k) return launch_tile<64, 32, 2, 1, 2, 4, OutT>(a, st);
      return launch_tile<64, 32, 2, 1, 2, 1, OutT>(a, st);
    case F8Kernel::TOKENS: break;
  }
  if (long_k) return launch_tokens<16, OutT>(a, st);
  return launch_tokens<4, OutT>(a, st);
}

}  // namespace p24

using namespace p24;

extern "C" P24_API size_t spmm24_f8_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  (void)M;
  (void)K;
  (void)N;
  return 0;
}

extern "C" P24_API p24_status spmm24_f8(const void* data, const float* w_scale, int64_t M, int64_t K, const void* X,
                                        int64_t ldx, const float* x_scale, int64_t N, void* Y, int32_t y_dtype,
                                        int64_t ldy, const float* bias, int32_t act, const void* residual, int64_t ldr,
                                        void* workspace, size_t ws_bytes, void* stream) {
  if (y_dtype != P24_F32 && y_dtype != P24_BF16) return P24_ERR_DTYPE;
  if (!f8_act_known(act)) return P24_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return P24_ERR_SHAPE;
  if (ldx < K || ldy < M || (residual && ldr < M)) return P24_ERR_SHAPE;
  if (K % 64) return P24_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return P24_OK;
  if (K == 0 || K >= (1 << 24) || M >= (1 << 24) || N > 65535 * 32 || (uint64_t)ldx * 512 >= (1ull << 32)) return P24_ERR_UNSUPPORTED;
  if (!data || !w_scale || !X || !x_scale || !Y) return P24_ERR_NULL;
  const size_t ye = y_dtype == P24_F32 ? 4 : 2;
  if (!aligned(data, 16) || !aligned(X, 16) || ldx % 16 || !aligned(Y, ye) || (residual && !aligned(residual, ye)) ||
      !aligned(w_scale, 4) || !aligned(x_scale, 4) || (bias && !aligned(bias, 4)))
    return P24_ERR_ALIGN;
  const size_t need = spmm24_f8_workspace_bytes(M, K, N);
  if (need && (!workspace || ws_bytes < need)) return P24_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return P24_ERR_ALIGN;
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
  if (y_dtype == P24_F32) return launch_f8<float>(a, (hipStream_t)stream);
  return launch_f8<uint16_t>(a, (hipStream_t)stream);
}
