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
#include <cstring>
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
  int stream;     // the output's rows are whole cache lines (bf16)
  int res_dma;    // the residual is whole aligned 16 B chunks: it can go straight to LDS
};

// Eight e4m3 values widened to bf16 (exact).
__device__ __forceinline__ bf16x8 widen8(uint32_t v0, uint32_t v1) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v0, 1.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v0, 1.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v1, 1.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v1, 1.0f, true);
  return (bf16x8){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// On the bf16 unit instruction j takes stored values 8 j .. 8 j + 7 of each lane,
// which are k 16 j + [0, 16) of lanes 0..31 and 32 + 16 j + [0, 16) of lanes 32..63; its
// token operand is then, in lane L, k 16 j + 8 (L / 32) + [0, 8) and the same 32
// further on.  Of a 16 B chunk as the 8-bit unit takes it (k 16 (L / 32) + [0, 16))
// that is its own half and the other lane's: one exchange between the halves of
// the wave per register, after which register pair j belongs to instruction j.
__device__ __forceinline__ u32x4 halves_by_instruction(u32x4 x) {
  const auto a = __builtin_amdgcn_permlane32_swap(x[0], x[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(x[1], x[3], false, false);
  return (u32x4){a[0], b[0], a[1], b[1]};
}

// The two bf16 products of a 64-k block: `lo` and `hi` are the token's two chunks
// by instruction.
__device__ __forceinline__ f32x16 exact_product(i32x4 w, int pos, u32x4 lo, u32x4 hi, f32x16 acc) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const bf16x16 b = __builtin_shufflevector(widen8(lo[2 * j], lo[2 * j + 1]), widen8(hi[2 * j], hi[2 * j + 1]), 0, 1, 2,
                                              3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
    const bf16x8 a = widen8((uint32_t)w[2 * j], (uint32_t)w[2 * j + 1]);
    acc = j == 0 ? __builtin_amdgcn_smfmac_f32_32x32x32_bf16(a, b, acc, pos, 0, 0)
                 : __builtin_amdgcn_smfmac_f32_32x32x32_bf16(a, b, acc, pos, 0, 1);
  }
  return acc;
}

// One lane's operands of a 64-k block of a 32 x 32 tile, and their product.
template <bool EXACT>
struct F8Block {
  i32x4 a;
  int pos;
  u32x4 x[2];
  // `w` and `p`: this lane's values and positions, `xp`: the block's first k of this lane's token
  __device__ __forceinline__ void load(const uint8_t* w, const uint8_t* p, const uint8_t* xp, int half) {
    a = *reinterpret_cast<const i32x4*>(w);
    pos = *reinterpret_cast<const int*>(p);
#pragma unroll
    for (int q = 0; q < 2; ++q) x[q] = *reinterpret_cast<const u32x4*>(xp + 32 * q + 16 * half);
  }
  __device__ __forceinline__ f32x16 product(f32x16 acc) const {
    if constexpr (EXACT) {
      return exact_product(a, pos, halves_by_instruction(x[0]), halves_by_instruction(x[1]), acc);
    } else {
      const i32x8 b = __builtin_shufflevector(__builtin_bit_cast(i32x4, x[0]), __builtin_bit_cast(i32x4, x[1]), 0, 1, 2,
                                              3, 4, 5, 6, 7);
      return __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(a, b, acc, pos, 0, 0);
    }
  }
};

// A 32-row x 32-token tile per block; its W waves split K, every wave taking
// 64-k blocks w, w + W, ..., four of them on the way at a time, and the partial
// tiles meet in LDS, summed in wave order.  Nothing is shared between the waves
// before that, so each streams its part of the weights at its own pace.  With few
// tokens the time is the launch and one trip to memory, so what the last part
// needs (scales, bias, residual) is asked for first.
template <int W, typename OutT>
__global__ __launch_bounds__(W * 64) void k_f8_tokens(const F8Args args) {
  constexpr bool EXACT = sizeof(OutT) == 4;
  constexpr int PITCH = 36;   // floats per token: 32 rows, padded so that the 16-byte writes spread over the banks
  __shared__ __attribute__((aligned(16))) float part[W][32 * PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int rb = blockIdx.x;
  const int n0 = blockIdx.y * 32;
  const int blocks = args.K / 64;
  const uint8_t* x = args.X + (int64_t)min(n0 + (lane & 31), args.N - 1) * args.ldx;
  const uint8_t* group = args.W + (rb / 4) * f8_steps(args.K) * F8_PIECE;
  const uint8_t* w = group + (rb % 4) * 1024 + lane * 16;
  const uint8_t* p = group + 4096 + (rb % 4) * 256 + lane * 4;

  // the four features of a token that this thread finishes (the first 256 threads)
  const int tn = threadIdx.x / 8, tm = (threadIdx.x % 8) * 4;
  const int n = n0 + tn, m = rb * 32 + tm;
  const bool finisher = tn < 32 && n < args.N && m < args.M;
  float ws[4], bs[4] = {0, 0, 0, 0}, r[4] = {0, 0, 0, 0}, sx = 0.0f;
  if (finisher) {
    sx = args.x_scale[n];
    load_row<4>(args.w_scale + m, args.M - m, ws);
    if (args.bias) load_row<4>(args.bias + m, args.M - m, bs);
    if (args.residual) load_row<4>((const OutT*)args.residual + (int64_t)n * args.ldr + m, args.M - m, r);
  }

  constexpr int U = 4;
  f32x16 acc = {};
  for (int s = wave; s < blocks; s += U * W) {
    F8Block<EXACT> b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = s + u * W;
      if (u == 0 || at < blocks) b[u].load(w + at * F8_PIECE, p + at * F8_PIECE, x + at * 64, half);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u == 0 || s + u * W < blocks) acc = b[u].product(acc);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<f32x4*>(&part[wave][(lane & 31) * PITCH + 8 * q + 4 * half]) =
        (f32x4){acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
  __syncthreads();
  if (finisher) {
    f32x4 sum = {};
#pragma unroll
    for (int v = 0; v < W; ++v) sum += *reinterpret_cast<const f32x4*>(&part[v][tn * PITCH + tm]);
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = fmaf(sum[i] * sx, ws[i], bs[i]);
    f8_act<sizeof(OutT) == 4>(z, args.act);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] += r[i];
    store_row<4>((OutT*)args.Y + (int64_t)n * args.ldy + m, args.M - m, z);
  }
}

// ---------------------------------------------------------------------------
// Block tiles for many tokens
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void lds_void;

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
__device__ __forceinline__ int lds_b32(uint32_t addr) {
  int v;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
  return v;
}

// The fragments of one 64-k block in a wave: weights, positions, tokens.
template <int TM, int TN>
struct F8Frags {
  static constexpr int PIECES = 2;                         // LDS reads per token fragment
  i32x4 a[TM];
  int pos[TM];
  i32x4 b[TN][PIECES];
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

// 16 bytes per lane from voff + soff straight to LDS, lane l at dst + 16 l.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, voff, soff, 0, 0);
}
// the same with 4 bytes per lane
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, void* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 4, voff, soff, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int BM, int BN, int WGM, int WGN, int LW, int KG, typename OutT>
__global__ __launch_bounds__(WGM * WGN * KG * 64) void k_gemm_f8(const F8Args args) {
  using C = F8Tile<BM, BN, WGM, WGN, LW, KG>;
  constexpr bool EXACT = sizeof(OutT) == 4, INPLACE = !EXACT && KG == 1;
  constexpr int TM = C::TM, TN = C::TN, NSTAGE = C::NSTAGE;
  typedef F8Frags<TM, TN> Frags;
  __shared__ __attribute__((aligned(1024))) uint8_t lds_all[KG * NSTAGE * C::STAGE + (INPLACE ? C::SCALES : 0)];

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

  const int n_rows = min(args.N - n0, BN);
  const __amdgpu_buffer_rsrc_t x_rsrc =
      f8_rsrc(args.X + (int64_t)n0 * ldx, F8XReads<C>::bytes(n_rows, ldx, args.K));
  const F8XReads<C> x_reads(lane, wave, ldx, args.K);
  const F8WReads<C> w_reads(m0, args.M, args.K);
  const __amdgpu_buffer_rsrc_t a_rsrc =
      f8_rsrc(args.W + (int64_t)(m0 / 128) * steps * F8_PIECE, w_reads.bytes());
  uint32_t a_soff[C::A_DMA], a_dst[C::A_DMA];
#pragma unroll
  for (int j = 0; j < C::A_DMA; ++j) {
    a_dst[j] = C::X_BYTES + w_reads.unit(j, wave) * 1024;
    a_soff[j] = w_reads.scalar(j, wave);
  }
  const bool last_load = C::A_LAST == 0 || wave < C::A_LAST;
  const bool loader = wave < C::LW;

  // load Q of a loading wave for the group's step `it` (its last one past the end) into the stage at byte st
  // (WHOLE: no token of the tile lies past N, and the rows go into the scalar offset, which spares
  // an addition a load: 8192^3 257 -> 254 us)
  auto issue = [&](auto Q, int it, uint32_t st, auto WHOLE) {
    constexpr int q = decltype(Q)::value;
    uint8_t* stage = lds + st;
    const int g = k_first + min(it, count - 1);
    if constexpr (q < C::X_DMA) {
      uint32_t rows = x_reads.rows(q);
      if constexpr (decltype(WHOLE)::value) {
        load_to_lds(x_rsrc, stage + (q * C::LW + wave) * 1024, x_reads.vector(0, g == nk - 1), x_reads.scalar(g) + rows);
      } else {
        asm volatile("" : "+s"(rows));   // added here: kept over the loop, the loads' offsets would take a register each
        load_to_lds(x_rsrc, stage + (q * C::LW + wave) * 1024, x_reads.vector(rows, g == nk - 1), x_reads.scalar(g));
      }
    } else {
      constexpr int j = q - C::X_DMA;
      if (C::A_LAST != 0 && j == C::A_DMA - 1 && !last_load) return;
      load_to_lds(a_rsrc, stage + a_dst[j], w_reads.vector(lane, j, wave), (uint32_t)g * (2 * F8_PIECE) + a_soff[j]);
    }
  };

  // The residual of region r (wave r's output tile) on its way to LDS, in the
  // stages that the last steps leave free: RPS regions a stage, the stage of
  // "step" count + r / RPS.  A region is [token][16 B chunk c of its features], the
  // chunks exchanged (F8RReads) so that both the accumulators' order (one
  // feature quad of 32 tokens) and whole rows spread over the banks.
  const __amdgpu_buffer_rsrc_t r_rsrc =
      f8_rsrc((const uint8_t*)args.residual + ((int64_t)n0 * args.ldr + m0) * 2,
              INPLACE && args.res_dma ? F8RReads<C>::bytes(n_rows, args.ldr, args.M - m0) : 0u);
  const F8RReads<C> r_reads(lane, wave, args.ldr);
  const int r_t = lane / C::CH;                                  // token of a lane in its load, 64 / CH a load
  auto issue_residual = [&](auto Q, int it, uint32_t st) {
    constexpr int q = decltype(Q)::value;
    const int l = q * LW + wave;                                 // load l of the stage, of its region l / RL
    const int r = (it - count) * C::RPS + l / C::RL;
    if (q < C::RDMA && r < C::GWAVES) {
      uint32_t rest = r_reads.uniform(l, r, WGN);
      asm volatile("" : "+s"(rest));   // as for X
      load_to_lds(r_rsrc, lds + st + l * 1024, r_reads.vector(rest), 0);
    } else if (it == count || it < NSTAGE) {
      issue(Q, it, st, std::false_type{});     // until the last step has landed the waits count on a whole step's loads
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
      // piece q: 16 B chunk 2 q + h of the block's four
      const int c = 4 * ss + 2 * q + h;
      b_addr[ss][q] = lds_base + b_row + (uint32_t)((c ^ (nl & 7)) * 16);
    }
  // row blocks wm * TM .. of the tile: group wm * TM / RBG (a wave's rows lie in one group, or are whole groups)
  const uint32_t a_group = lds_base + C::X_BYTES + (uint32_t)(wm * TM / C::RBG) * (C::UNITS * 1024);
  const uint32_t a_addr = a_group + (uint32_t)(wm * TM % C::RBG) * 1024 + lane * 16;
  const uint32_t p_addr = a_group + C::P_FIRST + (uint32_t)(wm * TM % C::RBG) * 256 + lane * 4;
  static_assert(TM <= C::RBG ? C::RBG % TM == 0 : TM % C::RBG == 0, "a wave's row blocks and row groups nest");

  // read r of the TM + TM + TN * PIECES of 64-k block SS of the stage at byte `st`
  constexpr int NR = 2 * TM + TN * Frags::PIECES;
  auto read_one = [&](auto SS, auto R, uint32_t st, Frags& f) {
    constexpr int ss = decltype(SS)::value, r = decltype(R)::value;
    if constexpr (r < TM) {
      constexpr int off = (r / C::RBG) * C::UNITS * 1024 + ss * C::P_NEXT + (r % C::RBG) * 256;
      f.pos[r] = lds_b32<off>(p_addr + st);
    } else if constexpr (r < 2 * TM) {
      constexpr int i = r - TM;
      constexpr int off = (i / C::RBG) * C::UNITS * 1024 + ss * C::BLOCK + (i % C::RBG) * 1024;
      f.a[i] = lds_b128<off>(a_addr + st);
    } else {
      constexpr int j = (r - 2 * TM) / Frags::PIECES, q = (r - 2 * TM) % Frags::PIECES;
      f.b[j][q] = lds_b128<j * 4096>(b_addr[ss][q] + st);
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
  // multiply (LD 1: operands, 2: the residual, 3: operands of a tile with no token past N).
  auto block = [&](auto LD, const Frags& f, Frags& next, auto RSS, uint32_t rst, int g, uint32_t lst) {
    constexpr int NM = TM * TN, SPREAD = NM * 3 / 4 > 0 ? NM * 3 / 4 : 1;
    static_for<0, NM>([&](auto K) {
      constexpr int k = decltype(K)::value, i = k / TN, j = k % TN;
      if constexpr (EXACT) {
        acc[i][j] = exact_product(f.a[i], f.pos[i], halves_by_instruction(__builtin_bit_cast(u32x4, f.b[j][0])),
                                  halves_by_instruction(__builtin_bit_cast(u32x4, f.b[j][1])), acc[i][j]);
      } else {
        const i32x8 bv = __builtin_shufflevector(f.b[j][0], f.b[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
        acc[i][j] = __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(f.a[i], bv, acc[i][j], f.pos[i], 0, 0);
      }
      if constexpr (decltype(LD)::value == 1 && k < C::DMA) issue(K, g, lst, std::false_type{});
      if constexpr (decltype(LD)::value == 3 && k < C::DMA) issue(K, g, lst, std::true_type{});
      if constexpr (decltype(LD)::value == 2 && k < C::DMA) issue_residual(K, g, lst);
      constexpr int lo = k < SPREAD ? NR * k / SPREAD : NR, hi = k < SPREAD ? NR * (k + 1) / SPREAD : NR;
      static_for<lo, hi>([&](auto R) { read_one(RSS, R, rst, next); });
      __builtin_amdgcn_sched_barrier(0);
    });
    static_for<NM < C::DMA ? NM : C::DMA, C::DMA>([&](auto Q) {
      if constexpr (decltype(LD)::value == 1) issue(Q, g, lst, std::false_type{});
      if constexpr (decltype(LD)::value == 3) issue(Q, g, lst, std::true_type{});
      if constexpr (decltype(LD)::value == 2) issue_residual(Q, g, lst);
    });
  };

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  // until at most n steps' loads of this wave are in flight
  auto wait_steps = [&](auto N) {
    constexpr int n = decltype(N)::value;
    if (last_load) wait_loads<n * C::DMA>();
    else wait_loads<n * (C::DMA - 1)>();
  };
  const bool residual_dma = INPLACE && args.res_dma;
  if constexpr (INPLACE) {
    // scales and bias, 64 at a time, ahead of everything else
    uint8_t* sc = lds_all + NSTAGE * C::STAGE;
    const __amdgpu_buffer_rsrc_t ws = f8_rsrc((const uint8_t*)(args.w_scale + m0), (uint32_t)(args.M - m0) * 4);
    const __amdgpu_buffer_rsrc_t bs =
        f8_rsrc((const uint8_t*)(args.bias ? args.bias + m0 : nullptr), args.bias ? (uint32_t)(args.M - m0) * 4 : 0);
    const __amdgpu_buffer_rsrc_t xs = f8_rsrc((const uint8_t*)(args.x_scale + n0), (uint32_t)n_rows * 4);
    for (int u = wave; u < BM / 64; u += C::GWAVES) load4_to_lds(ws, sc + u * 256, lane * 4 + u * 256, 0);
    if (args.bias)
      for (int u = wave; u < BM / 64; u += C::GWAVES) load4_to_lds(bs, sc + BM * 4 + u * 256, lane * 4 + u * 256, 0);
    for (int u = wave; u < C::X_SCALES / 64; u += C::GWAVES) load4_to_lds(xs, sc + BM * 8 + u * 256, lane * 4 + u * 256, 0);
  }
#pragma unroll
  for (int g = 0; g < NSTAGE; ++g)
    if (loader) {
      if (residual_dma && g >= count) static_for<0, C::DMA>([&](auto Q) { issue_residual(Q, g, g * C::STAGE); });
      else static_for<0, C::DMA>([&](auto Q) { issue(Q, g, g * C::STAGE, std::false_type{}); });
    }
  wait_steps(std::integral_constant<int, NSTAGE - 1>{});
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frags f0, f1;
  static_for<0, NR>([&](auto R) { read_one(I0{}, R, 0, f0); });
  f0.wait();

  // Step `it` lives in stage it % NSTAGE.  The barrier between its two 64-k
  // blocks says that every wave has read the stage (its reads were waited for)
  // and that step it + 1 has landed (every loading wave waited for its part):
  // the stage is then refilled with step it + NSTAGE.  Steps past the end load
  // the last one again, or the residual, into stages that are not read.
  auto body = [&](auto LD, int it, uint32_t st) {
    const uint32_t nx = st == (NSTAGE - 1) * C::STAGE ? 0 : st + C::STAGE;
    block(I0{}, f0, f1, I1{}, st, 0, 0);
    f1.wait();
    if constexpr (decltype(LD)::value) wait_steps(std::integral_constant<int, NSTAGE - 2>{});
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    block(LD, f1, f0, I0{}, nx, it + NSTAGE, st);
    f0.wait();
    return nx;
  };
  auto loop = [&](auto LD) {
    const int common = nk / KG;
    const int plain = LD && residual_dma ? max(common - NSTAGE, 0) : common;
    uint32_t st = 0;
    int it = 0;
    if constexpr (decltype(LD)::value)
      if (n_rows == BN)
        for (; it < plain; ++it) st = body(I3{}, it, st);
    for (; it < plain; ++it) st = body(LD, it, st);
    if constexpr (decltype(LD)::value && INPLACE)
      for (; it < common; ++it) st = body(I2{}, it, st);
    if (KG > 1 && nk % KG) {
      if (count > common) body(LD, common, st);
      else __builtin_amdgcn_s_barrier();        // the other groups' last step
    }
  };
  if (loader) loop(I1{});
  else loop(I0{});

  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  if constexpr (INPLACE) {
    // Epilogue in place: every value is finished in the accumulators' order,
    // residual and rounding included, and goes into the wave's region as bf16;
    // whole rows of the region then go out 16 B a lane.
    const float* sc = reinterpret_cast<const float*>(lds_all + NSTAGE * C::STAGE);
    uint8_t* region = lds_all + (count + wave / C::RPS) % NSTAGE * C::STAGE + wave % C::RPS * C::REGION;
    const int m_wave = m0 + wm * C::WTM, n_wave = n0 + wn * C::WTN;
    const int m = m_wave + 8 * (lane % C::CH), left = args.M - m;     // a lane's features of a whole row
    constexpr int TPP = 64 / C::CH, PASSES = 32 / TPP;                  // tokens a pass, passes a slice
    // Rows of whole cache lines stream past the L2, which would only flush them
    // (8192^3 277 -> 263 us, 2304 x 768 with 4096 tokens 13.0 -> 10.7); parts of
    // lines are joined there (7023 x 192 with 5744 tokens 36 us, 49 streamed).
    const __amdgpu_buffer_rsrc_t y_rsrc =
        f8_rsrc((const uint8_t*)args.Y + ((int64_t)n_wave * args.ldy + m_wave) * 2, 0xFFFFFFFFu);
    // a lane's 16 B of the region's token t
    auto chunk = [&](int t) { return region + t * (C::CH * 16) + ((lane % C::CH) ^ (t % C::CH)) * 16; };
    if (args.residual && !residual_dma) {
      // rows at any alignment come through registers, four passes at a time
#pragma unroll 1
      for (int t0 = r_t; t0 < C::WTN; t0 += 4 * TPP) {
        u32x4 r[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int n = n_wave + t0 + t * TPP;
          const uint16_t* p = (const uint16_t*)args.residual + (int64_t)n * args.ldr + m;
          r[t] = (u32x4){0, 0, 0, 0};
          if (n < args.N && left >= 8) {
            r[t] = *reinterpret_cast<const u32x4_a2*>(p);
          } else if (n < args.N) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
              if (u < left) r[t][u / 2] |= (uint32_t)p[u] << (16 * (u & 1));
          }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (t0 + t * TPP < C::WTN) *reinterpret_cast<u32x4*>(chunk(t0 + t * TPP)) = r[t];
      }
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const float sx = sc[2 * BM + wn * C::WTN + 32 * j + nl];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        float z[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int f = wm * C::WTM + 32 * i + 8 * q + 4 * h;
          const f32x4 w = *reinterpret_cast<const f32x4*>(sc + f);
#pragma unroll
          for (int u = 0; u < 4; ++u) z[4 * q + u] = acc[i][j][4 * q + u] * sx * w[u];   // sx w alone can leave fp32
        }
        if (args.bias) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 b4 = *reinterpret_cast<const f32x4*>(sc + BM + wm * C::WTM + 32 * i + 8 * q + 4 * h);
#pragma unroll
            for (int u = 0; u < 4; ++u) z[4 * q + u] += b4[u];
          }
        }
        f8_act<sizeof(OutT) == 4>(z, args.act);
        uint8_t* place[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          place[q] = region + (32 * j + nl) * (C::CH * 16) + (((4 * i + q) ^ (nl % C::CH)) * 16) + 8 * h;
        if (args.residual) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x2 r = *reinterpret_cast<const u32x2*>(place[q]);
            z[4 * q] += bf16_lo(r[0]);
            z[4 * q + 1] += bf16_hi(r[0]);
            z[4 * q + 2] += bf16_lo(r[1]);
            z[4 * q + 3] += bf16_hi(r[1]);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<u32x2*>(place[q]) =
              (u32x2){pack_bf16(z[4 * q], z[4 * q + 1]), pack_bf16(z[4 * q + 2], z[4 * q + 3])};
      }
      u32x4 v[PASSES];
#pragma unroll
      for (int t = 0; t < PASSES; ++t) v[t] = *reinterpret_cast<const u32x4*>(chunk(32 * j + t * TPP + r_t));
#pragma unroll
      for (int t = 0; t < PASSES; ++t) {
        const int n = n_wave + 32 * j + t * TPP + r_t;
        if (n >= args.N) continue;
        uint16_t* p = (uint16_t*)args.Y + (int64_t)n * args.ldy + m;
        if (left >= 8) {
          if (args.stream) stream_16b(y_rsrc, v[t], (uint32_t)((32 * j + t * TPP + r_t) * args.ldy + 8 * (lane % C::CH)) * 2);
          else *reinterpret_cast<u32x4_a2*>(p) = v[t];
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (u < left) p[u] = (uint16_t)(v[t][u / 2] >> (16 * (u & 1)));
        }
      }
    }
    return;
  }

  // Epilogue by slices of 32 tokens through LDS as fp32, so that a lane holds
  // eight consecutive features of a token for the residual, the rounding and the
  // store; with split K the groups' parts meet here, summed in group order.  A
  // lane's features are the same for every token.
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
    load_row<8>(args.w_scale + m, left, ws);
    if (args.bias) load_row<8>(args.bias + m, left, bs);
    // arrived here, so that no wait for them inside the loops below also waits for stores
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(ws[i]), "+v"(bs[i]));
#pragma unroll
    for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(sx[j]));
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
        f8_act<sizeof(OutT) == 4>(z, args.act);
        if (args.residual) {
          float r[U][8];
#pragma unroll
          for (int t = 0; t < U; ++t)
            load_row<8>((const OutT*)args.residual + (int64_t)(n + t * TPI) * args.ldr + m,
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
          OutT* y = (OutT*)args.Y + (int64_t)(n + t * TPI) * args.ldy + m;
          store_row<8>(y, left, v);
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
