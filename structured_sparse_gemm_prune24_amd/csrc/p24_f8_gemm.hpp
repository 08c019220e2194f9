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
#pragma once

#include <type_traits>

#include "p24_f8.hpp"
#include "p24_f8_groups.hpp"

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

// Which row of X a row of the output takes (of the grouped products: the others' is the same).
struct F8RowMap {
  const int* tokens;   // nullptr: the same row
  uint32_t last;       // of X
  template <bool GROUPED>
  __device__ __forceinline__ int of(int n) const {
    if constexpr (GROUPED)
      if (tokens) return (int)min((uint32_t)tokens[n], last);
    return n;
  }
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
// GROUPED: `args` is one expert's part, `rows` says which row of X a row of it takes.
template <int W, typename OutT, bool GROUPED>
__device__ __forceinline__ void f8_tokens_tile(const F8Args& args, const int n0, const F8RowMap rows) {
  constexpr bool EXACT = sizeof(OutT) == 4;
  constexpr int PITCH = 36;   // floats per token: 32 rows, padded so that the 16-byte writes spread over the banks
  __shared__ __attribute__((aligned(16))) float part[W][32 * PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
  const int rb = blockIdx.x;
  const int blocks = args.K / 64;
  const uint8_t* x = args.X + (int64_t)rows.template of<GROUPED>(min(n0 + (lane & 31), args.N - 1)) * args.ldx;
  const uint8_t* group = args.W + (rb / 4) * f8_steps(args.K) * F8_PIECE;
  const uint8_t* w = group + (rb % 4) * 1024 + lane * 16;
  const uint8_t* p = group + 4096 + (rb % 4) * 256 + lane * 4;

  // the four features of a token that this thread finishes (the first 256 threads)
  const int tn = threadIdx.x / 8, tm = (threadIdx.x % 8) * 4;
  const int n = n0 + tn, m = rb * 32 + tm;
  const bool finisher = tn < 32 && n < args.N && m < args.M;
  float ws[4], bs[4] = {0, 0, 0, 0}, r[4] = {0, 0, 0, 0}, sx = 0.0f;
  if (finisher) {
    sx = args.x_scale[rows.template of<GROUPED>(n)];
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

template <int W, typename OutT>
__global__ __launch_bounds__(W * 64) void k_f8_tokens(const F8Args args) {
  f8_tokens_tile<W, OutT, false>(args, blockIdx.y * 32, F8RowMap{});
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
// a read that is waited for at once
__device__ __forceinline__ int lds_b32_now(const void* p) {
  int v;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(v) : "v"((uint32_t)(uintptr_t)(lds_void*)p) : "memory");
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
constexpr int f8_lds_bytes() {
  using C = F8Tile<BM, BN, WGM, WGN, LW, KG>;
  return KG * C::NSTAGE * C::STAGE + (sizeof(OutT) != 4 && KG == 1 ? C::SCALES : 0);
}

// A block that has a CU to itself and walks over tiles: the loads of a tile's last steps bring the first two steps of the
// next one, and its epilogue keeps to the stage of its last step, so that they are on their way, and
// the stores drain, while the other goes on (4096 tokens of 8 of 64 experts with 4096 x 2048: 244 -> 232 us;
// 8192 of 8 of 64 with 2048 x 768 126 -> 112).
template <int BM, int BN, int WGM, int WGN, int LW, int KG, typename OutT>
constexpr bool f8_chained() {
  return sizeof(OutT) != 4 && KG == 1 && 2 * f8_lds_bytes<BM, BN, WGM, WGN, LW, KG, OutT>() > 160 * 1024;
}
// What it takes from a tile to the next.
template <class C>
struct F8Chain {
  static constexpr int TOKENS = C::X_SCALES * 4;   // LDS bytes behind the scales: the next tile's tokens
  bool primed = false;               // its first two steps have landed,
  uint32_t st = 0;                   // the first in the stage at this byte
  uint32_t x_row[C::X_DMA];          // its rows of X
  // the next tile
  bool more;
  const uint8_t *W, *X;
  const int* tokens;
  int N, m0, n0;
};

// One tile: rows m0 on and tokens n0 on.  GROUPED: as for f8_tokens_tile, without a residual; X's rows
// then lie anywhere, at a 32-bit offset that a lane keeps for each of its loads.
template <int BM, int BN, int WGM, int WGN, int LW, int KG, typename OutT, bool GROUPED, bool CHAIN = false>
__device__ __forceinline__ void f8_block_tile(const F8Args& args, uint8_t* lds_all, const int m0, const int n0,
                                              const F8RowMap rows, F8Chain<F8Tile<BM, BN, WGM, WGN, LW, KG>>* chain = nullptr) {
  using C = F8Tile<BM, BN, WGM, WGN, LW, KG>;
  constexpr bool EXACT = sizeof(OutT) == 4, INPLACE = !EXACT && KG == 1;
  static_assert(!CHAIN || (GROUPED && INPLACE && C::NSTAGE == 3), "a chain's stages");
  constexpr int TM = C::TM, TN = C::TN, NSTAGE = C::NSTAGE;
  typedef F8Frags<TM, TN> Frags;

  int thread = threadIdx.x;
  // a block that walks over tiles works its addresses out for each: kept over the tiles they would spill
  if constexpr (GROUPED) asm volatile("" : "+v"(thread));
  const int lane = thread & 63, h = lane >> 5;
  const int wave_id = __builtin_amdgcn_readfirstlane(thread >> 6);
  // the same in all lanes, and known to be: else the loads would loop over their values
  const bool primed = CHAIN && __builtin_amdgcn_readfirstlane(chain->primed);
  const uint32_t st_first = CHAIN ? __builtin_amdgcn_readfirstlane(chain->st) : 0;
  const int kg = KG == 1 ? 0 : wave_id / C::GWAVES, wave = KG == 1 ? wave_id : wave_id % C::GWAVES;
  // GROUPED: every other row of waves takes the tokens from the far end, so that the two waves of a SIMD (w and
  // w + 4) have different ones, and a tile of few tokens leaves each SIMD one of the waves that have some.
  const int wm = wave / WGN, wn = GROUPED && wm % 2 ? WGN - 1 - wave % WGN : wave % WGN;
  uint8_t* lds = lds_all + kg * (NSTAGE * C::STAGE);     // this group's stages

  const int64_t ldx = args.ldx;
  const uint32_t steps = (uint32_t)f8_steps(args.K);
  const int nk = (int)(steps / 2);
  // this group's steps: k_first .. k_first + count - 1; the groups' counts differ by one at most
  const int k_first = (int)((int64_t)nk * kg / KG), count = (int)((int64_t)nk * (kg + 1) / KG) - k_first;
  const uint32_t lds_base = (uint32_t)(uintptr_t)(lds_void*)lds;

  const int n_rows = min(args.N - n0, BN);
  const bool gather = GROUPED && rows.tokens;
  __amdgpu_buffer_rsrc_t x_rsrc =
      gather ? f8_rsrc(args.X, F8XReads<C>::bytes((int)rows.last + 1, ldx, args.K))
             : f8_rsrc(args.X + (int64_t)n0 * ldx, F8XReads<C>::bytes(n_rows, ldx, args.K));
  const F8XReads<C> x_reads(lane, wave, ldx, args.K);
  // rows past the tile's repeat its last one
  uint32_t x_row[GROUPED ? C::X_DMA : 1], x_back = 0;
  if constexpr (GROUPED) {
    x_back = F8XReads<C>::back(F8XReads<C>::chunk(lane, wave), args.K);
    if (primed) {
#pragma unroll
      for (int q = 0; q < C::X_DMA; ++q) x_row[q] = chain->x_row[q];
    } else {
#pragma unroll
      for (int q = 0; q < C::X_DMA; ++q) {
        const int r = min(F8XReads<C>::row(lane, wave, q), n_rows - 1);
        x_row[q] = (uint32_t)(gather ? rows.template of<true>(n0 + r) : r) * (uint32_t)ldx + F8XReads<C>::chunk(lane, wave) * 16;
      }
    }
  }
  const F8WReads<C> w_reads(m0, args.M, args.K);
  __amdgpu_buffer_rsrc_t a_rsrc =
      f8_rsrc(args.W + (int64_t)(m0 / 128) * steps * F8_PIECE, w_reads.bytes());
  uint32_t a_soff[C::A_DMA], a_dst[C::A_DMA];
#pragma unroll
  for (int j = 0; j < C::A_DMA; ++j) {
    a_dst[j] = C::X_BYTES + w_reads.unit(j, wave) * 1024;
    a_soff[j] = w_reads.scalar(j, wave);
  }
  const bool last_load = C::A_LAST == 0 || wave < C::A_LAST;
  const bool loader = C::LW == C::GWAVES || wave < C::LW;

  // load Q of a loading wave for the group's step `it` (its last one past the end) into the stage at byte st
  // (WHOLE: no token of the tile lies past N, and the rows go into the scalar offset, which spares
  // an addition a load: 8192^3 257 -> 254 us)
  auto issue = [&](auto Q, int it, uint32_t st, auto WHOLE) {
    constexpr int q = decltype(Q)::value;
    uint8_t* stage = lds + st;
    const int g = k_first + min(it, count - 1);
    if constexpr (q < C::X_DMA) {
      uint32_t more = x_reads.rows(q);
      if constexpr (GROUPED) {
        load_to_lds(x_rsrc, stage + (q * C::LW + wave) * 1024, x_row[q] - (x_back & (g == nk - 1 ? ~0u : 0u)), x_reads.scalar(g));
      } else if constexpr (decltype(WHOLE)::value) {
        load_to_lds(x_rsrc, stage + (q * C::LW + wave) * 1024, x_reads.vector(0, g == nk - 1), x_reads.scalar(g) + more);
      } else {
        asm volatile("" : "+s"(more));   // added here: kept over the loop, the loads' offsets would take a register each
        load_to_lds(x_rsrc, stage + (q * C::LW + wave) * 1024, x_reads.vector(more, g == nk - 1), x_reads.scalar(g));
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
  // multiply (LD 1: operands, 2: the residual, 3: operands of a tile with no token past N,
  // 4: the next tile's operands).
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
      if constexpr (decltype(LD)::value == 4 && k < C::DMA) issue(K, g, lst, std::false_type{});
      constexpr int lo = k < SPREAD ? NR * k / SPREAD : NR, hi = k < SPREAD ? NR * (k + 1) / SPREAD : NR;
      static_for<lo, hi>([&](auto R) { read_one(RSS, R, rst, next); });
      __builtin_amdgcn_sched_barrier(0);
    });
    static_for<NM < C::DMA ? NM : C::DMA, C::DMA>([&](auto Q) {
      if constexpr (decltype(LD)::value == 1) issue(Q, g, lst, std::false_type{});
      if constexpr (decltype(LD)::value == 3) issue(Q, g, lst, std::true_type{});
      if constexpr (decltype(LD)::value == 2) issue_residual(Q, g, lst);
      if constexpr (decltype(LD)::value == 4) issue(Q, g, lst, std::false_type{});
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
  const bool residual_dma = INPLACE && !GROUPED && args.res_dma;
  // (the next tile's tokens are there after two steps)
  const bool link = CHAIN && __builtin_amdgcn_readfirstlane(chain->more && count >= 5);
  uint8_t* next_tokens = lds_all + NSTAGE * C::STAGE + C::SCALES;
  if constexpr (INPLACE) {
    // scales and bias, 64 at a time, ahead of everything else
    uint8_t* sc = lds_all + NSTAGE * C::STAGE;
    const __amdgpu_buffer_rsrc_t ws = f8_rsrc((const uint8_t*)(args.w_scale + m0), (uint32_t)(args.M - m0) * 4);
    const __amdgpu_buffer_rsrc_t bs =
        f8_rsrc((const uint8_t*)(args.bias ? args.bias + m0 : nullptr), args.bias ? (uint32_t)(args.M - m0) * 4 : 0);
    const __amdgpu_buffer_rsrc_t xs =
        gather ? f8_rsrc((const uint8_t*)args.x_scale, (rows.last + 1) * 4) : f8_rsrc((const uint8_t*)(args.x_scale + n0), (uint32_t)n_rows * 4);
    for (int u = wave; u < BM / 64; u += C::GWAVES) load4_to_lds(ws, sc + u * 256, lane * 4 + u * 256, 0);
    if (args.bias)
      for (int u = wave; u < BM / 64; u += C::GWAVES) load4_to_lds(bs, sc + BM * 4 + u * 256, lane * 4 + u * 256, 0);
    for (int u = wave; u < C::X_SCALES / 64; u += C::GWAVES) {
      uint32_t at = lane * 4 + u * 256;
      if (gather && primed) {
        // (past the tile's rows: some row of X)
        at = min((uint32_t)lds_b32_now(next_tokens + at), rows.last) * 4;
      } else if (gather) {
        at = (uint32_t)rows.template of<true>(n0 + min(lane + u * 64, n_rows - 1)) * 4;
      }
      load4_to_lds(xs, sc + BM * 8 + u * 256, at, 0);
      if (CHAIN && link && chain->tokens)   // its own place, which no other wave reads before the next barrier
        load4_to_lds(f8_rsrc((const uint8_t*)(chain->tokens + chain->n0), (uint32_t)min(chain->N - chain->n0, BN) * 4),
                     next_tokens + u * 256, lane * 4 + u * 256, 0);
    }
  }
  if (primed) {
    if (loader)
      static_for<0, C::DMA>([&](auto Q) {
        issue(Q, 2, st_first == 0 ? 2 * C::STAGE : st_first - C::STAGE, std::false_type{});
      });
  } else {
#pragma unroll
    for (int g = 0; g < NSTAGE; ++g)
      if (loader) {
        if (residual_dma && g >= count) static_for<0, C::DMA>([&](auto Q) { issue_residual(Q, g, g * C::STAGE); });
        else static_for<0, C::DMA>([&](auto Q) { issue(Q, g, g * C::STAGE, std::false_type{}); });
      }
    wait_steps(std::integral_constant<int, NSTAGE - 1>{});
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  Frags f0, f1;
  static_for<0, NR>([&](auto R) { read_one(I0{}, R, st_first, f0); });
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
    // (a primed tile's second step is there; the wait would be for the last tile's stores)
    if constexpr (decltype(LD)::value)
      if (!CHAIN || it > 0 || !primed) wait_steps(std::integral_constant<int, NSTAGE - 2>{});
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    block(LD, f1, f0, I0{}, nx, decltype(LD)::value == 4 ? it + NSTAGE - count : it + NSTAGE, st);
    f0.wait();
    return nx;
  };
  // the loads go on with the next tile
  auto turn = [&]() {
    const int n_next = min(chain->N - chain->n0, BN);
    const bool gathered = chain->tokens != nullptr;
    x_rsrc = gathered ? f8_rsrc(chain->X, F8XReads<C>::bytes((int)rows.last + 1, ldx, args.K))
                      : f8_rsrc(chain->X + (int64_t)chain->n0 * ldx, F8XReads<C>::bytes(n_next, ldx, args.K));
#pragma unroll
    for (int q = 0; q < C::X_DMA; ++q) {
      int r = min(F8XReads<C>::row(lane, wave, q), n_next - 1);
      if (gathered) r = (int)min((uint32_t)lds_b32_now(next_tokens + r * 4), rows.last);
      x_row[q] = (uint32_t)r * (uint32_t)ldx + F8XReads<C>::chunk(lane, wave) * 16;
    }
    const F8WReads<C> reads(chain->m0, args.M, args.K);
    a_rsrc = f8_rsrc(chain->W + (int64_t)(chain->m0 / 128) * steps * F8_PIECE, reads.bytes());
#pragma unroll
    for (int j = 0; j < C::A_DMA; ++j) a_soff[j] = reads.scalar(j, wave);
  };
  uint32_t st_end = 0;    // the stage behind the last step's
  auto loop = [&](auto LD) {
    if constexpr (CHAIN) {
      uint32_t st = st_first;
      int it = 0;
      for (const int own = link ? count - NSTAGE : count - 1; it < own; ++it) st = body(LD, it, st);
      if (link) {
        if (decltype(LD)::value) turn();
        for (; it < count - 1; ++it) st = body(std::integral_constant<int, decltype(LD)::value ? 4 : 0>{}, it, st);
      }
      // (the last step's stage is the epilogue's)
      st_end = body(I0{}, count - 1, st);
      return;
    }
    const int common = nk / KG;
    const int plain = LD && residual_dma ? max(common - NSTAGE, 0) : common;
    uint32_t st = 0;
    int it = 0;
    if constexpr (decltype(LD)::value && !GROUPED)
      if (n_rows == BN)
        for (; it < plain; ++it) st = body(I3{}, it, st);
    for (; it < plain; ++it) st = body(LD, it, st);
    if constexpr (decltype(LD)::value && INPLACE && !GROUPED)
      for (; it < common; ++it) st = body(I2{}, it, st);
    if (KG > 1 && nk % KG) {
      if (count > common) body(LD, common, st);
      else __builtin_amdgcn_s_barrier();        // the other groups' last step
    }
  };
  // a wave without tokens loads and keeps step
  auto idle = [&]() {
    uint32_t st = st_first;
    for (int it = 0; it < nk / KG; ++it) {
      if constexpr (CHAIN)
        if (loader && link && it == count - NSTAGE) turn();
      if (loader && (!CHAIN || it > 0 || !primed)) wait_steps(std::integral_constant<int, NSTAGE - 2>{});
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (loader && (!CHAIN || it < count - 1))
        static_for<0, C::DMA>([&](auto Q) {
          issue(Q, CHAIN && link && it >= count - NSTAGE ? it + NSTAGE - count : it + NSTAGE, st, std::false_type{});
        });
      st = st == (NSTAGE - 1) * C::STAGE ? 0 : st + C::STAGE;
    }
    st_end = st;
  };
  static_assert(!GROUPED || KG == 1, "idle waves keep step with one group");
  if (GROUPED && wn * C::WTN >= n_rows) idle();
  else if (loader) loop(I1{});
  else loop(I0{});

  wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  if constexpr (CHAIN) {
    chain->primed = link;
    chain->st = link ? st_end : 0;
#pragma unroll
    for (int q = 0; q < C::X_DMA; ++q) chain->x_row[q] = x_row[q];
  }
  if (GROUPED && wn * C::WTN >= n_rows) return;

  if constexpr (INPLACE) {
    // Epilogue in place: every value is finished in the accumulators' order,
    // residual and rounding included, and goes into the wave's region as bf16;
    // whole rows of the region then go out 16 B a lane.
    const float* sc = reinterpret_cast<const float*>(lds_all + NSTAGE * C::STAGE);
    // a slice: 32 tokens and CH chunks of features; CHAIN: one at a time, in the last step's stage
    constexpr int CH = CHAIN && C::CH > 8 ? 8 : C::CH, SLICES = C::CH / CH, TMS = TM / SLICES;
    static_assert(!CHAIN || C::GWAVES * 32 * CH * 16 <= C::STAGE, "the slices fit a stage");
    uint8_t* region = CHAIN ? lds_all + (st_end == 0 ? (NSTAGE - 1) * C::STAGE : st_end - C::STAGE) + wave * (32 * CH * 16)
                            : lds_all + (count + wave / C::RPS) % NSTAGE * C::STAGE + wave % C::RPS * C::REGION;
    const int m_wave = m0 + wm * C::WTM, n_wave = n0 + wn * C::WTN;
    constexpr int TPP = 64 / CH, PASSES = 32 / TPP;                     // tokens a pass, passes a slice
    // Rows of whole cache lines stream past the L2, which would only flush them
    // (8192^3 277 -> 263 us, 2304 x 768 with 4096 tokens 13.0 -> 10.7); parts of
    // lines are joined there (7023 x 192 with 5744 tokens 36 us, 49 streamed).
    const __amdgpu_buffer_rsrc_t y_rsrc =
        f8_rsrc((const uint8_t*)args.Y + ((int64_t)n_wave * args.ldy + m_wave) * 2, 0xFFFFFFFFu);
    // a lane's 16 B of the region's token t
    auto chunk = [&](int t) { return region + t * (CH * 16) + ((lane % CH) ^ (t % CH)) * 16; };
    if (!GROUPED && args.residual && !residual_dma) {
      // rows at any alignment come through registers, four passes at a time
      const int m = m_wave + 8 * (lane % CH), left = args.M - m;
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
      for (int slice = 0; slice < SLICES; ++slice) {
        const int m = m_wave + 8 * (CH * slice + lane % CH), left = args.M - m;     // a lane's features of a whole row
        const int t_first = CHAIN ? 0 : 32 * j;                                     // in the region
#pragma unroll
        for (int i = slice * TMS; i < (slice + 1) * TMS; ++i) {
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
            place[q] = region + (t_first + nl) * (CH * 16) + (((4 * (i - slice * TMS) + q) ^ (nl % CH)) * 16) + 8 * h;
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
        for (int t = 0; t < PASSES; ++t) v[t] = *reinterpret_cast<const u32x4*>(chunk(t_first + t * TPP + lane / CH));
#pragma unroll
        for (int t = 0; t < PASSES; ++t) {
          const int token = 32 * j + t * TPP + lane / CH, n = n_wave + token;
          if (n >= args.N) continue;
          uint16_t* p = (uint16_t*)args.Y + (int64_t)n * args.ldy + m;
          if (left >= 8) {
            if (args.stream) stream_16b(y_rsrc, v[t], (uint32_t)(token * args.ldy + 8 * (CH * slice + lane % CH)) * 2);
            else *reinterpret_cast<u32x4_a2*>(p) = v[t];
          } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
              if (u < left) p[u] = (uint16_t)(v[t][u / 2] >> (16 * (u & 1)));
          }
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
      sx[j] = args.x_scale[rows.template of<GROUPED>(full ? n : min(n, args.N - 1))];
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

// A block a tile; each XCD a contiguous range of them.
template <int BM, int BN, int WGM, int WGN, int LW, int KG, typename OutT>
__global__ __launch_bounds__(WGM * WGN * KG * 64) void k_gemm_f8(const F8Args args) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[f8_lds_bytes<BM, BN, WGM, WGN, LW, KG, OutT>()];
  uint32_t bm, bn;
  f8_place(xcd_remap(blockIdx.x, (uint32_t)args.nbm * args.nbn), args.nbm, args.nbn, bm, bn);
  f8_block_tile<BM, BN, WGM, WGN, LW, KG, OutT, false>(args, lds, (int)bm * BM, (int)bn * BN, F8RowMap{});
}

}  // namespace p24
