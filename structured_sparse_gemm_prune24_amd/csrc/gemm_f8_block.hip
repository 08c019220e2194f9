// Y = act(sum_b sx[b][n] sw[m / 128][b] S_b + bias) + residual for dense 8-bit weights W (M x K)
// and 8-bit activations X (N x K), S_b the sum over a block of 128 k, on the 8-bit MFMA
// (v_mfma_f32_16x16x128_f8f6f4: 16 rows x 16 tokens x one whole block of k).
//
// One instruction makes one S_b of 16 x 16 outputs, from a zero accumulator; four
// fused multiply-adds a lane scale it into the running sums, 16 cycles of the vector unit beside
// 32 of the matrix unit.  In its result lane L holds token L % 16, rows 4 (L / 16) + [0, 4):
// a lane's four values share one token, and a wave's rows one block of weights, so that the scale is
// one number a lane for each 16 tokens and step.
//
// Bound by the matrix unit and the power it takes: 8192^3 in 427 to 474 us, 778 k cycles of which it is busy for 524 k
// (675 k without loads, fragment reads and epilogue; 705 k without scaling and epilogue).
//
// Operands: lane L takes row (token) L % 16 and 32 of the block's k, two chunks of 16 B.  Which k a lane holds is
// free as long as both operands agree.
#include <cstdlib>
#include <cstring>
#include <type_traits>

#include "../../include/prune24_f8_block.h"
#include "p24_api_internal.hpp"
#include "p24_f8.hpp"
#include "p24_f8_cost.hpp"
#include "p24_f8b_tile.hpp"

namespace p24 {

struct F8BArgs {
  const uint8_t* W;
  const float* w_scale;
  const uint8_t* X;
  const float* x_scale;
  void* Y;
  const float* bias;
  const void* residual;
  int64_t ldw, ldx, ldxs, ldy, ldr;
  int M, N, K;
  int act;
  int nbm, nbn;
  int stream;     // the output's rows are whole cache lines
};

typedef __attribute__((address_space(3))) void lds_void_b;

template <int I, int N, typename F>
__device__ __forceinline__ void steps_of(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    steps_of<I + 1, N>(f);
  }
}

// 32 values of a row: two chunks of 16
struct F8BFrag {
  i32x4 c[2];
};

__device__ __forceinline__ bf16x8 widen_b(uint32_t v0, uint32_t v1) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v0, 1.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v0, 1.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v1, 1.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v1, 1.0f, true);
  return (bf16x8){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Operands as the unit takes them: the 8 bits themselves, or (EXACT) widened to bf16.
template <bool EXACT>
struct F8BOperand;
template <>
struct F8BOperand<false> {
  i32x8 v;
  __device__ __forceinline__ void set(const F8BFrag& f) { v = __builtin_shufflevector(f.c[0], f.c[1], 0, 1, 2, 3, 4, 5, 6, 7); }
};
template <>
struct F8BOperand<true> {
  bf16x8 v[4];
  __device__ __forceinline__ void set(const F8BFrag& f) {
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = widen_b((uint32_t)f.c[t / 2][2 * (t % 2)], (uint32_t)f.c[t / 2][2 * (t % 2) + 1]);
  }
};
__device__ __forceinline__ f32x4 block_sum(const F8BOperand<false>& a, const F8BOperand<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, (f32x4){}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_sum(const F8BOperand<true>& a, const F8BOperand<true>& b) {
  f32x4 s = {};
#pragma unroll
  for (int t = 0; t < 4; ++t) s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[t], b.v[t], s, 0, 0, 0);
  return s;
}

// LDS reads are inline assembly, waited for by lgkmcnt: the compiler would hold
// each one back until every direct-to-LDS load has landed.
template <int OFF>
__device__ __forceinline__ i32x4 lds_read16(uint32_t addr) {
  i32x4 v;
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ float lds_read4(uint32_t addr) {
  float v;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF));
  return v;
}
__device__ __forceinline__ void tie(F8BFrag& f) {
  asm volatile("" : "+v"(f.c[0]), "+v"(f.c[1]));
}
// until at most N of this wave's LDS reads are in flight
template <int N>
__device__ __forceinline__ void wait_lds() {
  asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// f8_rsrc of a place that is the same in all lanes, and is known to be (else each load would loop over its values)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* p, uint32_t bytes) {
  const uint64_t at = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at), hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
  return f8_rsrc((const uint8_t*)(uintptr_t)((uint64_t)hi << 32 | lo), __builtin_amdgcn_readfirstlane(bytes));
}

template <int BM, int BN, int WGM, int WGN, int LW, int NST, int KG, int SPAN, typename OutT>
__device__ __forceinline__ void f8_block_scaled_tile(const F8BArgs& args, uint8_t* lds_all) {
  using C = F8BTile<BM, BN, WGM, WGN, LW, NST, KG>;
  constexpr bool EXACT = sizeof(OutT) == 4;
  constexpr int TM = C::TM, TN = C::TN, PAIRS = C::PAIRS;
  typedef F8BOperand<EXACT> Operand;

  const int lane = threadIdx.x & 63;
  const int wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG == 1 ? 0 : wave_id / C::WAVES, wave = KG == 1 ? wave_id : wave_id % C::WAVES;
  const int wm = wave / WGN, wn = wave % WGN;
  uint8_t* lds = lds_all + kg * (NST * C::STAGE);       // this group's stages

  // block -> tile: each XCD a contiguous range, in groups of eight row blocks
  const uint32_t b = xcd_remap(blockIdx.x, (uint32_t)args.nbm * args.nbn);
  constexpr uint32_t GROUP = 8;
  const uint32_t group_size = GROUP * args.nbn;
  const uint32_t first_m = (b / group_size) * GROUP;
  const uint32_t gsz = min((uint32_t)args.nbm - first_m, GROUP);
  const int m0 = (int)__builtin_amdgcn_readfirstlane(first_m + (b % group_size) % gsz) * BM;
  const int n0 = (int)__builtin_amdgcn_readfirstlane((b % group_size) / gsz) * BN;
  const int m_rows = min(args.M - m0, BM), n_rows = min(args.N - n0, BN);

  const F8BSteps steps(args.K);
  // this group's steps; the groups' counts differ by one at most
  const int k_first = (int)((int64_t)steps.count * kg / KG), count = (int)((int64_t)steps.count * (kg + 1) / KG) - k_first;
  const F8BReads<LW> x_reads(lane, wave, args.ldx, steps), w_reads(lane, wave, args.ldw, steps);
  const __amdgpu_buffer_rsrc_t x_rsrc =
      uniform_rsrc(args.X + (int64_t)n0 * args.ldx, F8BReads<LW>::bytes(n_rows, args.ldx, args.K));
  const __amdgpu_buffer_rsrc_t w_rsrc =
      uniform_rsrc(args.W + (int64_t)m0 * args.ldw, F8BReads<LW>::bytes(m_rows, args.ldw, args.K));
  const int row_blocks = min((args.M + 127) / 128 - m0 / 128, C::ROW_BLOCKS);
  const __amdgpu_buffer_rsrc_t sx_rsrc =
      uniform_rsrc(args.x_scale + n0, (uint32_t)((steps.count - 1) * args.ldxs + n_rows) * 4);
  const __amdgpu_buffer_rsrc_t sw_rsrc =
      uniform_rsrc(args.w_scale + (int64_t)(m0 / 128) * steps.count, (uint32_t)(row_blocks * steps.count) * 4);
  uint32_t s_voff[C::S_DMA];
#pragma unroll
  for (int q = 0; q < C::S_DMA; ++q)
    s_voff[q] = F8BScaleReads<C>::vector(lane, F8BScaleReads<C>::number(wave, q), n_rows, row_blocks, steps.count);
  const bool loader = LW == C::WAVES || wave < LW;

  // load Q of this wave for its group's step `it` (its last one past the end) into the stage at byte st
  auto issue = [&](auto Q, int it, uint32_t st) {
    constexpr int q = decltype(Q)::value;
    const int s_all = k_first + last_of(it, count), block = steps.block(s_all);
    const bool part = s_all == 0;
    if constexpr (q < C::X_DMA) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(x_rsrc, (lds_void_b*)(lds + st + (q * LW + wave) * 1024), 16,
                                               x_reads.vector(q, part), F8BReads<LW>::scalar(block), 0, 0);
    } else if constexpr (q < C::X_DMA + C::W_DMA) {
      constexpr int j = q - C::X_DMA;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(w_rsrc, (lds_void_b*)(lds + st + C::X_BYTES + (j * LW + wave) * 1024), 16,
                                               w_reads.vector(j, part), F8BReads<LW>::scalar(block), 0, 0);
    } else {
      constexpr int j = q - C::X_DMA - C::W_DMA;
      const int number = F8BScaleReads<C>::number(wave, j);
      void* to = lds + st + C::X_BYTES + C::W_BYTES + number * 256;
      const uint32_t at = F8BScaleReads<C>::scalar(number, block, args.ldxs);
      if (F8BScaleReads<C>::tokens(number))
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sx_rsrc, (lds_void_b*)to, 4, s_voff[j], at, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sw_rsrc, (lds_void_b*)to, 4, s_voff[j], at, 0, 0);
    }
  };

  // LDS read addresses in stage 0: chunks 2 (L / 16) and one on of row L % 16 of a 16-row tile.  Sixteen lanes read
  // at a time, half of them of the next lane group: with chunk L / 16 there they met on the same banks
  // (8192^3 475 -> 450 us with the sums' delay below).
  const uint32_t base = (uint32_t)(uintptr_t)(lds_void_b*)lds;
  const int r = lane & 15, c0 = lane >> 4;
  const uint32_t in_tile = (uint32_t)((r ^ (r >> 3)) * 128);
  uint32_t x_addr[2], w_addr[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t at = base + in_tile + (uint32_t)(((2 * c0 + q) ^ (r & 7)) * 16);
    x_addr[q] = at + wn * (C::WTN * 128);
    w_addr[q] = at + C::X_BYTES + wm * (C::WTM * 128);
  }
  const uint32_t sx_addr = base + C::X_BYTES + C::W_BYTES + (wn * C::WTN + r) * 4;
  const uint32_t sw_addr = base + C::X_BYTES + C::W_BYTES + C::TOKEN_LOADS * 256 + (wm * C::WTM / 128) * 4;

  F8BFrag fa[2][2], fb[TN];       // rows: the pair in use and the next one; tokens
  float sx[TN], sw, s[TN];        // the next step's scales as they lie in LDS; this step's products
  f32x4 acc[TM][TN], sum[2][2];   // running sums; the block sums on their way into them
#pragma unroll
  for (int i = 0; i < 2; ++i) sum[0][i] = sum[1][i] = (f32x4){};
  s[TN - 1] = 0.0f;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = (f32x4){};

  auto read_pair = [&](auto P, uint32_t st, F8BFrag (&f)[2]) {
    constexpr int p = decltype(P)::value;
    steps_of<0, 2>([&](auto I) {
      constexpr int i = decltype(I)::value, off = (2 * p + i) * 2048;
      f[i].c[0] = lds_read16<off>(w_addr[0] + st);
      f[i].c[1] = lds_read16<off>(w_addr[1] + st);
    });
  };
  auto read_tokens = [&](auto J, uint32_t st) {
    constexpr int j = decltype(J)::value;
    fb[j].c[0] = lds_read16<j * 2048>(x_addr[0] + st);
    fb[j].c[1] = lds_read16<j * 2048>(x_addr[1] + st);
  };
  auto read_scales = [&](uint32_t st) {
    sw = lds_read4<0>(sw_addr + st);
    steps_of<0, TN>([&](auto J) { sx[decltype(J)::value] = lds_read4<decltype(J)::value * 64>(sx_addr + st); });
  };
  // Group g of a step is token tile g % TN of pair g / TN.  Its block sums go into the running sums one group behind
  // the matrix unit, the last group's in the next step (the first step finds zeros).
  constexpr int GROUPS = PAIRS * TN;
  auto scale_in = [&](auto G) {
    constexpr int g = decltype(G)::value, p = g / TN, j = g % TN;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[2 * p + i][j][u] = fmaf(sum[g & 1][i][u], s[j], acc[2 * p + i][j][u]);
  };
  using I0 = std::integral_constant<int, 0>;

  // A stage's refill goes out over SPAN groups: from the last pair of the step that read it into the next step.
  constexpr int EARLY = C::DMA * (SPAN < TN ? SPAN : TN) / SPAN;      // its loads under that last pair
  static_assert(SPAN >= 1 && SPAN <= GROUPS, "the refill has gone out before the next one starts");
  if (loader) {
#pragma unroll
    for (int g = 0; g < NST - 1; ++g) steps_of<0, C::DMA>([&](auto Q) { issue(Q, g, g * C::STAGE); });
    steps_of<0, EARLY>([&](auto Q) { issue(Q, NST - 1, (NST - 1) * C::STAGE); });
    wait_vm<(NST - 2) * C::DMA + EARLY>();
  }
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  if (steps.rest) {
    // the first step's weights past K, whose tokens repeat chunk 0: zeros
    for (int u = threadIdx.x; u < BM * 8; u += C::WAVES * KG * 64) {
      const int n = u >> 3, c = u & 7;
      if (16 * c >= steps.rest)
        *reinterpret_cast<u32x4*>(lds_all + C::X_BYTES + (n ^ ((n >> 3) & 1)) * 128 + ((c ^ (n & 7)) * 16)) = (u32x4){0, 0, 0, 0};
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  read_scales(0);
  read_pair(I0{}, 0, fa[0]);
  steps_of<0, TN>([&](auto J) { read_tokens(J, 0); });

  // Step `it` lives in stage it % NST.  Ahead of its last pair of row tiles, whose operands are in
  // registers by then, every wave has read the stage and step it + 1 has landed: a barrier says so, the
  // stage is refilled, and the next step's first operands are read under that pair's products.
  auto step = [&](auto LOAD, int it, uint32_t st) {
    const uint32_t nx = st == (NST - 1) * C::STAGE ? 0 : st + C::STAGE, before = st == 0 ? (NST - 1) * C::STAGE : st - C::STAGE;
    steps_of<0, PAIRS>([&](auto P) {
      constexpr int p = decltype(P)::value;
      constexpr bool last = p == PAIRS - 1;
      F8BFrag(&now)[2] = fa[p & 1];
      F8BFrag(&next)[2] = fa[(p + 1) & 1];
      if constexpr (p > 0) {
        wait_lds<0>();
        tie(now[0]);
        tie(now[1]);
      }
      if constexpr (last) {
        if constexpr (decltype(LOAD)::value) wait_vm<(NST - 2) * C::DMA>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
      Operand a[2];
      steps_of<0, TN>([&](auto J) {
        constexpr int j = decltype(J)::value;
        if constexpr (p == 0) {
          // in flight behind tokens j: the later tokens, and the next pair once it has been asked for
          wait_lds<2 * (TN - 1 - j) + (j > 0 ? 4 : 0)>();
          if constexpr (j == 0) {
            tie(now[0]);
            tie(now[1]);
            asm volatile("" : "+v"(sw));
#pragma unroll
            for (int v = 0; v < TN; ++v) asm volatile("" : "+v"(sx[v]));
          }
          tie(fb[j]);
        }
        if constexpr (j == 0) {
          a[0].set(now[0]);
          a[1].set(now[1]);
          if constexpr (!last) read_pair(std::integral_constant<int, p + 1>{}, st, next);
          else {
            read_scales(nx);
            read_pair(I0{}, nx, next);
          }
        }
        Operand t;
        t.set(fb[j]);
#pragma unroll
        for (int i = 0; i < 2; ++i) sum[(p * TN + j) & 1][i] = block_sum(a[i], t);
        if constexpr (last) {
          read_tokens(J, nx);
        }
        if constexpr (decltype(LOAD)::value) {
          constexpr int at = last ? j : TN + p * TN + j;       // group of the refill
          constexpr int lo = at < SPAN ? C::DMA * at / SPAN : C::DMA, hi = at < SPAN ? C::DMA * (at + 1) / SPAN : C::DMA;
          steps_of<lo, hi>([&](auto Q) { issue(Q, last ? it + NST : it + NST - 1, last ? st : before); });
        }
        __builtin_amdgcn_sched_barrier(0);
        scale_in(std::integral_constant<int, (p * TN + j + GROUPS - 1) % GROUPS>{});
        if constexpr (p == 0) s[j] = sx[j] * sw;       // the step's scale, ahead of its first use
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    return nx;
  };
  static_assert(PAIRS % 2 == 0, "pairs and groups alternate between two buffers: a step ends where the next expects it");
  auto loop = [&](auto LOAD) {
    uint32_t st = 0;
    for (int it = 0; it < count; ++it) st = step(LOAD, it, st);
    if (KG > 1 && count * KG < steps.count) __builtin_amdgcn_s_barrier();      // the other groups' last step
  };
  if (loader) loop(std::true_type{});
  else loop(std::false_type{});
  scale_in(std::integral_constant<int, GROUPS - 1>{});

  wait_vm<0>();
  wait_lds<0>();
  steps_of<0, TN>([&](auto J) { tie(fb[decltype(J)::value]); });
  tie(fa[0][0]);
  tie(fa[0][1]);
  asm volatile("" : "+v"(sw));
#pragma unroll
  for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(sx[j]));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  // Epilogue by slices of 16 tokens through LDS as fp32, so that a lane holds eight consecutive
  // features of a token for bias, activation, residual and store, the same features for every token.  With split K the
  // groups' parts meet here, summed in group order, and the groups share the slice's passes.
  constexpr int LPT = C::WTM / 8, TPI = 64 / LPT;      // lanes per token, tokens per pass
  constexpr int PASSES = 16 / TPI / KG;                // a group's passes
  static_assert(PASSES * KG * TPI == 16, "the groups share the passes evenly");
  constexpr int PARTS = C::WAVES * 16 * C::PITCH;      // floats of one group's slices
  float* part = reinterpret_cast<float*>(lds_all) + wave * 16 * C::PITCH;
  const int m = m0 + wm * C::WTM + 8 * (lane % LPT), left = args.M - m;
  float bs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bs[i] = 0.0f;
  if (args.bias) load_row<8>(args.bias + m, left, bs);
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(bs[i]));
  // Rows of whole cache lines stream past the L2, which would only flush them (4096 x 2304 x 768 18.2 -> 16.1 us).
  const __amdgpu_buffer_rsrc_t y_rsrc = uniform_rsrc(
      (const OutT*)args.Y + (int64_t)(n0 + wn * C::WTN) * args.ldy + m0 + wm * C::WTM, 0xFFFFFFFFu);
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    // token of pass t, within the wave's
    auto token = [&](int t) { return 16 * j + (kg * PASSES + t) * TPI + lane / LPT; };
    const int n_wave = n0 + wn * C::WTN;
    float z[8 * PASSES], res[PASSES][8];
    if (args.residual) {
#pragma unroll
      for (int t = 0; t < PASSES; ++t) {
        const int n = n_wave + token(t);
        if constexpr (EXACT) {
          float lo[4], hi[4];
          load_row<4>((const float*)args.residual + (int64_t)n * args.ldr + m, n < args.N ? left : 0, lo);
          load_row<4>((const float*)args.residual + (int64_t)n * args.ldr + m + 4, n < args.N ? left - 4 : 0, hi);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            res[t][i] = lo[i];
            res[t][4 + i] = hi[i];
          }
        } else {
          load_row<8>((const uint16_t*)args.residual + (int64_t)n * args.ldr + m, n < args.N ? left : 0, res[t]);
        }
      }
    }
    if (KG > 1 && j > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
      *reinterpret_cast<f32x4*>(part + kg * PARTS + r * C::PITCH + 16 * i + 4 * c0) = acc[i][j];
    if (KG > 1) __syncthreads();
#pragma unroll
    for (int t = 0; t < PASSES; ++t) {
      const float* row = part + (token(t) - 16 * j) * C::PITCH + 8 * (lane % LPT);
      f32x4 lo = *reinterpret_cast<const f32x4*>(row), hi = *reinterpret_cast<const f32x4*>(row + 4);
#pragma unroll
      for (int g = 1; g < KG; ++g) {
        lo += *reinterpret_cast<const f32x4*>(row + g * PARTS);
        hi += *reinterpret_cast<const f32x4*>(row + g * PARTS + 4);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) z[8 * t + i] = (i < 4 ? lo[i] : hi[i - 4]) + bs[i];
    }
    f8_act<EXACT>(z, args.act);
#pragma unroll
    for (int t = 0; t < PASSES; ++t) {
      if (n_wave + token(t) >= args.N) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = args.residual ? z[8 * t + i] + res[t][i] : z[8 * t + i];
      if (args.stream && left >= 8) {
        const uint32_t at = ((uint32_t)token(t) * (uint32_t)args.ldy + 8 * (lane % LPT)) * sizeof(OutT);
        if constexpr (EXACT) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            stream_16b(y_rsrc, (u32x4){__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                                       __float_as_uint(v[4 * h + 3])}, at + 16 * h);
        } else {
          stream_16b(y_rsrc, (u32x4){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])}, at);
        }
      } else {
        store_row<8>((OutT*)args.Y + (int64_t)(n_wave + token(t)) * args.ldy + m, left, v);
      }
    }
  }
}

// (two waves a SIMD: with more registers the compiler would hand the block sums to the accumulation
// registers, from where each goes back one by one)
template <int BM, int BN, int WGM, int WGN, int LW, int NST, int KG, int SPAN, typename OutT>
__global__ __launch_bounds__(WGM * WGN * KG * 64, 2) void k_gemm_f8_block(const F8BArgs args) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KG * NST * F8BTile<BM, BN, WGM, WGN, LW, NST, KG>::STAGE];
  f8_block_scaled_tile<BM, BN, WGM, WGN, LW, NST, KG, SPAN, OutT>(args, lds);
}

// Few tokens: a block has RT x 16 rows and TT x 16 tokens, and its W waves split K, wave w taking blocks of
// scales w, w + W, ..., U of them on the way at a time straight from memory; the partial tiles meet in
// LDS, summed in wave order.  Bound by the launch and the first bytes' way (4096 x 4096, 1 token: 5.2 us, 3.2 TB/s).
template <int W, int RT, int TT, typename OutT>
__global__ __launch_bounds__(W * 64) void k_f8_block_tokens(const F8BArgs args) {
  constexpr bool EXACT = sizeof(OutT) == 4;
  constexpr int U = RT * TT > 2 ? 2 : 4, PITCH = RT * 16 + 4;
  __shared__ __attribute__((aligned(16))) float part[W][TT * 16 * PITCH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c0 = lane >> 4;
  const int m0 = blockIdx.x * (RT * 16), n0 = blockIdx.y * (TT * 16);
  const int blocks = (args.K + 127) / 128;
  const uint8_t* w[RT];
  const uint8_t* x[TT];
  const float* sx[TT];
#pragma unroll
  for (int i = 0; i < RT; ++i) w[i] = args.W + (int64_t)min(m0 + 16 * i + r, args.M - 1) * args.ldw + 16 * c0;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int n = min(n0 + 16 * j + r, args.N - 1);
    x[j] = args.X + (int64_t)n * args.ldx + 16 * c0;
    sx[j] = args.x_scale + n;
  }
  const float* sw = args.w_scale + (int64_t)(m0 / 128) * blocks;

  // the four features of a token that a thread finishes
  constexpr int FINISH = TT * 16 * RT * 4;
  const int tn = threadIdx.x / (RT * 4), tm = (threadIdx.x % (RT * 4)) * 4;
  const int n = n0 + tn, m = m0 + tm;
  static_assert(FINISH <= W * 64, "one quad of features a thread");
  const bool finisher = (int)threadIdx.x < FINISH && n < args.N && m < args.M;
  float bs[4] = {0, 0, 0, 0}, res[4] = {0, 0, 0, 0};
  if (finisher) {
    if (args.bias) load_row<4>(args.bias + m, args.M - m, bs);
    if (args.residual) load_row<4>((const OutT*)args.residual + (int64_t)n * args.ldr + m, args.M - m, res);
  }

  f32x4 acc[RT][TT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = (f32x4){};
  for (int s = wave; s < blocks; s += U * W) {
    F8BFrag fa[U][RT], fb[U][TT];
    float scale[U][TT], ws[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = s + u * W;
      if (u > 0 && at >= blocks) continue;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool in = at * 128 + 16 * (c0 + 4 * q) < args.K;     // K's part of the block
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          fa[u][i].c[q] = (i32x4){0, 0, 0, 0};
          if (in) fa[u][i].c[q] = *reinterpret_cast<const i32x4*>(w[i] + at * 128 + 64 * q);
        }
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          fb[u][j].c[q] = (i32x4){0, 0, 0, 0};
          if (in) fb[u][j].c[q] = *reinterpret_cast<const i32x4*>(x[j] + at * 128 + 64 * q);
        }
      }
      ws[u] = sw[at];
#pragma unroll
      for (int j = 0; j < TT; ++j) scale[u][j] = sx[j][at * args.ldxs];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u > 0 && s + u * W >= blocks) continue;
      F8BOperand<EXACT> a[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) a[i].set(fa[u][i]);
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        F8BOperand<EXACT> t;
        t.set(fb[u][j]);
        const float f = scale[u][j] * ws[u];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const f32x4 sum = block_sum(a[i], t);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(sum[v], f, acc[i][j][v]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int i = 0; i < RT; ++i) *reinterpret_cast<f32x4*>(&part[wave][(16 * j + r) * PITCH + 16 * i + 4 * c0]) = acc[i][j];
  __syncthreads();
  if (finisher) {
    f32x4 sum = {};
#pragma unroll
    for (int v = 0; v < W; ++v) sum += *reinterpret_cast<const f32x4*>(&part[v][tn * PITCH + tm]);
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = sum[i] + bs[i];
    f8_act<EXACT>(z, args.act);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] += res[i];
    store_row<4>((OutT*)args.Y + (int64_t)n * args.ldy + m, args.M - m, z);
  }
}

template <int W, int RT, int TT, typename OutT>
static p24_status launch_block_tokens(const F8BArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.M + RT * 16 - 1) / (RT * 16)), (unsigned)((a.N + TT * 16 - 1) / (TT * 16)));
  hipLaunchKernelGGL((k_f8_block_tokens<W, RT, TT, OutT>), grid, dim3(W * 64), 0, st, a);
  return launch_status();
}

template <int BM, int BN, int WGM, int WGN, int LW, int NST, int KG, int SPAN, typename OutT>
static p24_status launch_block_tile(F8BArgs a, hipStream_t st) {
  a.nbm = (a.M + BM - 1) / BM;
  a.nbn = (a.N + BN - 1) / BN;
  constexpr int THREADS = WGM * WGN * KG * 64;
  if ((int64_t)a.nbm * a.nbn * THREADS > UINT32_MAX) return P24_ERR_UNSUPPORTED;   // a grid's threads
  hipLaunchKernelGGL((k_gemm_f8_block<BM, BN, WGM, WGN, LW, NST, KG, SPAN, OutT>), dim3((unsigned)(a.nbm * a.nbn)),
                     dim3(THREADS), 0, st, a);
  return launch_status();
}

// Which kernel: that of the fewest microseconds by forecast (p24_f8_cost.hpp).  Over 80 shapes drawn at random
// (1 to 8192 tokens and features, K 16 to 8192) it is 3.8 % behind the fastest, fp32 outputs 2.8 % (geometric means), at
// the median 1.8 and 0.9 %, a tenth of the shapes 11 and 6 %, the worst 54 % (88 tokens, 2965 x 3184: tokens 12.7,
// 64x32 8.2) and 36 %.  The forecast is smooth in rounds of 256 blocks, and so too low where a round has just begun.
// Measured, us, M x K with N tokens (bf16; fp32), * the one that is taken:
//   8192 x 8192, 8192    256x256 432*, 256x128 495, 128x128 544; 128x128 907*, 128x64 1090
//   8192 x 4096, 4096    256x256 114*, 256x128 133, 128x128 144; 128x128 240*, 128x64 289
//   4096 x 11264, 2048   256x128 85*, 128x128 92, 256x256 115; 128x128 160*, 128x64 193
//   4096 x 4096, 512     128x64 15.4*, 64x64 16.0, 64x32 19.0; 128x64 22.5*, 64x64 26.3
//   2304 x 768, 4096     256x256 14.3, 128x64 17.4, 128x128 17.6*, 64x64 18.0; 128x128 24.0*, 128x64 24.1
//   1000 x 4048, 517     64x64 11.0, 64x32 14.1*, 128x64 18.6; 64x64 16.4, 64x32 16.6*, 128x64 22.1
//   4096 x 4096, 32      tokens 8.1*, 64x32 8.8;  1 token 4.7*, 8.7
enum F8BKernel { B_TOKENS, B_64x32, B_64x64, B_128x64, B_128x128, B_256x128, B_256x256, B_KERNELS };

constexpr TileCost BLOCK_BF16[B_KERNELS] = {
    {16, 32, 3.45, 0.053, 1.07, 0.108},  {64, 32, 4.19, 0.195, 0.75, 0.189},   {64, 64, 4.21, 0.251, 1.14, 0.276},
    {128, 64, 4.84, 0.330, 2.04, 0.413}, {128, 128, 5.45, 0.620, 2.74, 0.621}, {256, 128, 6.18, 0.690, 6.77, 1.01},
    {256, 256, 7.78, 1.19, 9.83, 1.70},
};
// (with the conversions of an fp32 output taller tiles are no faster)
constexpr TileCost BLOCK_F32[B_256x128] = {
    {16, 32, 3.52, 0.060, 1.27, 0.111},  {64, 32, 4.73, 0.292, 0.93, 0.224},   {64, 64, 4.43, 0.438, 1.51, 0.353},
    {128, 64, 5.40, 0.554, 2.71, 0.544}, {128, 128, 6.06, 1.02, 4.36, 0.872},
};

static int64_t block_tiles(const F8BArgs& a, int bm, int bn) {
  return ((a.M + (int64_t)bm - 1) / bm) * ((a.N + (int64_t)bn - 1) / bn);
}

static F8BKernel choose_block(const F8BArgs& a, bool exact) {
  if (const char* e = getenv("P24_F8_TILE")) {
    static const char* const names[B_KERNELS] = {"tokens", "64x32", "64x64", "128x64", "128x128", "256x128", "256x256"};
    for (int i = 0; i < B_KERNELS; ++i)
      if (strcmp(e, names[i]) == 0) return exact && i > B_128x128 ? B_128x128 : (F8BKernel)i;
  }
  const TileCost* costs = exact ? BLOCK_F32 : BLOCK_BF16;
  int best = 0;
  double least = 0;
  for (int i = 0; i < (exact ? B_256x128 : B_KERNELS); ++i) {
    const double us = costs[i].us((double)block_tiles(a, costs[i].bm, costs[i].bn), a.K);
    if (i == 0 || us < least) {
      least = us;
      best = i;
    }
  }
  return (F8BKernel)best;
}

template <typename OutT>
static p24_status launch_block(const F8BArgs& a, hipStream_t st) {
  constexpr bool EXACT = sizeof(OutT) == 4;
  // one round of blocks: groups of waves split K inside a block
  auto split = [&](int bm, int bn, int round) { return a.K >= 1024 && block_tiles(a, bm, bn) <= round; };
  switch (choose_block(a, EXACT)) {
    case B_256x256:
      if constexpr (!EXACT) return launch_block_tile<256, 256, 2, 4, 8, 2, 1, 12, OutT>(a, st);
    case B_256x128:
      if constexpr (!EXACT) return launch_block_tile<256, 128, 4, 2, 8, 3, 1, 8, OutT>(a, st);
    case B_128x128: return launch_block_tile<128, 128, 2, 2, 4, 2, 1, 8, OutT>(a, st);
    case B_128x64:
      if (split(128, 64, 256)) return launch_block_tile<128, 64, 2, 2, 4, 3, 2, 4, OutT>(a, st);
      return launch_block_tile<128, 64, 2, 2, 4, 3, 1, 4, OutT>(a, st);
    case B_64x64:
      if (split(64, 64, 256)) return launch_block_tile<64, 64, 1, 4, 4, 4, 2, 2, OutT>(a, st);
      return launch_block_tile<64, 64, 1, 4, 4, 3, 1, 2, OutT>(a, st);
    case B_64x32:
      if (split(64, 32, 512)) return launch_block_tile<64, 32, 1, 2, 2, 3, 2, 2, OutT>(a, st);
      return launch_block_tile<64, 32, 1, 2, 2, 3, 1, 2, OutT>(a, st);
    default: break;
  }
  if (a.N <= 16) return launch_block_tokens<8, 1, 1, OutT>(a, st);
  return launch_block_tokens<8, 1, 2, OutT>(a, st);
}

}  // namespace p24

using namespace p24;

extern "C" P24_API p24_status gemm_f8_block(const void* W, int64_t ldw, const float* w_scale, int64_t M, int64_t K,
                                            const void* X, int64_t ldx, const float* x_scale, int64_t ldxs, int64_t N,
                                            void* Y, int32_t y_dtype, int64_t ldy, const float* bias, int32_t act,
                                            const void* residual, int64_t ldr, void* stream) {
  if (y_dtype != P24_F32 && y_dtype != P24_BF16) return P24_ERR_DTYPE;
  if (!f8_act_known(act)) return P24_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0) return P24_ERR_SHAPE;
  if (ldw < K || ldx < K || ldxs < N || ldy < M || (residual && ldr < M)) return P24_ERR_SHAPE;
  if (K % 16) return P24_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return P24_OK;
  if (N == 1) ldx = K;   // a single row has no stride of its own
  if (M == 1) ldw = K;
  if (K == 0 || K >= (1 << 24) || M >= (1 << 24) || N > 65535 * 16 || ldx >= (1 << 23) || ldw >= (1 << 23) ||
      ldxs >= (1ll << 30) / ((K + 127) / 128) - 1)
    return P24_ERR_UNSUPPORTED;
  if (!W || !w_scale || !X || !x_scale || !Y) return P24_ERR_NULL;
  const size_t ye = y_dtype == P24_F32 ? 4 : 2;
  if (!aligned(W, 16) || !aligned(X, 16) || ldw % 16 || ldx % 16 || !aligned(Y, ye) || (residual && !aligned(residual, ye)) ||
      !aligned(w_scale, 4) || !aligned(x_scale, 4) || (bias && !aligned(bias, 4)))
    return P24_ERR_ALIGN;
  F8BArgs a{};
  a.W = (const uint8_t*)W;
  a.w_scale = w_scale;
  a.X = (const uint8_t*)X;
  a.x_scale = x_scale;
  a.Y = Y;
  a.bias = bias;
  a.residual = residual;
  a.ldw = ldw;
  a.ldx = ldx;
  a.ldxs = ldxs;
  a.ldy = ldy;
  a.ldr = ldr;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.act = act;
  a.stream = aligned(Y, 128) && ldy * (int64_t)ye % 128 == 0 && (uint64_t)ldy * 2048 < (1ull << 32);
  if (y_dtype == P24_F32) return launch_block<float>(a, (hipStream_t)stream);
  return launch_block<uint16_t>(a, (hipStream_t)stream);
}
