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
};

// Four consecutive features m .. m+3 of token n from the fp32 sums: scales,
// bias, activation, residual, one rounding.
template <typename OutT>
__device__ __forceinline__ void finish4(const F8Args& a, int n, int m, f32x4 z) {
  const float sx = a.x_scale[n];
  OutT* y = (OutT*)a.Y + (int64_t)n * a.ldy + m;
  const OutT* r = a.residual ? (const OutT*)a.residual + (int64_t)n * a.ldr + m : nullptr;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (m + i >= a.M) break;
    float v = z[i] * (sx * a.w_scale[m + i]);
    if (a.bias) v += a.bias[m + i];
    v = f8_act(v, a.act);
    if constexpr (sizeof(OutT) == 2) {
      if (r) v += __uint_as_float((uint32_t)r[i] << 16);
      y[i] = (uint16_t)pack_bf16(v, 0.0f);
    } else {
      if (r) v += r[i];
      y[i] = v;
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

template <typename OutT>
static p24_status launch_f8(const F8Args& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.M + 31) / 32), (unsigned)((a.N + 31) / 32));
  hipLaunchKernelGGL((k_f8_tokens<4, OutT>), grid, dim3(256), 0, st, a);
  return launch_status();
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
  if (K == 0 || M >= (1 << 24) || N > 65535 * 32 || (uint64_t)ldx * 512 >= (1ull << 32)) return P24_ERR_UNSUPPORTED;
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
