// Values to 8 bits with a scale per block of 128: activations (a scale per token and 128 features)
// after an optional gated activation, and weights (per 128 x 128).
//
// Bound by HBM: 3 bytes a value of a bf16 row, 5 with a gate.  Sixteen lanes hold a
// block, eight values each; its maximum is four lane exchanges away.  8192 x 8192 bf16: 42 us, 4.8 TB/s;
// 2048 x 11264 with a gate 29 us, 4.0 TB/s.
//
// The quotient y / s is correctly rounded, so that a value's 8 bits follow from the formula alone:
// with i = 1 / s rounded, q = y i is within a step of it and q - (q s - y) i, the remainder taken
// exactly by an fma, is the rounded quotient (Markstein).  Three instructions a value.  The remainder is a number of fp32
// while s is 2^-90 or more; below, both are taken 2^64 times.
#include "../../include/prune24_f8_block.h"
#include "p24_api_internal.hpp"
#include "p24_f8.hpp"

namespace p24 {

struct QuantArgs {
  const void* x;
  const void* up;
  uint8_t* values;
  float* scale;
  int64_t ldx, ldu, ldv, lds;
  int rows, width, blocks;
  int act;
};

// Maximum over 16 lanes, in each: quads, mirrored halves, mirrored rows.
template <int CTRL>
__device__ __forceinline__ uint32_t quant_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t quant_max16(uint32_t v) {
  v = max(v, quant_dpp<0xB1>(v));
  v = max(v, quant_dpp<0x4E>(v));
  v = max(v, quant_dpp<0x141>(v));
  return max(v, quant_dpp<0x140>(v));
}

struct BlockScale {
  float s, lift, finite, inverse;
  __device__ __forceinline__ explicit BlockScale(uint32_t top) {
    s = f8_scale(__uint_as_float(top));
    lift = s < 0x1p-90f ? 0x1p64f : 1.0f;    // below, remainders would end under the smallest subnormal
    const float lifted = s * lift;
    inverse = 1.0f / lifted;
    finite = s == INFINITY ? 0.0f : lifted;    // then q s - y is -y, and the quotient y * 0
  }
  __device__ __forceinline__ void divide(float (&v)[8]) const {
    if (lift != 1.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= lift;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = v[i] * inverse;
      v[i] = fmaf(-inverse, fmaf(q, finite, -v[i]), q);      // in this order -0 stays -0
    }
  }
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    load_row<8>(p, left, v);
  } else {
    float a[4], b[4];
    load_row<4>(p, left, a);
    load_row<4>(p + 4, left - 4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

// Sixteen tokens a block of threads, U blocks of 128 on the way at a time; a scale's sixteen tokens
// lie side by side.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_block(const QuantArgs a) {
  constexpr int U = sizeof(T) == 2 ? 4 : 2;
  const int t = blockIdx.y * 16 + threadIdx.x / 16, lane = threadIdx.x % 16;
  if (t >= a.rows) return;      // whole rows of lanes
  const T* x = (const T*)a.x + t * a.ldx;
  const T* up = a.up ? (const T*)a.up + t * a.ldu : nullptr;
  uint8_t* out = a.values + t * a.ldv;
  const int b0 = blockIdx.x * U;
  float v[U][8], w[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (b0 + u) * 128 + 8 * lane;
    load8(x + c, a.width - c, v[u]);
    if (up) load8(up + c, a.width - c, w[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (b0 + u >= a.blocks) break;
    f8_act<false>(v[u], a.act);       // act(0) = 0: values past the row stay zero
    if (up) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] *= w[u][i];
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, mag(v[u][i]));
    const BlockScale s(quant_max16(top));
    s.divide(v[u]);
    const int c = (b0 + u) * 128 + 8 * lane;
    store_row<8>((f8_t*)out + c, a.width - c, v[u]);
    if (lane == 0) a.scale[(b0 + u) * a.lds + t] = s.s;
  }
}

// A block of weights a block of threads: 8 rows of 16 at a time.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize_weight(const QuantArgs a) {
  __shared__ uint32_t tops[4];
  const int lane = threadIdx.x % 16, c = blockIdx.x * 128 + 8 * lane;
  const int r0 = blockIdx.y * 128 + threadIdx.x / 16;
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int r = r0 + 16 * u;
    load8((const T*)a.x + (int64_t)min(r, a.rows - 1) * a.ldx + c, r < a.rows ? a.width - c : 0, v[u]);
  }
#pragma unroll
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, mag(v[u][i]));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = top;
  __syncthreads();
  const BlockScale s(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int r = r0 + 16 * u;
    if (r >= a.rows) break;
    s.divide(v[u]);
    store_row<8>((f8_t*)(a.values + r * a.ldv) + c, a.width - c, v[u]);
  }
  if (threadIdx.x == 0) a.scale[(int64_t)blockIdx.y * a.blocks + blockIdx.x] = s.s;
}

}  // namespace p24

using namespace p24;

extern "C" P24_API p24_status quantize_f8_block(const void* x, int32_t x_dtype, int64_t ldx, const void* up, int64_t ldu,
                                                int32_t act, int64_t tokens, int64_t width, void* values, int64_t ldv,
                                                float* scale, int64_t lds, void* stream) {
  if (x_dtype != P24_F32 && x_dtype != P24_BF16) return P24_ERR_DTYPE;
  if (!f8_act_known(act)) return P24_ERR_UNSUPPORTED;
  if (tokens < 0 || width < 1 || ldx < width || ldv < width || (up && ldu < width) || lds < tokens) return P24_ERR_SHAPE;
  if (width >= (1 << 24) || tokens > 65535 * 16) return P24_ERR_UNSUPPORTED;
  if (tokens == 0) return P24_OK;
  if (!x || !values || !scale) return P24_ERR_NULL;
  const size_t xe = x_dtype == P24_F32 ? 4 : 2;
  if (!aligned(x, xe) || (up && !aligned(up, xe)) || !aligned(scale, 4)) return P24_ERR_ALIGN;
  QuantArgs a{};
  a.x = x;
  a.up = up;
  a.values = (uint8_t*)values;
  a.scale = scale;
  a.ldx = ldx;
  a.ldu = ldu;
  a.ldv = ldv;
  a.lds = lds;
  a.rows = (int)tokens;
  a.width = (int)width;
  a.blocks = (int)((width + 127) / 128);
  a.act = act;
  const int per = x_dtype == P24_F32 ? 2 : 4;
  const dim3 grid((unsigned)((a.blocks + per - 1) / per), (unsigned)((tokens + 15) / 16));
  if (x_dtype == P24_F32) hipLaunchKernelGGL((k_quantize_block<float>), grid, dim3(256), 0, (hipStream_t)stream, a);
  else hipLaunchKernelGGL((k_quantize_block<uint16_t>), grid, dim3(256), 0, (hipStream_t)stream, a);
  return launch_status();
}

extern "C" P24_API p24_status quantize_weight_f8_block(const void* W, int32_t w_dtype, int64_t M, int64_t K, int64_t ldw,
                                                       void* values, int64_t ldv, float* scale, void* stream) {
  if (w_dtype != P24_F32 && w_dtype != P24_BF16) return P24_ERR_DTYPE;
  if (M < 0 || K < 0 || ldw < K || ldv < K) return P24_ERR_SHAPE;
  if (M >= (1 << 22) || K >= (1 << 22)) return P24_ERR_UNSUPPORTED;
  if (M == 0 || K == 0) return P24_OK;
  if (!W || !values || !scale) return P24_ERR_NULL;
  if (!aligned(W, w_dtype == P24_F32 ? 4 : 2) || !aligned(scale, 4)) return P24_ERR_ALIGN;
  QuantArgs a{};
  a.x = W;
  a.values = (uint8_t*)values;
  a.scale = scale;
  a.ldx = ldw;
  a.ldv = ldv;
  a.rows = (int)M;
  a.width = (int)K;
  a.blocks = (int)((K + 127) / 128);
  const dim3 grid((unsigned)a.blocks, (unsigned)((M + 127) / 128));
  if (w_dtype == P24_F32) hipLaunchKernelGGL((k_quantize_weight<float>), grid, dim3(256), 0, (hipStream_t)stream, a);
  else hipLaunchKernelGGL((k_quantize_weight<uint16_t>), grid, dim3(256), 0, (hipStream_t)stream, a);
  return launch_status();
}
