// Compression of 8-bit 2:4 weights and its inverse.  Run once when a weight is
// loaded: bound by its two reads of W (8192 x 8192 fp32 92-109 us; 188 with a
// lane per operand lane, whose loads stride by rows).
#include "p24_api_internal.hpp"
#include "p24_f8.hpp"

namespace p24 {

// Four consecutive weights, at any alignment.
template <typename T>
__device__ __forceinline__ void w_group(const T* w, float (&f)[4]) {
  if constexpr (sizeof(T) == 4) {
    const u32x4 x = *reinterpret_cast<const u32x4_a4*>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(x[i]);
  } else {
    const u32x2 x = *reinterpret_cast<const u32x2_a2*>(w);
    f[0] = bf16_lo(x[0]);
    f[1] = bf16_hi(x[0]);
    f[2] = bf16_lo(x[1]);
    f[3] = bf16_hi(x[1]);
  }
}

// One block per row: scale[m] = max(max|W[m][:]| / 448, 2^-126).  The row's
// largest magnitude is always kept by the 2:4 selection, so the scale of the
// pruned row is the scale of the row.
template <typename T>
__global__ __launch_bounds__(256) void k_f8_scale(const T* W, int64_t ldw, int K, float* scale) {
  const T* w = W + (int64_t)blockIdx.x * ldw;
  uint32_t top = 0;
  for (int k = 4 * threadIdx.x; k < K; k += 1024) {
    float f[4];
    w_group<T>(w + k, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, mag(f[i]));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t other = __shfl_xor(top, o);
    top = top > other ? top : other;
  }
  __shared__ uint32_t tops[4];
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0)
    scale[blockIdx.x] = f8_scale(__uint_as_float(max(max(tops[0], tops[1]), max(tops[2], tops[3]))));
}

// One wave per (32-row block, 64-k block), four rows at a time: a lane compresses
// one group of four, so that a row's 64 weights are one run of the load; eight
// lanes then join their pairs of values and their positions into the 16 B and the
// word of an operand lane.
template <typename T>
__global__ __launch_bounds__(256) void k_f8_compress(const T* W, int64_t ldw, int64_t M, int K, int64_t steps,
                                                     int64_t nblocks, const float* scale, uint8_t* data) {
  const int lane = threadIdx.x & 63;
  const int64_t q = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);   // (row block, step)
  if (q >= nblocks) return;
  const int64_t rb = q / steps, s = q % steps;
  const int g = lane % 16, j = g % 8;                               // group of the row, of the operand lane
  const int64_t k = s * 64 + 4 * g;
  uint8_t* piece = data + ((rb / 4) * steps + s) * F8_PIECE;
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int r = it * 4 + lane / 16;
    const int64_t row = rb * 32 + r;
    uint32_t two = 0, code = 0x4u;      // padding: zeros at positions 0, 1
    if (row < M && k < K) {
      float f[4];
      w_group<T>(W + row * ldw + k, f);
      const float sc = scale[row];
      code = select_2of4(mag(f[0]), mag(f[1]), mag(f[2]), mag(f[3]));
      const uint32_t p0 = code & 3u, p1 = code >> 2;
      const float a = p0 == 0 ? f[0] : p0 == 1 ? f[1] : f[2];
      const float b = p1 == 1 ? f[1] : p1 == 2 ? f[2] : f[3];
      two = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a / sc, b / sc, 0, false) & 0xFFFFu;
    }
    const uint32_t pair = two | (__shfl_xor(two, 1) << 16);         // whole in even lanes
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl(pair, (lane & ~7) + 2 * i);
    uint32_t pos = code << (4 * j);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) pos |= __shfl_xor(pos, o);
    if (j == 0) {
      const int L = r + 32 * (g / 8);
      *reinterpret_cast<u32x4*>(piece + (rb % 4) * 1024 + L * 16) = v;
      *reinterpret_cast<uint32_t*>(piece + 4096 + (rb % 4) * 256 + L * 4) = pos;
    }
  }
}

__global__ __launch_bounds__(256) void k_f8_decompress(const uint8_t* data, const float* scale, int64_t M, int K,
                                                       int64_t steps, int64_t nblocks, float* out, int64_t ldo) {
  const int lane = threadIdx.x & 63;
  const int64_t q = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (q >= nblocks) return;
  const int64_t rb = q / steps, s = q % steps;
  const int64_t row = rb * 32 + (lane & 31);
  const int64_t k0 = s * 64 + 32 * (lane >> 5);
  if (row >= M || k0 >= K) return;
  const uint8_t* piece = data + ((rb / 4) * steps + s) * F8_PIECE;
  const u32x4 v = *reinterpret_cast<const u32x4*>(piece + (rb % 4) * 1024 + lane * 16);
  const uint32_t pos = *reinterpret_cast<const uint32_t*>(piece + 4096 + (rb % 4) * 256 + lane * 4);
  const float sc = scale[row];
  float* o = out + row * ldo + k0;
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const uint32_t two = v[g / 2] >> (16 * (g & 1));
    const f32x2 ab = __builtin_amdgcn_cvt_pk_f32_fp8((int)two, false);
    const uint32_t code = (pos >> (4 * g)) & 15u, p0 = code & 3u, p1 = code >> 2;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) o[4 * g + i] = p0 == i ? ab[0] * sc : p1 == i ? ab[1] * sc : 0.0f;
  }
}

template <typename T>
static p24_status run_compress(const T* W, int64_t M, int64_t K, int64_t ldw, uint8_t* data, float* scale,
                               hipStream_t st) {
  const int64_t steps = f8_steps(K), nblocks = f8_groups(M) * 4 * steps;
  hipLaunchKernelGGL(k_f8_scale<T>, dim3((unsigned)M), dim3(256), 0, st, W, ldw, (int)K, scale);
  if (K == 0) return launch_status();   // rows of no values have their scales and nothing else
  hipLaunchKernelGGL(k_f8_compress<T>, dim3((unsigned)((nblocks + 3) / 4)), dim3(256), 0, st, W, ldw, M, (int)K, steps,
                     nblocks, scale, data);
  return launch_status();
}

}  // namespace p24

using namespace p24;

extern "C" P24_API size_t prune24_f8_bytes(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || K % 64 || M > INT32_MAX || K > INT32_MAX) return 0;
  return (size_t)(f8_groups(M) * f8_steps(K)) * F8_PIECE;
}

// M, K and the count of blocks (one wave each, four to a workgroup) within the grid's range
static p24_status check_mk(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || M > INT32_MAX || K > INT32_MAX) return P24_ERR_SHAPE;
  if (K % 64) return P24_ERR_UNSUPPORTED;
  // a grid holds fewer than 2^32 threads: 256 per row, 64 per block of values
  if (M >= (1 << 24) || f8_groups(M) * 4 * f8_steps(K) >= (1 << 26) - 4) return P24_ERR_UNSUPPORTED;
  return P24_OK;
}

extern "C" P24_API p24_status prune24_compress_f8(const void* W, int32_t w_dtype, int64_t M, int64_t K, int64_t ldw,
                                                  void* data, float* scale, void* stream) {
  if (w_dtype != P24_F32 && w_dtype != P24_BF16) return P24_ERR_DTYPE;
  const p24_status s = check_mk(M, K);
  if (s != P24_OK) return s;
  if (ldw < K) return P24_ERR_SHAPE;
  if (M == 0) return P24_OK;
  if (!scale || (K > 0 && (!W || !data))) return P24_ERR_NULL;
  if (!aligned(W, w_dtype == P24_F32 ? 4 : 2) || !aligned(data, 16) || !aligned(scale, 4)) return P24_ERR_ALIGN;
  if (w_dtype == P24_F32)
    return run_compress((const float*)W, M, K, ldw, (uint8_t*)data, scale, (hipStream_t)stream);
  return run_compress((const uint16_t*)W, M, K, ldw, (uint8_t*)data, scale, (hipStream_t)stream);
}

extern "C" P24_API p24_status prune24_decompress_f8(const void* data, const float* scale, int64_t M, int64_t K,
                                                    float* W_out, int64_t ldo, void* stream) {
  const p24_status s = check_mk(M, K);
  if (s != P24_OK) return s;
  if (ldo < K) return P24_ERR_SHAPE;
  if (M == 0 || K == 0) return P24_OK;
  if (!data || !scale || !W_out) return P24_ERR_NULL;
  if (!aligned(data, 16) || !aligned(scale, 4) || !aligned(W_out, 4)) return P24_ERR_ALIGN;
  const int64_t steps = f8_steps(K), nblocks = f8_groups(M) * 4 * steps;
  hipLaunchKernelGGL(k_f8_decompress, dim3((unsigned)((nblocks + 3) / 4)), dim3(256), 0, (hipStream_t)stream,
                     (const uint8_t*)data, scale, M, (int)K, steps, nblocks, W_out, ldo);
  return launch_status();
}
