// Compression of 8-bit 2:4 weights and its inverse.  Run once when a weight is
// loaded: bound by the read of W (the second kernel finds most of it in the
// Infinity Cache).
#include "p24_api_internal.hpp"
#include "p24_f8.hpp"

namespace p24 {

template <typename T> __device__ __forceinline__ float w_value(T v);
template <> __device__ __forceinline__ float w_value<float>(float v) { return v; }
template <> __device__ __forceinline__ float w_value<uint16_t>(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// One block per row: scale[m] = max(max|W[m][:]| / 448, 2^-126).  The row's
// largest magnitude is always kept by the 2:4 selection, so the scale of the
// pruned row is the scale of the row.
template <typename T>
__global__ __launch_bounds__(256) void k_f8_scale(const T* W, int64_t ldw, int K, float* scale) {
  const T* w = W + (int64_t)blockIdx.x * ldw;
  uint32_t top = 0;
  for (int k = threadIdx.x; k < K; k += 256) top = max(top, mag(w_value<T>(w[k])));
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

// One wave per (32-row block, 64-k block): lane L compresses row L % 32,
// k 32 (L / 32) .. +32 of the block, eight groups of four, into its 16 values and
// its position word.
template <typename T>
__global__ __launch_bounds__(256) void k_f8_compress(const T* W, int64_t ldw, int64_t M, int K, int64_t steps,
                                                     int64_t nblocks, const float* scale, uint8_t* data) {
  const int lane = threadIdx.x & 63;
  const int64_t q = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);   // (row block, step)
  if (q >= nblocks) return;
  const int64_t rb = q / steps, s = q % steps;
  const int64_t row = rb * 32 + (lane & 31);
  const int64_t k0 = s * 64 + 32 * (lane >> 5);
  uint32_t v[4] = {0, 0, 0, 0}, pos = 0x44444444u;
  if (row < M && k0 < K) {    // K % 64 == 0: a half block is inside or outside
    const T* w = W + row * ldw + k0;
    const float sc = scale[row];
    pos = 0;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = w_value<T>(w[4 * g + i]);
      const uint32_t code = select_2of4(mag(f[0]), mag(f[1]), mag(f[2]), mag(f[3]));
      const uint32_t p0 = code & 3u, p1 = code >> 2;
      const float a = p0 == 0 ? f[0] : p0 == 1 ? f[1] : f[2];
      const float b = p1 == 1 ? f[1] : p1 == 2 ? f[2] : f[3];
      const uint32_t two = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a / sc, b / sc, 0, false) & 0xFFFFu;
      v[g / 2] |= two << (16 * (g & 1));
      pos |= code << (4 * g);
    }
  }
  uint8_t* piece = data + ((rb / 4) * steps + s) * F8_PIECE;
  *reinterpret_cast<u32x4*>(piece + (rb % 4) * 1024 + lane * 16) = (u32x4){v[0], v[1], v[2], v[3]};
  *reinterpret_cast<uint32_t*>(piece + 4096 + (rb % 4) * 256 + lane * 4) = pos;
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
  if (M == 0 || K == 0) return P24_OK;
  if (!W || !data || !scale) return P24_ERR_NULL;
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
