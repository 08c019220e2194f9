// Row operators around the 8-bit products: RMS norm with the residual's
// addition, and the gated activation, each with an 8-bit, bf16 or fp32 output.
//
// One row (token) belongs to G threads, E chunks of 16 input bytes each,
// held in registers from the one read to the one write: the row's statistics
// (sum of squares, largest magnitude) need the whole row before the first
// output, and a second read would cost what the first did.  Bound by HBM: the
// norm moves 7 bytes per value (bf16 in, residual, sum, 8-bit out), the gated
// activation 5.
//
// Norm: with r = 1 / sqrt(mean(h^2) + eps), y_i = h_i r w_i, so
// max|y| = r max|h_i w_i|: the sum of squares and the maximum of |h w| come out
// of one pass and one reduction.
#include "p24_api_internal.hpp"
#include "p24_f8.hpp"

namespace p24 {

struct RowArgs {
  const void* a;        // x, or the gate
  const void* b;        // residual, or `up`; may be nullptr
  const float* weight;  // norm only
  void* h;              // norm with a residual: the sum
  void* y;
  float* scale;         // 8-bit output
  int64_t lda, ldb, ldh, ldy;
  int rows, width;
  float eps;
  int act;
};

// Sum and magnitude maximum over the G threads of a row, the same in each.
template <int G>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top) {
#pragma unroll
  for (int o = (G < 64 ? G : 64) / 2; o > 0; o >>= 1) {
    sum += __shfl_xor(sum, o);
    const uint32_t other = __shfl_xor(top, o);
    top = top > other ? top : other;
  }
  if constexpr (G > 64) {
    constexpr int W = G / 64;
    __shared__ float sums[W];
    __shared__ uint32_t tops[W];
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      sums[wave] = sum;
      tops[wave] = top;
    }
    __syncthreads();
    sum = 0.0f;
    top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      sum += sums[i];
      top = top > tops[i] ? top : tops[i];
    }
  }
}

// G threads a row; a block of 256 threads holds several rows where G is a wave or less.
template <int G> constexpr int ROW_BLOCK = G <= 64 ? 256 : G;

template <typename T, typename OutT, int G, int E, bool NORM>
__global__ __launch_bounds__(ROW_BLOCK<G>) void k_rows(const RowArgs args) {
  constexpr int V = 16 / sizeof(T);   // values of a chunk: 16 bytes of input
  const int t = threadIdx.x % G;
  const int64_t row = (int64_t)blockIdx.x * (ROW_BLOCK<G> / G) + threadIdx.x / G;
  if (row >= args.rows) return;   // whole groups of G threads, and whole blocks where G spans waves
  const int width = args.width;
  const T* a = (const T*)args.a + row * args.lda;
  const T* b = args.b ? (const T*)args.b + row * args.ldb : nullptr;

  float v[E][V], u[E][V], w[NORM ? E : 1][V];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (t + e * G) * V;
    load_row<V>(a + c, width - c, v[e]);
    if (b) load_row<V>(b + c, width - c, u[e]);
  }
  // the weights are asked for ahead of the sum's store, which the compiler must keep in its place
  if constexpr (NORM) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (t + e * G) * V;
      load_row<V>(args.weight + c, width - c, w[e]);
    }
  }
  if constexpr (!NORM) {
#pragma unroll
    for (int e = 0; e < E; ++e) f8_act(v[e], args.act);
  }
  if (b) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (t + e * G) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) v[e][i] = NORM ? v[e][i] + u[e][i] : v[e][i] * u[e][i];
      if constexpr (NORM) store_row<V>((T*)args.h + row * args.ldh + c, width - c, v[e]);
    }
  }
  // values past the row are zero: act(0) = 0 for every activation
  float sum = 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (NORM) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sum = fmaf(v[e][i], v[e][i], sum);
        v[e][i] *= w[e][i];
      }
    }
    if constexpr (sizeof(OutT) == 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) top = max(top, mag(v[e][i]));
    }
  }
  // two factors, not their product: with a tiny scale the product overflows
  float k = 1.0f, inv = 1.0f;
  if constexpr (NORM || sizeof(OutT) == 1) {
    row_reduce<G>(sum, top);
    if constexpr (NORM) k = 1.0f / sqrtf(sum / (float)width + args.eps);
    if constexpr (sizeof(OutT) == 1) {
      const float s = f8_scale(__uint_as_float(top) * k);
      if (t == 0) args.scale[row] = s;
      inv = 1.0f / s;
    }
  }
  OutT* y = (OutT*)args.y + row * args.ldy;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (t + e * G) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (NORM) v[e][i] *= k;
      if constexpr (sizeof(OutT) == 1) v[e][i] *= inv;
    }
    store_row<V>(y + c, width - c, v[e]);
  }
}

template <typename T, typename OutT, int G, int E, bool NORM>
static p24_status launch_rows(const RowArgs& a, hipStream_t st) {
  constexpr int R = ROW_BLOCK<G> / G;
  hipLaunchKernelGGL((k_rows<T, OutT, G, E, NORM>), dim3((unsigned)(((int64_t)a.rows + R - 1) / R)), dim3(ROW_BLOCK<G>), 0, st, a);
  return launch_status();
}

// Threads and chunks of a row, by its count of 16-byte chunks: as few chunks a
// thread as a block of 512 or 1024 allows, because a row's time is its trips to
// memory and the reduction.  Measured, us (bf16 unless said):
//   norm 8192 x 8192   512 x 2 89.4 (5.3 TB/s), 256 x 4 100.7, 1024 x 1 89.2
//   gate 4096 x 8192   512 x 2 31.6 (5.3 TB/s), 256 x 4 35.8, 1024 x 1 34.5
//   norm 4096 x 4096 fp32   1024 x 1 39.8, 512 x 2 41.9;  gate 777 x 2051 fp32  6.0, 6.5
//   gate 2000 x 4096   512 x 1 9.6, 256 x 2 10.2;  norm 1 x 4096  3.3, 3.5
//   norm 8192 x 1024   64 x 2 12.4, 128 x 1 13.8, 256 x 1 15.7;  norm 2 x 700  128 x 1 3.8, 64 x 2 4.3
template <typename T, typename OutT, bool NORM>
static p24_status rows_by_width(const RowArgs& a, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int chunks = (a.width + V - 1) / V;
  if (chunks <= 16) return launch_rows<T, OutT, 16, 1, NORM>(a, st);
  if (chunks <= 32) return launch_rows<T, OutT, 32, 1, NORM>(a, st);
  if (chunks <= 64) return launch_rows<T, OutT, 64, 1, NORM>(a, st);
  if (chunks <= 128) {
    if (a.rows >= 1024) return launch_rows<T, OutT, 64, 2, NORM>(a, st);   // four rows a block, no barrier
    return launch_rows<T, OutT, 128, 1, NORM>(a, st);
  }
  if (chunks <= 256) return launch_rows<T, OutT, 256, 1, NORM>(a, st);
  if (chunks <= 512) return launch_rows<T, OutT, 512, 1, NORM>(a, st);
  if (chunks <= 1024) {
    if constexpr (sizeof(T) == 4) return launch_rows<T, OutT, 1024, 1, NORM>(a, st);
    else return launch_rows<T, OutT, 512, 2, NORM>(a, st);
  }
  if (chunks <= 2048) return launch_rows<T, OutT, 1024, 2, NORM>(a, st);
  if (chunks <= 4096) return launch_rows<T, OutT, 1024, 4, NORM>(a, st);
  if (chunks <= 8192) return launch_rows<T, OutT, 1024, 8, NORM>(a, st);
  if constexpr (sizeof(T) == 4) return launch_rows<T, OutT, 1024, 16, NORM>(a, st);
  else return P24_ERR_SHAPE;
}

template <bool NORM>
static p24_status rows_by_type(const RowArgs& a, int32_t x_dtype, int32_t y_dtype, hipStream_t st) {
  if (x_dtype == P24_F32) {
    if (y_dtype == P24_F8) return rows_by_width<float, f8_t, NORM>(a, st);
    if (y_dtype == P24_F32) return rows_by_width<float, float, NORM>(a, st);
    return rows_by_width<float, uint16_t, NORM>(a, st);
  }
  if (y_dtype == P24_F8) return rows_by_width<uint16_t, f8_t, NORM>(a, st);
  if (y_dtype == P24_F32) return rows_by_width<uint16_t, float, NORM>(a, st);
  return rows_by_width<uint16_t, uint16_t, NORM>(a, st);
}

static size_t elem_bytes(int32_t dtype) { return dtype == P24_F32 ? 4 : dtype == P24_BF16 ? 2 : 1; }

// What the two entry points check alike.  P24_OK with tokens == 0 means a no-op.
static p24_status check_rows(const void* a, int32_t x_dtype, int64_t lda, const void* b, int64_t ldb, int64_t tokens,
                             int64_t width, const void* y, int32_t y_dtype, int64_t ldy, const float* scale) {
  if (x_dtype != P24_F32 && x_dtype != P24_BF16) return P24_ERR_DTYPE;
  if (y_dtype != P24_F32 && y_dtype != P24_BF16 && y_dtype != P24_F8) return P24_ERR_DTYPE;
  if (tokens < 0 || tokens > INT32_MAX || width < 1 || width > P24_ROW_MAX) return P24_ERR_SHAPE;
  if (lda < width || ldy < width || (b && ldb < width)) return P24_ERR_SHAPE;
  if (tokens >= 1 << 22) return P24_ERR_UNSUPPORTED;   // 1024 threads a row, fewer than 2^32 in a grid
  if (tokens == 0) return P24_OK;
  if (!a || !y || (y_dtype == P24_F8 && !scale)) return P24_ERR_NULL;
  const size_t xe = elem_bytes(x_dtype);
  if (!aligned(a, xe) || (b && !aligned(b, xe)) || !aligned(y, elem_bytes(y_dtype))) return P24_ERR_ALIGN;
  if (scale && !aligned(scale, 4)) return P24_ERR_ALIGN;
  return P24_OK;
}

}  // namespace p24

using namespace p24;

extern "C" P24_API p24_status rms_norm(const void* x, int32_t x_dtype, int64_t ldx, const void* residual, int64_t ldr,
                                       const float* weight, float eps, int64_t tokens, int64_t width, void* h,
                                       int64_t ldh, void* y, int32_t y_dtype, int64_t ldy, float* scale,
                                       void* stream) {
  const p24_status s = check_rows(x, x_dtype, ldx, residual, ldr, tokens, width, y, y_dtype, ldy, scale);
  if (s != P24_OK) return s;
  if (!(eps >= 0.0f) || eps > 3.4028235e38f) return P24_ERR_SHAPE;
  if (residual && ldh < width) return P24_ERR_SHAPE;
  if (tokens == 0) return P24_OK;
  if (!weight || (residual && !h)) return P24_ERR_NULL;
  if (!residual && h) return P24_ERR_UNSUPPORTED;
  if (!aligned(weight, 4) || (h && !aligned(h, elem_bytes(x_dtype)))) return P24_ERR_ALIGN;
  RowArgs a{};
  a.a = x;
  a.b = residual;
  a.weight = weight;
  a.h = h;
  a.y = y;
  a.scale = scale;
  a.lda = ldx;
  a.ldb = ldr;
  a.ldh = ldh;
  a.ldy = ldy;
  a.rows = (int)tokens;
  a.width = (int)width;
  a.eps = eps;
  return rows_by_type<true>(a, x_dtype, y_dtype, (hipStream_t)stream);
}

extern "C" P24_API p24_status gated_act(const void* gate, int32_t x_dtype, int64_t ldg, const void* up, int64_t ldu,
                                        int32_t act, int64_t tokens, int64_t width, void* y, int32_t y_dtype,
                                        int64_t ldy, float* scale, void* stream) {
  if (!f8_act_known(act)) return P24_ERR_UNSUPPORTED;
  const p24_status s = check_rows(gate, x_dtype, ldg, up, ldu, tokens, width, y, y_dtype, ldy, scale);
  if (s != P24_OK || tokens == 0) return s;
  RowArgs a{};
  a.a = gate;
  a.b = up;
  a.y = y;
  a.scale = scale;
  a.lda = ldg;
  a.ldb = ldu;
  a.ldy = ldy;
  a.rows = (int)tokens;
  a.width = (int)width;
  a.act = act;
  return rows_by_type<false>(a, x_dtype, y_dtype, (hipStream_t)stream);
}
