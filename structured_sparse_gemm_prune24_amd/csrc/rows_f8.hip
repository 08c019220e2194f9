// Row operators around the 8-bit products: RMS norm with the residual's
// addition, and the gated activation, each with an 8-bit, bf16 or fp32 output.
//
// One row (token) belongs to G threads, E <= 4 chunks of 16 input bytes each,
// held in registers from the one read to the one write: the row's statistics
// (sum of squares, largest magnitude) need the whole row before the first
// output, and a second read would cost what the first did.  Bound by HBM: the
// norm moves 7 bytes per value (bf16 in, residual, sum, 8-bit out), the gated
// activation 5.  Rows past the registers are read twice (k_rows_wide).
//
// Norm: with r = 1 / sqrt(mean(h^2) + eps), y_i = h_i r w_i, so
// max|y| = r max|h_i w_i|: the sum of squares and the maximum of |h w| come out
// of one pass and one reduction.  Where the squares leave fp32 (below, above
// about 1e19), both are taken again from h f, f a power of two:
// y = h f w / sqrt(mean (h f)^2 + eps f^2).
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
  int stream;           // h's rows are whole cache lines
  int64_t ref, ldref;   // place of row 0 of the tensor whose chunks are aligned, in elements, and its leading dimension
  int shift;            // bf16 rows off the 16-byte grid: chunks start on it, the first and last are parts
  int rows, width;
  float eps;
  int threads;          // of a block, where a row has one to itself
  int act;
};

// Sum and magnitude maximum over the threads of a row, the same in each: G lanes
// of a wave, or (G = 0) the whole block.
template <int G>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top, int threads) {
#pragma unroll
  for (int o = (G ? G : 64) / 2; o > 0; o >>= 1) {
    sum += __shfl_xor(sum, o);
    const uint32_t other = __shfl_xor(top, o);
    top = top > other ? top : other;
  }
  if constexpr (G == 0) {
    constexpr int MAX_WAVES = 16;
    __shared__ __attribute__((aligned(16))) float sums[MAX_WAVES];
    __shared__ __attribute__((aligned(16))) uint32_t tops[MAX_WAVES];
    const int wave = threadIdx.x >> 6, waves = threads >> 6;
    if ((threadIdx.x & 63) == 0) {
      sums[wave] = sum;
      tops[wave] = top;
    }
    __syncthreads();
    // all entries are read at once; those past the block's waves are dropped
    float s[MAX_WAVES];
    uint32_t m[MAX_WAVES];
#pragma unroll
    for (int i = 0; i < MAX_WAVES; ++i) {
      s[i] = sums[i];
      m[i] = tops[i];
    }
    sum = 0.0f;
    top = 0;
#pragma unroll
    for (int i = 0; i < MAX_WAVES; ++i) {
      sum += i < waves ? s[i] : 0.0f;
      top = max(top, i < waves ? m[i] : 0u);
    }
  }
}

// Factor of a norm's row (or of a thread's part of it) by its sum of squares.  Large
// values overflow it, small ones lose bits that only an eps of 2^-100 or more covers.
// (A NaN takes the factor of large values and stays.)
__device__ __forceinline__ float norm_factor(float sum, float eps) {
  if (sum < 0x1p-80f && eps < 0x1p-100f) return 0x1p100f;
  return sum <= 0x1p120f ? 1.0f : 0x1p-80f;
}

// G lanes a row, several rows to a block of 256 threads; G = 0: a block a row.
template <typename T, typename OutT, int G, int E, bool NORM>
__global__ __launch_bounds__(G ? 256 : 1024) void k_rows(const RowArgs args) {
  constexpr int V = 16 / sizeof(T);   // values of a chunk: 16 bytes of input
  const int t = G ? threadIdx.x % (G ? G : 1) : threadIdx.x, threads = G ? G : args.threads;
  const int64_t row = G ? (int64_t)blockIdx.x * (256 / (G ? G : 1)) + threadIdx.x / (G ? G : 1) : blockIdx.x;
  if (row >= args.rows) return;   // whole groups of G lanes
  const int width = args.width;
  const T* a = (const T*)args.a + row * args.lda;
  const T* b = args.b ? (const T*)args.b + row * args.ldb : nullptr;

  // chunk k of the row is its values [k V - d, k V - d + V)
  int d = 0;
  if constexpr (sizeof(T) == 2)
    if (args.shift) d = (int)((args.ref + row * args.ldref) % V);

  float v[E][V], u[E][V], w[NORM ? E : 1][V];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (t + e * threads) * V - d;
    load_row<V>(a + c, width - c, v[e], -c);
    if (b) load_row<V>(b + c, width - c, u[e], -c);
  }
  // the weights are asked for ahead of the sum's store, which the compiler must keep in its place
  if constexpr (NORM) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (t + e * threads) * V - d;
      load_row<V>(args.weight + c, width - c, w[e], -c);
    }
  }
  // The sum is read again only after the layer's products: where its rows are
  // whole cache lines it streams past the L2, which keeps the 8-bit rows for the
  // product behind (norm 8192 x 8192 93.6 -> 89.7 us, 2048 x 4096 15.0 -> 13.4).
  const __amdgpu_buffer_rsrc_t h_rsrc = f8_rsrc((const uint8_t*)((const T*)args.h + row * args.ldh), (uint32_t)width * sizeof(T));
  if constexpr (!NORM) {
#pragma unroll
    for (int e = 0; e < E; ++e) f8_act<sizeof(OutT) == 4>(v[e], args.act);
  }
  if (b) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (t + e * threads) * V - d;
#pragma unroll
      for (int i = 0; i < V; ++i) v[e][i] = NORM ? v[e][i] + u[e][i] : v[e][i] * u[e][i];
      if constexpr (NORM) {
        if (args.stream && c + V <= width) {       // whole lines: d is 0
          u32x4 x;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (V == 8) x[i] = pack_bf16(v[e][2 * i], v[e][2 * i + 1]);
            else x[i] = __float_as_uint(v[e][i]);
          }
          stream_16b(h_rsrc, x, (uint32_t)c * sizeof(T));
        } else {
          store_row<V>((T*)args.h + row * args.ldh + c, width - c, v[e], -c);
        }
      }
    }
  }
  // values past the row are zero: act(0) = 0 for every activation
  float sum = 0.0f;
  uint32_t top = 0;
  float part = 0.0f, ft = 1.0f;   // this thread's squares, of h ft, with a factor of its own; v becomes h ft w
  if constexpr (NORM) {
    auto squares = [&]() {
      float p = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < V; ++i) p = fmaf(v[e][i], v[e][i], p);
      return p;
    };
    part = sum = squares();
    ft = norm_factor(sum, args.eps);
    if (__builtin_expect(ft != 1.0f, 0)) {
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < V; ++i) v[e][i] *= ft;
      part = squares();
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int i = 0; i < V; ++i) v[e][i] *= w[e][i];
  }
  if constexpr (sizeof(OutT) == 1) {
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int i = 0; i < V; ++i) top = max(top, mag(v[e][i]));
  }
  // two factors, not their product: with a tiny scale the product overflows
  float k = 1.0f, inv = 1.0f;
  if constexpr (NORM || sizeof(OutT) == 1) {
    const float own = __uint_as_float(top);
    if constexpr (NORM)
      if (__builtin_expect(ft != 1.0f, 0)) top = mag(own * (1.0f / ft));
    row_reduce<G>(sum, top, threads);
    if constexpr (NORM) {
      // The row's factor.  A thread of large values makes it theirs, and a row of small
      // ones has only such threads: where it is not this thread's, that is 1 or 2^100,
      // and undone first nothing leaves fp32 that the row's result would show.
      const float f = norm_factor(sum, args.eps), undo = 1.0f / ft;
      if (__builtin_expect(f != 1.0f, 0)) {        // the whole row
        sum = f == ft ? part : part * undo * undo * f * f;
        top = f == ft ? mag(own) : mag(own * undo * f);
        if constexpr (G == 0) __syncthreads();     // the first reduction's parts have been read
        row_reduce<G>(sum, top, threads);
      }
      if (__builtin_expect(f != ft, 0)) {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int i = 0; i < V; ++i) v[e][i] = v[e][i] * undo * f;
      }
      k = 1.0f / sqrtf(sum / (float)width + args.eps * f * f);
    }
    if constexpr (sizeof(OutT) == 1) {
      const float s = f8_scale(__uint_as_float(top) * k);
      if (t == 0) args.scale[row] = s;
      inv = 1.0f / s;
    }
  }
  OutT* y = (OutT*)args.y + row * args.ldy;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (t + e * threads) * V - d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (NORM) v[e][i] *= k;
      if constexpr (sizeof(OutT) == 1) v[e][i] *= inv;
    }
    store_row<V>(y + c, width - c, v[e], -c);
  }
}

// Rows past the registers of a block (more than 4 chunks of each of 1024 threads):
// the statistics in one pass over the row, the outputs in a second one, whose
// reads the caches serve in part.  A thread takes chunks t, t + threads, ..., U of
// them on the way at a time; its values of a row are 64 at most.  `h` may be x or
// the residual: it is written in the second pass, each chunk by the thread that has
// read it.  Nothing spills, where 8 and 17 chunks held by a thread did, us:
//   norm 4096 x 53248 bf16, 8-bit out   430 (3.6 TB/s of 7 B a value), held 882;  bf16 out 431, 1120
//   norm 512 x 65535 bf16, 8-bit out     63, held 466;  512 x 53248 fp32 86, 198
//   gate 4096 x 53248 bf16, 8-bit out   277 (3.9 TB/s of 5 B a value), held 511
template <typename T, typename OutT, bool NORM>
__global__ __launch_bounds__(1024) void k_rows_wide(const RowArgs args) {
  constexpr int V = 16 / sizeof(T), U = sizeof(T) == 2 ? 2 : 4;
  const int t = threadIdx.x, threads = args.threads, width = args.width;
  const int64_t row = blockIdx.x;
  const T* a = (const T*)args.a + row * args.lda;
  const T* b = args.b ? (const T*)args.b + row * args.ldb : nullptr;
  int d = 0;
  if constexpr (sizeof(T) == 2)
    if (args.shift) d = (int)((args.ref + row * args.ldref) % V);
  const int chunks = (width + d + V - 1) / V;

  // f(first value of the chunk, its values before the row's factors, the norm's weights)
  auto each = [&](bool weights, auto&& f) {
    for (int q0 = t; q0 < chunks; q0 += U * threads) {
      float v[U][V], u[U][V], w[NORM ? U : 1][V];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int c = (q0 + e * threads) * V - d;
        load_row<V>(a + c, width - c, v[e], -c);
        if (b) load_row<V>(b + c, width - c, u[e], -c);
      }
      if constexpr (NORM)
        if (weights) {
#pragma unroll
          for (int e = 0; e < U; ++e) {
            const int c = (q0 + e * threads) * V - d;
            load_row<V>(args.weight + c, width - c, w[e], -c);
          }
        }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        if constexpr (!NORM) f8_act<sizeof(OutT) == 4>(v[e], args.act);
        if (b) {
#pragma unroll
          for (int i = 0; i < V; ++i) v[e][i] = NORM ? v[e][i] + u[e][i] : v[e][i] * u[e][i];
        }
        f((q0 + e * threads) * V - d, v[e], w[NORM ? e : 0]);
      }
    }
  };

  float k = 1.0f, inv = 1.0f, f = 1.0f;
  if constexpr (NORM || sizeof(OutT) == 1) {
    float sum;
    uint32_t top;
    auto statistics = [&]() {
      sum = 0.0f;
      top = 0;
      each(sizeof(OutT) == 1, [&](int, float (&v)[V], float (&w)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if constexpr (NORM) v[i] *= f;
          if constexpr (NORM) sum = fmaf(v[i], v[i], sum);
          if constexpr (sizeof(OutT) == 1) top = max(top, mag(NORM ? v[i] * w[i] : v[i]));
        }
      });
      row_reduce<0>(sum, top, threads);
    };
    statistics();
    if constexpr (NORM) {
      f = norm_factor(sum, args.eps);
      if (__builtin_expect(f != 1.0f, 0)) {
        __syncthreads();
        statistics();
      }
      k = 1.0f / sqrtf(sum / (float)width + args.eps * f * f);
    }
    if constexpr (sizeof(OutT) == 1) {
      const float s = f8_scale(__uint_as_float(top) * k);
      if (t == 0) args.scale[row] = s;
      inv = 1.0f / s;
    }
  }
  OutT* y = (OutT*)args.y + row * args.ldy;
  T* h = NORM && b ? (T*)args.h + row * args.ldh : nullptr;
  each(true, [&](int c, float (&v)[V], float (&w)[V]) {
    if constexpr (NORM)
      if (h) store_row<V>(h + c, width - c, v, -c);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (NORM) v[i] = v[i] * f * w[i] * k;
      if constexpr (sizeof(OutT) == 1) v[i] *= inv;
    }
    store_row<V>(y + c, width - c, v, -c);
  });
}

template <typename T, typename OutT, int G, int E, bool NORM>
static p24_status launch_rows(RowArgs a, int chunks, hipStream_t st) {
  const int per = G ? 256 / (G ? G : 1) : 1;                                       // rows of a block
  const int threads = G ? 256 : ((chunks + E - 1) / E + 63) / 64 * 64;
  a.threads = threads;
  hipLaunchKernelGGL((k_rows<T, OutT, G, E, NORM>), dim3((unsigned)((a.rows + (int64_t)per - 1) / per)), dim3(threads), 0,
                     st, a);
  return launch_status();
}

// Threads and chunks of a row, by its count of 16-byte chunks: whole waves, as few
// chunks a thread as blocks of up to ten waves allow, because a row's time is its
// trips to memory and the reduction; several rows to a block where one needs a
// wave or less.  Measured, us (bf16 unless said):
//   norm 8192 x 8192   512 x 2 89.4 (5.3 TB/s), 256 x 4 100.7, 1024 x 1 89.2
//   gate 4096 x 8192   512 x 2 31.6 (5.3 TB/s), 256 x 4 35.8, 1024 x 1 34.5
//   gate 2000 x 4096   512 x 1 9.6, 256 x 2 10.2;  norm 1 x 4096  3.3, 3.5
//   norm 8192 x 1024   64 x 2 12.4, 128 x 1 13.8, 256 x 1 15.7;  norm 2 x 700  128 x 1 3.8, 64 x 2 4.3
//   gate 6526 x 140    32 lanes 5.1, 64 lanes 7.0;  gate 777 x 2051 fp32  576 x 1 4.9, 1024 x 1 5.7
// bf16 rows that do not all start on 16 bytes take their chunks on that grid, at
// the price of a part of a chunk at either end: loads and above all stores across
// it cost more (norm 8192 x 4095, bf16 out: 67 us, 83 on the row's own grid, 47 for
// 4096).
template <typename T, typename OutT, bool NORM>
static p24_status rows_by_width(RowArgs a, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  if constexpr (sizeof(T) == 2) {
    // the sum's rows where there is one, else the output's, else the input's
    const void* ref = NORM && a.h ? a.h : sizeof(OutT) == 2 ? a.y : a.a;
    a.ldref = NORM && a.h ? a.ldh : sizeof(OutT) == 2 ? a.ldy : a.lda;
    a.ref = (int64_t)((uintptr_t)ref / sizeof(T) % V);
    a.shift = a.ref != 0 || a.ldref % V != 0;
  }
  a.stream = NORM && a.h && aligned(a.h, 128) && a.ldh * sizeof(T) % 128 == 0;
  const int chunks = (a.width + V - 1 + (a.shift ? V - 1 : 0)) / V;
  if (chunks <= 16) return launch_rows<T, OutT, 16, 1, NORM>(a, chunks, st);
  if (chunks <= 32) return launch_rows<T, OutT, 32, 1, NORM>(a, chunks, st);
  if (chunks <= 64) return launch_rows<T, OutT, 64, 1, NORM>(a, chunks, st);
  if (chunks <= 128 && a.rows >= 1024) return launch_rows<T, OutT, 64, 2, NORM>(a, chunks, st);   // no barrier
  if (chunks <= 640 || (sizeof(T) == 4 && chunks <= 1024)) return launch_rows<T, OutT, 0, 1, NORM>(a, chunks, st);
  if (chunks <= 2048) return launch_rows<T, OutT, 0, 2, NORM>(a, chunks, st);
  if (chunks <= 4096) return launch_rows<T, OutT, 0, 4, NORM>(a, chunks, st);
  a.threads = 1024;   // 4096 chunks and more
  hipLaunchKernelGGL((k_rows_wide<T, OutT, NORM>), dim3((unsigned)a.rows), dim3(a.threads), 0, st, a);
  return launch_status();
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
