// Device-side building blocks of the 8-bit feed-forward operators (gfx950 only).
#pragma once

#include "p24_device.hpp"
#include "p24_f8_tile.hpp"
#include "../../include/prune24_f8.h"

namespace p24 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr float F8_MAX = 448.0f;
constexpr float F32_TINY = 1.17549435e-38f;   // 2^-126

// Vectors loaded and stored at any element alignment: rows of an odd leading
// dimension start anywhere, and global memory takes such accesses whole.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

// Row storage types: fp32, bf16 bits, e4m3 bits.
struct f8_t {
  uint8_t v;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// two fp32 -> packed bf16, round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
// four fp32 -> packed e4m3, round to nearest even; |v| <= 448 up to rounding, or NaN
__device__ __forceinline__ uint32_t pack_f8(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// NaN-propagating magnitude maximum: on the bits with the sign cleared NaN
// ranks above infinity.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Row scale of a magnitude maximum (NaN stays NaN).
__device__ __forceinline__ float f8_scale(float amax) {
  const float s = amax / F8_MAX;
  return s < F32_TINY ? F32_TINY : s;
}

// GELU z/2 erfc(-z / sqrt 2) in fp32.  With x = |z| / sqrt 2 and
// erfc(x) = erfcx(x) exp(-x^2), the smooth factor erfcx / 2 is t Q(t) with
// t = 1 / (1 + p x), Q a least-squares fit at Chebyshev nodes reweighted to an even
// relative error; the negative side has no cancellation.  For fp32 outputs
// p = 0.45 and degree 9, fit within 3.3e-8; for bf16 and 8-bit ones, rounded by 2^-8 and
// 2^-4 at most, p = 0.46 and degree 5, fit within 1.8e-5: an epilogue with little K under
// it is bound by these instructions (3106 x 128 with 7981 tokens 43.5 -> 36.8 us).
// Beside the fit count the reciprocal and exp2 (one ulp each) and the rounding of
// z^2 in the exponent: (1.5 z^2 + 40) 2^-24 of the result.
template <bool F32>
__device__ __forceinline__ float gelu_erfc(float z) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), F32 ? 0.3181980515339464f : 0.3252691193458121f, 1.0f));
  float q;
  if constexpr (F32) {
    q = fmaf(-0.02069577232116633f, t, 0.09534486297670204f);
    q = fmaf(q, t, -0.1502928110955076f);
    q = fmaf(q, t, 0.07120189653123436f);
    q = fmaf(q, t, -0.011179689575678579f);
    q = fmaf(q, t, 0.05997542432208766f);
    q = fmaf(q, t, 0.08762603125038634f);
    q = fmaf(q, t, 0.11413582334817399f);
    q = fmaf(q, t, 0.12694158134658862f);
    q = fmaf(q, t, 0.12694266037563537f);
  } else {
    q = fmaf(-0.06317690894011742f, t, 0.12090257661401217f);
    q = fmaf(q, t, 0.06272410890294544f);
    q = fmaf(q, t, 0.12026239948686118f);
    q = fmaf(q, t, 0.12951712403373283f);
    q = fmaf(q, t, 0.12976586047574853f);
  }
  q *= t * __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
  return z * (z >= 0.0f ? 1.0f - q : q);
}

// The activations of the 8-bit operators, over N values at a time: one uniform
// branch, then straight code.  F32: for an fp32 output.  -inf gives NaN under SiLU and GELU (infinity times
// zero), as their formulas do.
__device__ __forceinline__ float silu_f32(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}
template <bool F32, int N>
__device__ __forceinline__ void f8_act(float (&z)[N], int act) {
  if (act == P24_ACT_NONE) return;
  if (act == P24_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = silu_f32(z[i]);
  } else if (act == P24_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = gelu_erfc<F32>(z[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];   // NaN stays NaN
  }
}

// V consecutive values from p, of which [first, left) lie inside the row (the
// others read as zero).  Any element alignment.  A part of a chunk is loaded value
// by value at clamped places, all on the way at once.
template <int V, typename T>
__device__ __forceinline__ void load_row(const T* p, int left, float (&v)[V], int first = 0) {
  static_assert(V % 4 == 0 && (sizeof(T) == 4 || V == 8 || V == 4), "whole vectors");
  if (first <= 0 && left >= V) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[V / 2];
      if constexpr (V == 8) {
        const u32x4 x = *reinterpret_cast<const u32x4_a2*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = x[i];
      } else {
        const u32x2 x = *reinterpret_cast<const u32x2_a2*>(p);
        w[0] = x[0];
        w[1] = x[1];
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const u32x4 x = *reinterpret_cast<const u32x4_a4*>(p + 4 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * q + i] = __uint_as_float(x[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    if (left > 0 && first < V) {
      T x[V];
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = p[min(max(i, first), left - 1)];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f;
        if constexpr (sizeof(T) == 2) f = __uint_as_float((uint32_t)x[i] << 16);
        else f = x[i];
        v[i] = i >= first && i < left ? f : 0.0f;
      }
    }
  }
}

// Buffer over [base, base + bytes): loads past it return zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t f8_rsrc(const uint8_t* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, (int)bytes, 0x00020000);
}
// 16 bytes per lane to the buffer at voff, past the L2 (nt).  Only as a buffer
// store: the compiler merges a non-temporal store through a pointer with the plain
// one of the other branch.
__device__ __forceinline__ void stream_16b(__amdgpu_buffer_rsrc_t r, u32x4 v, uint32_t voff) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, voff, 0, 2);
}

// V consecutive values to p, rounded to nearest even, [first, left) of them inside the row.
template <int V, typename T>
__device__ __forceinline__ void store_row(T* p, int left, const float (&v)[V], int first = 0) {
  if constexpr (sizeof(T) == 4) {
    if (first <= 0 && left >= V) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[4 * q + i]);
        *reinterpret_cast<u32x4_a4*>(p + 4 * q) = w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i >= first && i < left) p[i] = v[i];
    }
  } else {
    constexpr int PER = 4 / sizeof(T), W = V / PER;    // values per word, words
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (sizeof(T) == 1) w[i] = pack_f8(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      else w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
    if (first <= 0 && left >= V) {
      if constexpr (W == 4) *reinterpret_cast<u32x4_a2*>(p) = (u32x4){w[0], w[1], w[2], w[3]};
      else if constexpr (W == 2) *reinterpret_cast<u32x2_a1*>(p) = (u32x2){w[0], w[1]};
      else *reinterpret_cast<u32_a1*>(p) = w[0];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i >= first && i < left) {
          const uint32_t x = w[i / PER] >> (8 * sizeof(T) * (i % PER));
          if constexpr (sizeof(T) == 1) p[i].v = (uint8_t)x;
          else p[i] = (uint16_t)x;
        }
    }
  }
}

static inline bool f8_act_known(int32_t act) {
  return act == P24_ACT_NONE || act == P24_ACT_RELU || act == P24_ACT_GELU || act == P24_ACT_SILU;
}

}  // namespace p24
