/*
 * prune24_f8.h -- C ABI of libprune24.so, 8-bit feed-forward operators: RMS
 * norm with the residual's addition, gated activation, and the 2:4-sparse
 * product of 8-bit weights and 8-bit activations with a fused epilogue.
 *
 * Together they are one feed-forward layer of a language model whose pruned
 * weights and whose activations are held in 8 bits:
 *     xq, h = rms_norm(x + residual)      8-bit rows for the first product
 *     gu    = W_gate_up xq                2:4-sparse, bf16 out
 *     aq    = silu(gate) * up             8-bit rows for the second product
 *     y     = W_down aq + h               2:4-sparse, residual in the epilogue
 *
 * Conventions beyond those of prune24.h (device pointers, caller-owned
 * buffers, stream order, status codes, nothing allocated, stateless)
 *   - Activations are tokens x features, row-major, features contiguous.
 *   - 8-bit values are OCP e4m3 (no infinities, largest finite 448).  A row y
 *     is held as q = e4m3(y / s) with one fp32 scale
 *         s = max(max|y| / 448, 2^-126)
 *     per token (activations) or per output feature (weights), rounded to
 *     nearest even; y is about q s.  A NaN in a row makes its scale and all
 *     its values NaN; an infinity makes the scale infinite, the infinite
 *     entries NaN and the finite ones 0.
 *   - Statistics, sums and activations are computed in fp32; the squares of a
 *     norm's row that would leave its range are scaled by a power of two.
 *   - GELU's smooth factor is a polynomial.  For P24_F32 outputs its fit is within
 *     3.3e-8, and the result within (1.5 z^2 + 40) 2^-24 of itself (the roundings
 *     of z^2 in the exponent); for P24_BF16 and P24_F8 outputs the fit is within
 *     1.8e-5, below their rounding of 2^-9 and 2^-4 -- but not below that of a sum
 *     with a residual that cancels it.
 *   - Results are deterministic: no atomics, fixed summation order.
 */
#ifndef PRUNE24_F8_H
#define PRUNE24_F8_H

#include "prune24.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { P24_F8 = 2 };          /* element dtype: e4m3, next to P24_F32 and P24_BF16 */
enum { P24_ACT_SILU = 3 };    /* z / (1 + exp(-z)), next to P24_ACT_NONE, _RELU, _GELU */

/* Widest row of rms_norm and gated_act. */
#define P24_ROW_MAX 65536

/*
 * rms_norm -- per token t (row of `width` values):
 *     h = x + residual   (h = x without a residual)
 *     y = h / sqrt(mean(h^2) + eps) * weight
 *   x         tokens x width, x_dtype P24_F32 or P24_BF16, leading dimension
 *             ldx >= width, naturally aligned (any leading dimension).
 *   residual  as x, leading dimension ldr, or NULL.
 *   weight    width fp32 values, 4 B aligned.
 *   h         output, x_dtype, leading dimension ldh: the sum rounded to
 *             x_dtype (the next layer's residual).  Required with a residual,
 *             NULL without one.  h may be x or residual itself (same pointer
 *             and leading dimension); y is computed from the unrounded sum.
 *   y         output, y_dtype P24_F8, P24_BF16 or P24_F32, leading dimension ldy.
 *   scale     output, one fp32 per token, with P24_F8; NULL otherwise.
 *   y and scale overlap no input and not h.
 *   1 <= width <= P24_ROW_MAX; tokens < 2^22 (else
 *   P24_ERR_UNSUPPORTED); tokens == 0 is a no-op.
 *   eps >= 0 and finite.
 */
P24_API p24_status rms_norm(const void* x, int32_t x_dtype, int64_t ldx, const void* residual,
                            int64_t ldr, const float* weight, float eps, int64_t tokens,
                            int64_t width, void* h, int64_t ldh, void* y, int32_t y_dtype,
                            int64_t ldy, float* scale, void* stream);

/*
 * gated_act -- a = act(gate) * up per element (act(gate) without `up`).
 *   gate, up  tokens x width, x_dtype P24_F32 or P24_BF16, leading dimensions
 *             ldg, ldu; `up` may be NULL.  The two are usually halves of one
 *             product's output rows.
 *   act       P24_ACT_NONE, _RELU (z > 0 ? z : 0, and NaN for NaN), _GELU
 *             (z/2 erfc(-z / sqrt 2)) or _SILU.
 *   y, scale  as for rms_norm.  With act P24_ACT_NONE, no `up` and P24_F8 the
 *             call is the plain row quantization.
 */
P24_API p24_status gated_act(const void* gate, int32_t x_dtype, int64_t ldg, const void* up,
                             int64_t ldu, int32_t act, int64_t tokens, int64_t width, void* y,
                             int32_t y_dtype, int64_t ldy, float* scale, void* stream);

/*
 * 8-bit 2:4-compressed weights.
 * prune24_f8_bytes -- bytes of the compressed M x K matrix (0 for an invalid
 *   request: negative, or K % 64 != 0).
 * prune24_compress_f8 -- magnitude 2:4 selection of W's rows (the rule of
 *   prune24_compress), then the kept values as 8-bit rows.
 *   W         M x K, P24_F32 or P24_BF16, leading dimension ldw >= K,
 *             naturally aligned; K % 64 == 0; M < 2^24 and fewer than 2^26
 *             blocks of 32 x 64 (else P24_ERR_UNSUPPORTED).
 *   data      output, prune24_f8_bytes(M, K) bytes, 16 B aligned.
 *   scale     output, M fp32 values: the rows' scales.
 * prune24_decompress_f8 -- W_out[m][k] = q s at the kept positions, +0
 *   elsewhere; fp32, leading dimension ldo >= K.
 *
 * Layout of `data` (operand order of v_smfmac_f32_32x32x64_fp8_fp8): row
 * groups of 128, K padded to a multiple of 128; for row group g and 64-k block
 * s one 5 KiB piece at ((g * 2 ceil(K/128)) + s) * 5120: four 1 KiB blocks of
 * values (rows 128 g + 32 b + [0, 32), b = 0..3), then four 256 B blocks of
 * positions.  Lane L of a value block holds row L % 32, the 16 kept values of
 * k = 64 s + 32 (L / 32) + [0, 32) in ascending order; lane L's position word
 * holds their positions inside their groups of four, 2 bits each.  Padding
 * holds zero values and positions 0, 1.
 */
P24_API size_t prune24_f8_bytes(int64_t M, int64_t K);
P24_API p24_status prune24_compress_f8(const void* W, int32_t w_dtype, int64_t M, int64_t K,
                                       int64_t ldw, void* data, float* scale, void* stream);
P24_API p24_status prune24_decompress_f8(const void* data, const float* scale, int64_t M, int64_t K,
                                         float* W_out, int64_t ldo, void* stream);

/*
 * spmm24_f8 -- for tokens n and output features m:
 *     Y[n][m] = act(w_scale[m] x_scale[n] sum_k W[m][k] X[n][k] + bias[m])
 *               + residual[n][m]
 *   (the sum times x_scale, then times w_scale, in every kernel).
 *   data, w_scale   the compressed M x K weight; K % 64 == 0, K > 0.
 *   X         N x K e4m3, 16 B aligned, leading dimension ldx >= K; with more
 *             than one token ldx % 16 == 0 and 512 * ldx < 2^32.
 *             N <= 65535 * 32; M, K < 2^24 (else P24_ERR_UNSUPPORTED).
 *   x_scale   N fp32 values.
 *   Y         N x M, P24_F32 or P24_BF16 (round to nearest even), leading
 *             dimension ldy >= M, naturally aligned.
 *   bias      M fp32 values, or NULL.
 *   act       P24_ACT_NONE, _RELU, _GELU or _SILU (as for gated_act).
 *   residual  as Y, leading dimension ldr, or NULL.  It may be Y itself (same
 *             pointer and leading dimension); otherwise Y overlaps no input.
 * The kernel is picked from the shape.  The environment variable
 * P24_F8_TILE=tokens|64x32|64x64|128x64|128x128|256x128|256x192|256x256, read at
 * each call, forces one (a measurement and test aid; results stay within the
 * same bounds; the last two run as 256x128 for a P24_F32 output).
 * Sums.  For a P24_F32 output every product is exact and every sum fp32.  For
 * a P24_BF16 output the 8-bit matrix unit adds eight products at a time, each
 * cut toward zero to 2^-13 of the exponent of the largest of the eight, and
 * those sums in fp32: an error of at most 7 * 2^-13 of the largest product of each
 * eight.  Measured on Gaussian rows (K 512 to 8192) it is 8e-6 of a typical
 * output and 4e-5 at most, which shows where the sum cancels: 0.7 % of all
 * outputs are more than half a bf16 step off, 0.05 % more than two steps.  A
 * P24_F32 output avoids it.
 */
P24_API p24_status spmm24_f8(const void* data, const float* w_scale, int64_t M, int64_t K,
                             const void* X, int64_t ldx, const float* x_scale, int64_t N, void* Y,
                             int32_t y_dtype, int64_t ldy, const float* bias, int32_t act,
                             const void* residual, int64_t ldr, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PRUNE24_F8_H */
