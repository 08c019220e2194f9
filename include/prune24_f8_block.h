/*
 * prune24_f8_block.h -- C ABI of libprune24.so, the dense 8-bit product with a
 * scale for each block of 128: for the layers of a pruned model that stay dense.
 *     aq = act(x) * up                    8-bit values, a scale per token and 128 features
 *     y  = W aq + residual                dense, a scale per 128 x 128 weights
 *
 * The conventions of prune24.h and prune24_f8.h hold: activations are tokens x
 * features, 8-bit values are e4m3, and a block y is held as q = e4m3(y / s) with
 * one fp32 scale s = max(max|y| / 448, 2^-126); y / s is the correctly rounded
 * quotient.  A NaN makes its block's scale and values NaN; an infinity makes the
 * scale infinite, the infinite values NaN and the finite ones 0.  Inference only:
 * no gradients.
 */
#ifndef PRUNE24_F8_BLOCK_H
#define PRUNE24_F8_BLOCK_H

#include "prune24_f8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * quantize_f8_block -- a = act(x) * up per element (act(x) without `up`), as 8-bit
 * values with a scale per token and 128 features (the last block of a row may be a
 * part).
 *   x, up     tokens x width, x_dtype P24_F32 or P24_BF16, leading dimensions ldx,
 *             ldu >= width, naturally aligned; `up` may be NULL.
 *   act       as for gated_act; P24_ACT_NONE without `up` is the plain quantisation.
 *   values    output, tokens x width e4m3, leading dimension ldv >= width.
 *   scale     output, ceil(width / 128) x tokens fp32: scale[b][t] at
 *             b * lds + t, lds >= tokens, 4 B aligned.
 *   The outputs overlap no input.  1 <= width < 2^24, tokens <= 65535 * 16 (else
 *   P24_ERR_UNSUPPORTED); tokens == 0 is a no-op.
 */
P24_API p24_status quantize_f8_block(const void* x, int32_t x_dtype, int64_t ldx, const void* up,
                                     int64_t ldu, int32_t act, int64_t tokens, int64_t width,
                                     void* values, int64_t ldv, float* scale, int64_t lds,
                                     void* stream);

/*
 * quantize_weight_f8_block -- W (M x K) as 8-bit values with a scale per 128 x 128
 * block (those at the last rows and columns may be parts).
 *   W         M x K, P24_F32 or P24_BF16, leading dimension ldw >= K, naturally aligned.
 *   values    output, M x K e4m3, leading dimension ldv >= K.
 *   scale     output, ceil(M / 128) x ceil(K / 128) fp32, row-major.
 *   M, K < 2^22 (else P24_ERR_UNSUPPORTED); M == 0 or K == 0 is a no-op.
 */
P24_API p24_status quantize_weight_f8_block(const void* W, int32_t w_dtype, int64_t M, int64_t K,
                                            int64_t ldw, void* values, int64_t ldv, float* scale,
                                            void* stream);

/*
 * gemm_f8_block -- for tokens n and output features m:
 *     Y[n][m] = act(sum_b x_scale[b][n] w_scale[m / 128][b] S_b + bias[m]) + residual[n][m]
 *     S_b     = sum of X[n][k] W[m][k] over the k of block b (128 b to 128 b + 127)
 *   W         M x K e4m3, leading dimension ldw >= K.
 *   w_scale   ceil(M / 128) x ceil(K / 128) fp32, row-major.
 *   X         N x K e4m3, leading dimension ldx >= K.
 *   x_scale   ceil(K / 128) x N fp32, leading dimension ldxs >= N.
 *   W and X are 16 B aligned, ldw and ldx multiples of 16, and so is K (else
 *   P24_ERR_UNSUPPORTED); 512 * ldw, 512 * ldx and 4 ceil(K / 128) (ldxs + 1) are
 *   below 2^32, M and K below 2^24, N <= 65535 * 16 (else P24_ERR_UNSUPPORTED).
 *   Y         N x M, P24_F32 or P24_BF16 (round to nearest even), leading
 *             dimension ldy >= M, naturally aligned.
 *   bias, act, residual   as for spmm24_f8.
 * Sums.  Every S_b is scaled on its own in fp32, by the product of its two scales
 * rounded to fp32 (past its range S_b's part is infinite, or NaN where S_b is 0;
 * under 2^-126 it has the bits of a subnormal), and they are added in fp32 in a
 * fixed order.  For a P24_F32 output the products of S_b are exact and
 * its sum fp32.  For a P24_BF16 output the 8-bit matrix unit forms S_b, adding
 * eight products at a time, each cut toward zero to 2^-13 of the exponent of the
 * largest of the eight: an error of at most 7 * 2^-13 of the largest product of
 * each eight, on Gaussian rows (K 128 to 4096) 1.4e-5 of a typical output and
 * 1.5e-4 at most.
 * P24_F8_TILE=tokens|64x32|64x64|128x64|128x128|256x128|256x256, read at each
 * call, forces a kernel (a measurement and test aid; the last two run as 128x128
 * for a P24_F32 output).
 */
P24_API p24_status gemm_f8_block(const void* W, int64_t ldw, const float* w_scale, int64_t M, int64_t K,
                                 const void* X, int64_t ldx, const float* x_scale, int64_t ldxs,
                                 int64_t N, void* Y, int32_t y_dtype, int64_t ldy, const float* bias,
                                 int32_t act, const void* residual, int64_t ldr, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PRUNE24_F8_BLOCK_H */
