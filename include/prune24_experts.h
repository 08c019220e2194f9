/*
 * prune24_experts.h -- C ABI of libprune24.so, the operators of a feed-forward
 * layer of experts on 8-bit 2:4-sparse weights: routing, products grouped by
 * expert with ragged sizes, and the combination of a token's experts:
 *     plan  = route(logits, k)                  experts, weights, rows sorted by expert
 *     gu    = W_gate_up[e] xq                   2:4-sparse, rows gathered by token
 *     aq    = silu(gate) * up                   gated_act, 8-bit rows
 *     z     = W_down[e] aq                      2:4-sparse
 *     y     = sum of a token's rows * weights + residual
 *
 * The conventions of prune24.h and prune24_f8.h hold.  How many rows an expert
 * has is known on the device only: no call reads it back, so a layer can be
 * captured in a graph and replayed with other logits.  Inference only: no
 * gradients.
 */
#ifndef PRUNE24_EXPERTS_H
#define PRUNE24_EXPERTS_H

#include "prune24_f8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define P24_EXPERTS_MAX 1024      /* experts of a layer */
#define P24_EXPERTS_K_MAX 32      /* experts of a token */

enum { P24_SCORE_SOFTMAX = 0, P24_SCORE_SIGMOID = 1 };

/*
 * experts_route -- each token's k best experts, their weights, and the plan of
 * its rows: every chosen (token, expert) is a row, rows sorted by expert, those
 * of an expert in the order of the tokens.
 *   logits    T x E, l_dtype P24_F32 or P24_BF16, leading dimension ldl >= E,
 *             naturally aligned.  An expert whose logit is -inf is not open to the
 *             token: a padded token is a row of -inf.
 *   score     what the experts are ranked by: P24_SCORE_SOFTMAX the logit,
 *             P24_SCORE_SIGMOID the logit without a bias, with one
 *             1 / (1 + exp(-logit)) + bias in 64 bits.  NaN ranks above +inf, -0 and
 *             +0 tie; ties go to the lower expert.
 *   bias      E fp32 values with P24_SCORE_SIGMOID, or NULL.
 *   normalize softmax: weights exp(l - max) over their sum, of the chosen experts
 *             (1) or of all (0).  sigmoid: the sigmoids (without the bias), over
 *             their sum (1) or as they are (0).  Then times `scale` (finite).
 *             Computed in fp32; quotients of sigmoids that leave it are those of
 *             the sigmoids themselves.  A NaN logit, or +inf under softmax, gives
 *             the NaN that the formula gives, and so do normalized sigmoids whose
 *             largest logit lies below -709.78, 0 / 0 in 64 bits too (the lowest
 *             value of a type is no mask for them: -inf is).
 *   experts   T x k int32: the chosen experts, best first; -1 past the open ones.
 *   weights   T x k fp32; 0 where there is no expert.
 *   offsets   E + 1 int32: expert e's rows are [offsets[e], offsets[e + 1]).
 *   tokens    T k int32: the token of each row; -1 from offsets[E] on.
 *   positions T x k int32: the row of a token's slot; -1 where there is no expert.
 *   ws        experts_route_workspace(T, E) bytes (0 up to 64 tokens), 4 B aligned;
 *             its contents need no preparation and mean nothing afterwards.  Calls
 *             that may overlap need one each.
 *   1 <= k <= min(E, P24_EXPERTS_K_MAX), E <= P24_EXPERTS_MAX, T <= 2^18 (else
 *   P24_ERR_UNSUPPORTED).  T == 0 sets offsets to 0.  The outputs overlap no input
 *   and not each other.
 */
P24_API size_t experts_route_workspace(int64_t T, int64_t E);
P24_API p24_status experts_route(const void* logits, int32_t l_dtype, int64_t ldl, int64_t T, int64_t E,
                                 int64_t k, int32_t score, const float* bias, int32_t normalize,
                                 float scale, int32_t* experts, float* weights, int32_t* offsets,
                                 int32_t* tokens, int32_t* positions, void* ws, size_t ws_bytes,
                                 void* stream);

/*
 * spmm24_f8_grouped -- spmm24_f8 for E weights of the same shape, each with rows
 * of its own.  For expert e and its rows p in [offsets[e], offsets[e + 1]):
 *     Y[p][m] = act(w_scale[e][m] x_scale[r] sum_k W[e][m][k] X[r][k] + bias[e][m])
 *   with r = tokens[p], or p without `tokens`.
 *   data      the experts' compressed weights one after the other, each
 *             prune24_f8_bytes(M, K) bytes; w_scale E x M.
 *   X         x_rows x K e4m3, leading dimension ldx, as for spmm24_f8; with
 *             `tokens` x_rows * ldx < 2^32.  Without it x_rows is `rows`.
 *   offsets   E + 1 int32 on the device, not falling, offsets[0] >= 0.  Offsets past
 *             `rows` are taken as `rows`: nothing is read or written outside.  Where
 *             they fall, which rows are written is not said, but none outside Y.
 *   tokens    rows int32, or NULL.  A value outside [0, x_rows) in an expert's
 *             range reads the last row of X.
 *   Y         rows x M as for spmm24_f8.  Rows outside every expert's range, those
 *             from offsets[E] on among them, are left as they were.
 *   bias      E x M fp32, or NULL.  act as for spmm24_f8.
 *   1 <= E <= P24_EXPERTS_MAX; rows, M and K as N, M and K of spmm24_f8: at most
 *   65535 * 32 rows (the T k of a routing), else P24_ERR_UNSUPPORTED.
 * Sums are those of spmm24_f8: exact products and fp32 sums for P24_F32 outputs,
 * the 8-bit matrix unit's for P24_BF16.  P24_F8_TILE forces a kernel, as there.
 */
P24_API p24_status spmm24_f8_grouped(const void* data, const float* w_scale, int64_t E, int64_t M,
                                     int64_t K, const void* X, int64_t ldx, const float* x_scale,
                                     int64_t x_rows, const int32_t* offsets, const int32_t* tokens,
                                     int64_t rows, void* Y, int32_t y_dtype, int64_t ldy,
                                     const float* bias, int32_t act, void* stream);

/*
 * experts_combine -- y[t] = residual[t] + sum_j weights[t][j] Z[positions[t][j]],
 * in fp32: the products j ascending, each rounded into the sum once, then the
 * residual; rounded to y_dtype.
 *   Z         rows x width, z_dtype P24_F32 or P24_BF16, leading dimension ldz >= width,
 *             naturally aligned.
 *   positions T x k int32, weights T x k fp32.  A slot whose position lies outside
 *             [0, rows) adds nothing, whatever its weight.
 *   residual  T x width, y_dtype, leading dimension ldr, or NULL.  It may be y itself
 *             (same pointer and leading dimension); otherwise y overlaps no input.
 *   y         T x width, P24_F32 or P24_BF16, leading dimension ldy >= width.
 *   1 <= k <= P24_EXPERTS_K_MAX, 1 <= width <= P24_ROW_MAX, T < 2^22, rows < 2^31.
 */
P24_API p24_status experts_combine(const void* Z, int32_t z_dtype, int64_t ldz, int64_t rows,
                                   const int32_t* positions, const float* weights, int64_t T, int64_t k,
                                   int64_t width, const void* residual, int64_t ldr, void* y,
                                   int32_t y_dtype, int64_t ldy, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PRUNE24_EXPERTS_H */
