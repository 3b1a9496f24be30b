/*
 * svdq_i8.h -- C ABI of the 8-bit integer linear (W8A8) beside the 4-bit ones
 * of svdq.h, for the layers that lose too much in 4 bits:
 *
 *   Y = act(diag(sa) (qa qw^T) diag(sw) + bias)
 *
 * with one fp32 scale per token (sa) and per output channel (sw) and
 * symmetric codes in [-127, 127]:
 *   s = fl32(max|v| / 127) over the row, code = rint(fl32(v fl32(1/s))) (ties
 *   to even); s == 0, or a 1/s that is not finite, gives all-zero codes.
 * A row with a NaN or an infinity gets all-zero codes and a scale that is not
 * finite, so its outputs (a token's row, a channel's column of Y) are NaN; the
 * other rows do not change.
 * The activations may be smoothed first (v = fl32(x fl32(1/lambda)), as in
 * svdq_quantize_act_down).  The products are summed exactly in 32-bit
 * integers (K <= SVDQ_I8_MAX_K keeps every sum below 2^31).
 *
 * Conventions and status codes are those of svdq.h.  A workspace serves one
 * call at a time.
 */
#ifndef SVDQ_I8_H
#define SVDQ_I8_H

#include "svdq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SVDQ_I8_MAX_K (1 << 17) /* 127 * 127 * 2^17 < 2^31 */

/*
 * Offline weight preparation (nn.Linear orientation).
 *   W   device fp32 [N, K]
 *   qw  device int8 [N, K]  row-major codes (out)
 *   sw  device fp32 [N]     channel scales (out)
 * N >= 0 (0: no-op), K % 64 == 0, 64 <= K <= SVDQ_I8_MAX_K.  Codes and scales
 * made elsewhere are taken by the linear as they are, if no code is -128.
 */
int32_t svdq_i8_pack_weights(const float *W, int64_t N, int64_t K, int8_t *qw, float *sw,
                             void *stream);

/*
 * Activation quantization, one scale per token.
 *   X       device bf16 [M, K]
 *   lambda  device fp32 [K] smoothing factors (finite and > 0, 1/lambda finite), or
 *                              NULL: none
 *   qa      device int8 [M, K] (out)
 *   sa      device fp32 [M] (out)
 * M >= 0 (0: no-op), K as above.  Bit-exact with the definition.
 */
int32_t svdq_i8_quantize_act(const uint16_t *X, const float *lambda, int64_t M, int64_t K,
                             int8_t *qa, float *sa, void *stream);

/* Workspace of svdq_i8_gemm.  No shape needs any: 0, and `workspace` may be
 * NULL. */
size_t svdq_i8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * The product with its scales, bias and activation.
 *   qa, sa  device int8 [M, K], fp32 [M]
 *   qw, sw  device int8 [N, K], fp32 [N]   (codes in [-127, 127])
 *   bias    device bf16 [N] or NULL
 *   act     svdq_act
 *   Y       device bf16 [M, N] (out): act(float(S) fl32(sa sw) + bias) in
 *           fp32, rounded once to bf16
 * M >= 0 (0: no-op), N % 8 == 0, N >= 8, K as above.
 */
int32_t svdq_i8_gemm(const int8_t *qa, const float *sa, const int8_t *qw, const float *sw,
                     const uint16_t *bias, int32_t act, int64_t M, int64_t N, int64_t K,
                     uint16_t *Y, void *workspace, size_t ws_bytes, void *stream);

/* Workspace of svdq_i8_linear: qa and sa (0 for a few tokens, whose codes never
 * leave the chip; `workspace` may then be NULL). */
size_t svdq_i8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* The whole layer: svdq_i8_quantize_act, then svdq_i8_gemm on one stream,
 * intermediates carved out of `workspace`; for a few tokens one launch that does
 * both, with the same result to the bit. */
int32_t svdq_i8_linear(const uint16_t *X, const float *lambda, const int8_t *qw, const float *sw,
                       const uint16_t *bias, int32_t act, int64_t M, int64_t N, int64_t K,
                       uint16_t *Y, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_I8_H */
