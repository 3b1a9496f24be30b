/*
 * svdq_attention.h -- C ABI of the attention half of a diffusion transformer
 * block next to the quantized linears of svdq.h: rotary tables for tokens
 * with several position axes, the Q / K norm and rotary turn of a projection
 * that was written as [M, N], and attention over key blocks that a score of
 * block means selects.
 *
 * Conventions, status codes, svdq_last_error and svdq_status_string are
 * those of svdq.h: bf16 tensors as uint16_t bit patterns, row-major and
 * contiguous; device pointers 16-byte aligned and of the current HIP device;
 * work enqueued on `stream` without synchronizing; every argument checked
 * before anything is launched, arguments first, then the device; buffers
 * owned by the caller, nothing allocated, no state kept; outputs must not
 * alias inputs; results deterministic (no atomics).
 */
#ifndef SVDQ_ATTENTION_H
#define SVDQ_ATTENTION_H

#include "svdq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SVDQ_ROPE_MAX_AXES 4
#define SVDQ_ROPE_MAX_DIM 256   /* largest head_dim of the tables */

/*
 * How a head's dimension is divided among the position axes (e.g. time,
 * height, width): axis a turns dims[a] consecutive elements, dims[a] / 2
 * pairs; pair i of axis a turns by pos[s][a] theta[a]^(-2 i / dims[a]).
 */
typedef struct svdq_rope_axes {
    int32_t axes;                       /* 1 .. SVDQ_ROPE_MAX_AXES */
    int32_t dims[SVDQ_ROPE_MAX_AXES];   /* each even and >= 2; the sum D % 8 == 0, <= 256 */
    double theta[SVDQ_ROPE_MAX_AXES];   /* finite and > 0 */
} svdq_rope_axes;

/*
 * Rotary tables: cos_t[s][p] and sin_t[s][p] of the angle of token s and pair
 * p (the pairs of axis 0 first), as svdq_qkv_epilogue takes them.
 *   pos    device fp32 [S, axes]   positions (whole or fractional, finite)
 *   axes   host pointer, read during the call only
 *   cos_t  device fp32 [S, D/2]    (out)
 *   sin_t  device fp32 [S, D/2]    (out)
 * S >= 0 (0: no-op).  Angles are formed in 64 bits and reduced to one turn
 * there, so positions past 10^6 keep their accuracy; sine and cosine of the
 * reduced angle in fp32: absolute error at most 2^-21.
 */
int32_t svdq_rope_tables(const float *pos, int64_t S, const svdq_rope_axes *axes, float *cos_t,
                         float *sin_t, void *stream);

/*
 * The epilogue of svdq_w4a4_lr_gemm_qkv for a projection that another GEMM
 * has written (svdq_mx_linear, svdq_i8_linear, a 16-bit product):
 *   qkv  device bf16 [M, 3 H D]  columns [Q | K | V], heads of D columns each
 *   epi  as for svdq_w4a4_lr_gemm_qkv (host pointer), except that gamma_q and
 *        gamma_k may each be NULL: that section turns without a norm
 * Q and K are normed and turned in fp32 and rounded once to bf16, V is
 * copied; outputs bf16 [M/S, H, S, D].  M >= 0 (0: no-op), M % seq == 0.
 */
int32_t svdq_qkv_norm_rope(const uint16_t *qkv, int64_t M, const svdq_qkv_epilogue *epi,
                           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_ATTENTION_H */
