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
 * alias inputs; results deterministic (no atomics).  A workspace serves one
 * call at a time: calls that may run at once (on two streams, in two captured
 * graphs) need one each.
 */
#ifndef SVDQ_ATTENTION_H
#define SVDQ_ATTENTION_H

#include "svdq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SVDQ_ROPE_MAX_AXES 4
#define SVDQ_ROPE_MAX_DIM 256   /* largest head_dim of the tables */
#define SVDQ_QUERY_BLOCK 128    /* query rows that share one list of key blocks */
#define SVDQ_KEY_BLOCK 64       /* keys per block */
#define SVDQ_MAX_KEYS (1 << 18) /* largest seq_k of the sparse attention */

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
 * there; sine and cosine of the reduced angle in fp32: absolute error at most
 * 2^-21 for |pos| <= 2^26 and theta >= 1.  Farther positions add up to
 * 7 |pos| 2^-53, the rounding of the frequencies (2^-21 in all is passed near
 * 2^31); with theta < 1 the frequencies, and that error, grow with 1 / theta.
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

/* ------------------------------------------------------------------
 * Block-sparse attention.  The queries of a head are taken in blocks of 128
 * rows, the keys in blocks of 64.  The score of query block i and key block j
 * is the product of the two blocks' means (over the query rows that exist,
 * and over the keys below kv_len); query block i attends to the `keep` key
 * blocks with the highest scores:
 *   O[m] = sum_n p[m][n] v[n],  p = softmax over the keys n of those blocks
 *          of scale q[m] . k[n].
 * Keys at or past a sequence's kv_len take no part, whatever they hold.  A
 * query block without any key gives rows of zeros.
 * ------------------------------------------------------------------ */
typedef struct svdq_attention_shape {
    int64_t batch;      /* B >= 0 (0: no-op) */
    int64_t seq_q;      /* Sq >= 0 (0: no-op) */
    int64_t seq_k;      /* Sk, 1 .. SVDQ_MAX_KEYS */
    int32_t heads;      /* H >= 1 */
    int32_t kv_heads;   /* G >= 1, H % G == 0: head h reads key head h / (H / G) */
    int32_t head_dim;   /* D: 64 or 128 */
    int32_t keep;       /* key blocks per query block, 1 .. SVDQ_MAX_KEYS / 64 */
    int32_t first;      /* 0 .. keep: the first `first` key blocks are always taken (and count) */
} svdq_attention_shape;

/* Workspace of svdq_select_blocks: the blocks' means, or their scores (0 where
 * `keep` takes every block). */
size_t svdq_select_blocks_workspace_bytes(const svdq_attention_shape *shape);

/*
 * The lists of key blocks.
 *   q       device bf16 [B, H, Sq, D]
 *   k       device bf16 [B, G, Sk, D]
 *   kv_len  device int32 [B] valid keys of each sequence (clamped to 0 .. Sk),
 *           or NULL: all Sk
 *   blocks  device int32 [B, H, ceil(Sq/128), keep] (out): the block numbers
 *           in ascending order, -1 behind the last one where fewer than
 *           `keep` blocks hold a valid key
 * Means and scores are taken in 64 bits; equal scores go to the lower block
 * number.  q and the valid keys must be finite (otherwise which blocks are
 * taken is unspecified).
 */
int32_t svdq_select_blocks(const uint16_t *q, const uint16_t *k, const int32_t *kv_len,
                           const svdq_attention_shape *shape, int32_t *blocks, void *workspace,
                           size_t ws_bytes, void *stream);

/* Workspace of svdq_block_attention: partial results where few query blocks
 * are split over their keys (0 elsewhere). */
size_t svdq_block_attention_workspace_bytes(const svdq_attention_shape *shape);

/*
 * Attention over given lists (shape's `first` is not read).
 *   v       device bf16 [B, G, Sk, D]
 *   scale   > 0 and at most 2^127 (usually D^-1/2); the sum of |q[m][d] k[n][d]|
 *           over d, and scale times it, below 2^126 (a larger one may pass
 *           what fp32 holds and give NaN)
 *   blocks  device int32 [B, H, ceil(Sq/128), keep]: an entry that is
 *           negative, past the last block with a valid key, or not above
 *           every entry before it in its list is passed over, so a block
 *           named twice counts once
 *   out     device bf16 [B, Sq, H, D] (out): the rows [M, H D] of the output
 *           projection
 * Products in bf16 with fp32 sums; the softmax in fp32 with the running
 * maximum and sum; its weights are rounded once to bf16 for the product with
 * v; one rounding of the result to bf16.  A NaN or an infinity in a query row
 * gives a row of NaN, a NaN in a valid key NaN in the rows that take it, an
 * infinite valid v an infinity (or NaN beside weights of zero) in its column;
 * other rows do not see them.
 */
int32_t svdq_block_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                             const int32_t *kv_len, const svdq_attention_shape *shape,
                             float scale, const int32_t *blocks, uint16_t *out, void *workspace,
                             size_t ws_bytes, void *stream);

/* Workspace of svdq_sparse_attention (both steps and the lists). */
size_t svdq_sparse_attention_workspace_bytes(const svdq_attention_shape *shape);

/*
 * svdq_select_blocks then svdq_block_attention on one stream.  blocks: the
 * lists (out), or NULL: they stay in the workspace (where `keep` takes every
 * block there are none, and nothing is scored).
 */
int32_t svdq_sparse_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                              const int32_t *kv_len, const svdq_attention_shape *shape,
                              float scale, int32_t *blocks, uint16_t *out, void *workspace,
                              size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_ATTENTION_H */
