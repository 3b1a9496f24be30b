/*
 * svdq_paged.h -- C ABI of attention over sequences of different lengths: packed
 * one after another, or as new tokens over a paged key / value cache; the page
 * tables of that cache; and the Q / K norm and rotary turn that fills it.
 *
 * Conventions, status codes, svdq_last_error and svdq_status_string are those of
 * svdq.h: bf16 tensors as uint16_t bit patterns; device pointers 16-byte aligned
 * (of int32 arrays 4-byte) and of the current HIP device; work enqueued on
 * `stream` without synchronizing; every argument checked before anything is launched, arguments
 * first, then the device; buffers owned by the caller, nothing allocated, no
 * state kept; outputs must not alias inputs; results deterministic (no atomics).
 * A workspace serves one call at a time: calls that may run at once (on two
 * streams, in two captured graphs) need one each.
 *
 * Lengths, starts, tables, slots and positions are device data that no call
 * waits for.  Values outside their range are never followed out of a buffer;
 * what such a value gives is stated where it is read.
 */
#ifndef SVDQ_PAGED_H
#define SVDQ_PAGED_H

#include "svdq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SVDQ_MIN_PAGE 16           /* tokens of a page: a power of two, */
#define SVDQ_MAX_PAGE 256          /* 16 .. 256 */
#define SVDQ_MAX_SLOTS (1 << 30)   /* largest pages * page, and width * page */
#define SVDQ_MAX_REQUESTS 8192     /* largest batch of svdq_page_tables */
#define SVDQ_MAX_GROUP 64          /* largest heads / kv_heads */
#define SVDQ_MAX_STRIDE (1 << 20)  /* largest row stride */

/* ------------------------------------------------------------------
 * Attention of packed sequences.  Sequence b has the query rows q_starts[b] ..
 * q_starts[b+1] - 1 (Lq of them) and the key rows k_starts[b] .. k_starts[b+1]
 * - 1 (Lk):
 *   out[i] = sum_n p[i][n] v[n],  p = softmax over the keys n that row i sees of
 *            scale q[i] . k[n],
 * for every head (head h reads key head h / (heads / kv_heads)).  Without
 * `causal` a row sees all Lk keys; with it row i (0 .. Lq - 1 within its
 * sequence) sees the first Lk - Lq + i + 1: the last row sees all.  A row that
 * sees no key gives zeros.
 * ------------------------------------------------------------------ */
typedef struct svdq_packed_shape {
    int64_t tokens_q;    /* T: rows of q and out, >= 0 (0: no-op) */
    int64_t tokens_k;    /* rows of k and v, >= 0 */
    int64_t q_stride;    /* elements from one row of q to the next: a multiple of 8, */
    int64_t k_stride;    /*   at least its heads * head_dim and at most */
    int64_t v_stride;    /*   SVDQ_MAX_STRIDE */
    int32_t sequences;   /* >= 0 (0: no-op) */
    int32_t heads;       /* H >= 1 */
    int32_t kv_heads;    /* G >= 1, H % G == 0, H / G <= SVDQ_MAX_GROUP */
    int32_t head_dim;    /* D: 64 or 128 */
    int32_t causal;      /* 0 or 1 */
} svdq_packed_shape;

/* Workspace of svdq_packed_attention: partial results where the keys of a tile
 * of rows are shared among workgroups. */
size_t svdq_packed_attention_workspace_bytes(const svdq_packed_shape *shape);

/*
 *   q         device bf16 [T][H][D], rows q_stride apart
 *   k, v      device bf16 [tokens_k][G][D], rows k_stride and v_stride apart
 *   q_starts  device int32 [sequences + 1], ascending, 0 .. T
 *   k_starts  device int32 [sequences + 1], ascending, 0 .. tokens_k, or NULL:
 *             q_starts (then tokens_k == tokens_q)
 *   scale     > 0 and at most 2^127 (usually D^-1/2); the sum of |q[d] k[d]| over
 *             d, and scale times it, below 2^126 (a larger one may pass what
 *             fp32 holds and give NaN); the sum of |v| over the keys of a row below
 *             2^119 in each column (the sums of weights times v are divided by the
 *             weights' at the end, and a weight is at most 2^8; a larger one may give
 *             an infinity or NaN)
 *   out       device bf16 [T][H][D] (out), contiguous; rows of no sequence are
 *             left as they were
 * Starts are clamped to 0 .. T (tokens_k); a sequence that ends before it starts
 * has no rows.  Where starts descend, rows of several sequences hold the result
 * of one of them, or of a mixture; no row is written where that is more work
 * than ascending starts can name.
 * Products in bf16 with fp32 sums; the softmax in fp32 with the running maximum
 * and sum; its weights are rounded once to bf16 for the product with v; one
 * rounding of the result to bf16.  A key that a row does not see takes no part
 * in it, whatever it holds.  A NaN or an infinity in a query row gives a row of
 * NaN if the row sees a key, a NaN in a key NaN in the rows that see it (an
 * infinity likewise, or no weight where its score is minus infinity), a v that is
 * not finite an infinity or NaN in its column of the rows that see it.
 */
int32_t svdq_packed_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                              const int32_t *q_starts, const int32_t *k_starts,
                              const svdq_packed_shape *shape, float scale, uint16_t *out,
                              void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------
 * Attention of new tokens over a paged cache.  Request b has the query rows
 * q_starts[b] .. q_starts[b+1] - 1 (its Lq new tokens) and kv_len[b] keys, the
 * new tokens' own included: key n is row n % page of page tables[b][n / page].
 * What a row sees, and its result, are as above with Lk = kv_len[b].
 * ------------------------------------------------------------------ */
typedef struct svdq_paged_shape {
    int64_t tokens;      /* T: rows of q and out, >= 0 (0: no-op) */
    int64_t pages;       /* pages of the cache, >= 0; pages * page <= SVDQ_MAX_SLOTS */
    int64_t q_stride;    /* as above */
    int32_t requests;    /* >= 0 (0: no-op) */
    int32_t heads, kv_heads, head_dim;   /* as above */
    int32_t page;        /* tokens of a page: a power of two, 16 .. 256 */
    int32_t width;       /* entries of a table row, >= 0; width * page <= SVDQ_MAX_SLOTS */
    int32_t max_new;     /* the most new tokens of a request, >= 1: chooses the kernel; a
                            request with more is computed all the same, slower, and
                            so are requests with far fewer (64 with one token each
                            over up to 8192 keys: 70 us with 1, 85 with 64) */
    int32_t causal;      /* 0 or 1 */
} svdq_paged_shape;

size_t svdq_paged_attention_workspace_bytes(const svdq_paged_shape *shape);

/*
 *   k_cache, v_cache  device bf16 [pages][G][page][D], contiguous
 *   tables    device int32 [requests][width]: page numbers.  An entry outside
 *             0 .. pages - 1 holds no keys: the rows see the others
 *   q_starts  device int32 [requests + 1], as above
 *   kv_len    device int32 [requests], clamped to 0 .. width * page
 * q, scale, out, and what is not finite: as for svdq_packed_attention.
 */
int32_t svdq_paged_attention(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                             const int32_t *tables, const int32_t *q_starts,
                             const int32_t *kv_len, const svdq_paged_shape *shape, float scale,
                             uint16_t *out, void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------
 * Page tables of a step.  Request b holds cached[b] tokens, in the pages of its
 * first ceil(cached[b] / page) table entries, and gets added[b] more, packed one
 * request after another.  The pages it lacks are taken from `free_pages` in
 * order, request after request.
 * ------------------------------------------------------------------ */
typedef struct svdq_table_shape {
    int64_t tokens;      /* T: entries of slots and positions, >= 0 */
    int64_t pages;       /* pages of the cache, >= 0; pages * page <= SVDQ_MAX_SLOTS */
    int64_t free_count;  /* entries of free_pages, >= 0 */
    int32_t requests;    /* 0 .. SVDQ_MAX_REQUESTS */
    int32_t page;        /* a power of two, 16 .. 256 */
    int32_t width;       /* entries of a table row, >= 0; width * page <= SVDQ_MAX_SLOTS */
} svdq_table_shape;

/*
 *   cached     device int32 [requests]  tokens in the cache (below 0: 0; at most
 *              SVDQ_MAX_SLOTS)
 *   added      device int32 [requests]  new tokens (below 0: 0)
 *   free_pages device int32 [free_count]  distinct pages that no request holds
 *   tables     device int32 [requests][width] (in, out): the entries of the new
 *              pages are written (-1 where free_pages ends), others left alone
 *   q_starts   device int32 [requests + 1] (out): where each request's new tokens
 *              start, at most T
 *   kv_len     device int32 [requests] (out): cached + added, at most
 *              SVDQ_MAX_SLOTS
 *   slots      device int32 [T] (out): page number * page + row of each new
 *              token, -1 for a token without a page (free_pages or the table
 *              row ended, or its page number is outside 0 .. pages - 1) and for
 *              the rows behind the last request
 *   positions  device int32 [T] (out): the token's place in its request,
 *              cached[b] + i; -1 behind the last request
 *   counts     device int32 [2] (out): pages taken from free_pages (as many as
 *              are needed, whether there are so many or not, 2^31 - 1 at most,
 *              and no more entries are written); new tokens without
 *              a slot, those past T included.  The step can be used if the
 *              second is 0.
 * The result depends on cached, added, free_pages and the table entries of the
 * cached tokens alone: the same call again gives the same.
 */
int32_t svdq_page_tables(const int32_t *cached, const int32_t *added, const int32_t *free_pages,
                         const svdq_table_shape *shape, int32_t *tables, int32_t *q_starts,
                         int32_t *kv_len, int32_t *slots, int32_t *positions, int32_t *counts,
                         void *stream);

/* ------------------------------------------------------------------
 * Norm, turn and cache: a written projection [T][(H + 2 G) D], columns
 * [Q | K | V] of heads of D columns, with the per-head RMS norm
 *   x gamma / sqrt(mean x^2 + eps)
 * of Q and K (gamma NULL: none) and the rotary turn of the first `rotary`
 * columns of each head by the table row of the token's position.  Pair i of a
 * head is (2 i, 2 i + 1), or with `half` (i, rotary / 2 + i):
 *   (x, y) -> (x cos - y sin, x sin + y cos).
 * Q goes to rows of q, K and V to the cache rows of the tokens' slots.
 * ------------------------------------------------------------------ */
typedef struct svdq_cache_epilogue {
    int64_t tokens;           /* T >= 0 (0: no-op) */
    int64_t table_rows;       /* rows of cos_t and sin_t, >= 1 */
    int64_t pages;            /* pages of the cache, >= 0; pages * page <= SVDQ_MAX_SLOTS */
    int32_t heads, kv_heads;  /* H, G >= 1, H % G == 0, H / G <= SVDQ_MAX_GROUP */
    int32_t head_dim;         /* D: 64 or 128 */
    int32_t rotary;           /* columns that turn: a multiple of 16, 16 .. D */
    int32_t half;             /* 0: pairs of neighbours; 1: of the two halves */
    int32_t page;             /* a power of two, 16 .. 256 */
    const uint16_t *gamma_q, *gamma_k;   /* device bf16 [D], or NULL */
    float eps;                           /* finite and >= 0 */
    const float *cos_t, *sin_t;          /* device fp32 [table_rows][rotary / 2] */
    const int32_t *positions;            /* device int32 [T] */
    const int32_t *slots;                /* device int32 [T] */
    uint16_t *q;                         /* device bf16 [T][H][D] (out) */
    uint16_t *k_cache, *v_cache;         /* device bf16 [pages][G][page][D] (out) */
} svdq_cache_epilogue;

/*
 * qkv device bf16 [T][(H + 2 G) D], contiguous.  Norm and turn in fp32, one
 * rounding to bf16 (a head whose squares add up to 2^128 or more gives zeros); V
 * is copied.  A token whose slot is outside 0 .. pages * page - 1 leaves the cache
 * as it was; one whose position is outside the tables (rows behind the last
 * request) leaves its row of q and the cache as they were.
 * Slots of the call's tokens must be distinct (of equal ones the cache row holds
 * a mixture).
 */
int32_t svdq_qkv_norm_rope_cache(const uint16_t *qkv, const svdq_cache_epilogue *epi,
                                 void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_PAGED_H */
