// paged_internal.h -- launchers of the attention of packed and paged sequences,
// the page tables and the norm and turn into the cache (internal; not part of
// the ABI).
#pragma once

#include "svdq_internal.h"
#include "svdq_paged.h"

namespace svdq {

// A checked svdq_packed_shape or svdq_paged_shape with the call's tensors.
// Element (row n, head g, d) of K: packed k[n k_stride + g D + d]; paged page
// t = tables[b][n >> page_shift], k[((t G + g) page + n % page) D + d].
struct SpanArgs {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    const int32_t *q_starts;
    const int32_t *k_starts;             // packed (q_starts if the caller gave none)
    const int32_t *tables, *kv_len;      // paged; null otherwise
    int64_t T, Tk;                       // rows of q; rows of k, or keys a table row can name
    int64_t q_stride, k_stride, v_stride;
    int64_t pages;
    int B, H, G, D, group;
    int page_shift, width, max_new, causal;
    float scale_log2;                    // scale log2(e)
    float inv_group_f;                   // 1 / group
    double inv_group;
    double line;                         // the most that ascending starts can make of it (span_plan.h)
};

// Tiles of 128 or 256 rows; paged with at most 32 rows of a request and key head: a wave each.
size_t span_tile_workspace(const SpanArgs &a);
hipError_t launch_span_tiles(const SpanArgs &a, void *ws, hipStream_t stream);
size_t span_few_workspace(const SpanArgs &a);
hipError_t launch_span_few(const SpanArgs &a, void *ws, hipStream_t stream);

struct TableArgs {
    const int32_t *cached, *added, *free_pages;
    int32_t *tables, *q_starts, *kv_len, *slots, *positions, *counts;
    int64_t T, pages, free_count;
    int B, page_shift, width;
};
hipError_t launch_page_tables(const TableArgs &a, hipStream_t stream);

struct CacheArgs {
    const uint16_t *qkv, *gq, *gk;
    const float *cos_t, *sin_t;
    const int32_t *positions, *slots;
    uint16_t *q, *k_cache, *v_cache;
    int64_t T, P, pages;
    int H, G, D, R, half, page_shift;
    float eps;
};
int64_t cache_rope_groups(const CacheArgs &a);   // workgroups of 256
hipError_t launch_cache_rope(const CacheArgs &a, hipStream_t stream);

}  // namespace svdq
