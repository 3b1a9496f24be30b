// paged_api.hip -- the C ABI of include/svdq_paged.h: argument validation,
// workspace carving and launches.  Arguments are checked first (no device
// call), then the device, then the launches follow.
#include "paged_internal.h"
#include "svdq_checks.h"

using namespace svdq;

namespace {

int32_t read_heads(int32_t H, int32_t G, int32_t D) {
    if (H < 1) return fail(SVDQ_ERR_INVALID_ARG, "heads must be >= 1 (got %d)", H);
    if (G < 1 || H % G != 0)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "kv_heads = %d must divide heads = %d", G, H);
    if (H / G > SVDQ_MAX_GROUP)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "heads / kv_heads = %d exceeds the limit %d", H / G,
                    SVDQ_MAX_GROUP);
    if (D != 64 && D != 128)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "head_dim must be 64 or 128 (got %d)", D);
    return check_rows((int64_t)H * D, "heads * head_dim");
}

int32_t read_stride(int64_t stride, int64_t least, const char *name) {
    if (stride % 8 != 0 || stride < least || stride > SVDQ_MAX_STRIDE)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s must be a multiple of 8, %lld .. %d (got %lld)", name,
                    (long long)least, SVDQ_MAX_STRIDE, (long long)stride);
    return SVDQ_OK;
}

int32_t check_count(int64_t n, const char *name) {
    if (n < 0) return fail(SVDQ_ERR_INVALID_ARG, "%s must be >= 0 (got %lld)", name, (long long)n);
    return SVDQ_OK;
}

// An int32 array: parts of larger ones are usual, so any element may be its first.
int32_t need_index(const int32_t *p, const char *name) {
    if (!p) return fail(SVDQ_ERR_INVALID_ARG, "%s must not be NULL", name);
    if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(SVDQ_ERR_MISALIGNED, "%s is not 4-byte aligned", name);
    return SVDQ_OK;
}

int32_t check_flag(int32_t x, const char *name) {
    if (x != 0 && x != 1) return fail(SVDQ_ERR_INVALID_ARG, "%s must be 0 or 1 (got %d)", name, x);
    return SVDQ_OK;
}

// A page's tokens, pages and (of a table row) width -> the page's logarithm.
int32_t read_pages(int32_t page, int64_t pages, int64_t width, int &shift) {
    shift = 0;
    while (shift < 8 && 1 << shift < page) ++shift;
    if (page < SVDQ_MIN_PAGE || page > SVDQ_MAX_PAGE || 1 << shift != page)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "page must be a power of two, %d .. %d (got %d)",
                    SVDQ_MIN_PAGE, SVDQ_MAX_PAGE, page);
    SVDQ_TRY(check_count(pages, "pages"));
    SVDQ_TRY(check_count(width, "width"));
    if (pages > SVDQ_MAX_SLOTS / page || width > SVDQ_MAX_SLOTS / page)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%lld pages, %lld to a request, of %d tokens exceed the limit %d",
                    (long long)pages, (long long)width, page, SVDQ_MAX_SLOTS);
    return SVDQ_OK;
}

// The line of all tiles (span_plan.h) is exact in 64-bit floating point: whole numbers, over a
// cache quarters.  At most T group / R + B tiles of a key head, R >= 16 rows; a tile's
// length is at most (Tk + T + 512) group + 256.
int32_t check_line(SpanArgs &a) {
    const double tiles = (double)a.T * a.group / 16 + a.B;
    const double each = a.group * ((double)a.Tk + (double)a.T + 512) + 256;
    a.line = tiles * each * a.G;
    if (a.line > (a.max_new > 0 ? 0x1p51 : 0x1p52))
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%lld rows of %d sequences over %lld keys are too many",
                    (long long)a.T, a.B, (long long)a.Tk);
    return SVDQ_OK;
}

int32_t read_shape(const svdq_packed_shape *e, bool own_keys, SpanArgs &a) {
    a = SpanArgs{};
    if (!e) return fail(SVDQ_ERR_INVALID_ARG, "shape must not be NULL");
    SVDQ_TRY(check_rows(e->tokens_q, "tokens_q"));
    SVDQ_TRY(check_rows(e->tokens_k, "tokens_k"));
    SVDQ_TRY(check_rows(e->sequences, "sequences"));
    SVDQ_TRY(read_heads(e->heads, e->kv_heads, e->head_dim));
    SVDQ_TRY(check_flag(e->causal, "causal"));
    SVDQ_TRY(read_stride(e->q_stride, (int64_t)e->heads * e->head_dim, "q_stride"));
    SVDQ_TRY(read_stride(e->k_stride, (int64_t)e->kv_heads * e->head_dim, "k_stride"));
    SVDQ_TRY(read_stride(e->v_stride, (int64_t)e->kv_heads * e->head_dim, "v_stride"));
    if (!own_keys && e->tokens_k != e->tokens_q)
        return fail(SVDQ_ERR_INVALID_ARG, "without k_starts tokens_k = %lld must be tokens_q = %lld",
                    (long long)e->tokens_k, (long long)e->tokens_q);
    a.T = e->tokens_q;
    a.Tk = e->tokens_k;
    a.q_stride = e->q_stride;
    a.k_stride = e->k_stride;
    a.v_stride = e->v_stride;
    a.B = e->sequences;
    a.H = e->heads;
    a.G = e->kv_heads;
    a.D = e->head_dim;
    a.group = a.H / a.G;
    a.inv_group = 1.0 / a.group;
    a.inv_group_f = (float)a.inv_group;
    a.causal = e->causal;
    return check_line(a);
}

int32_t read_shape(const svdq_paged_shape *e, SpanArgs &a) {
    a = SpanArgs{};
    if (!e) return fail(SVDQ_ERR_INVALID_ARG, "shape must not be NULL");
    SVDQ_TRY(check_rows(e->tokens, "tokens"));
    SVDQ_TRY(check_rows(e->requests, "requests"));
    SVDQ_TRY(read_heads(e->heads, e->kv_heads, e->head_dim));
    SVDQ_TRY(check_flag(e->causal, "causal"));
    SVDQ_TRY(read_stride(e->q_stride, (int64_t)e->heads * e->head_dim, "q_stride"));
    SVDQ_TRY(read_pages(e->page, e->pages, e->width, a.page_shift));
    if (e->max_new < 1) return fail(SVDQ_ERR_INVALID_ARG, "max_new must be >= 1 (got %d)", e->max_new);
    a.T = e->tokens;
    a.Tk = (int64_t)e->width * e->page;
    a.q_stride = e->q_stride;
    a.pages = e->pages;
    a.B = e->requests;
    a.H = e->heads;
    a.G = e->kv_heads;
    a.D = e->head_dim;
    a.group = a.H / a.G;
    a.inv_group = 1.0 / a.group;
    a.inv_group_f = (float)a.inv_group;
    a.width = e->width;
    a.max_new = e->max_new;
    a.causal = e->causal;
    return check_line(a);
}

bool empty(const SpanArgs &a) { return a.T == 0 || a.B == 0; }

// 2^127 at most: the kernels take scale log2(e), which has to be finite.
int32_t read_scale(float scale, SpanArgs &a) {
    if (!(scale > 0.0f) || scale > 0x1p127f)
        return fail(SVDQ_ERR_INVALID_ARG, "scale must be > 0 and at most 2^127");
    a.scale_log2 = scale * 1.4426950408889634f;
    return SVDQ_OK;
}

// New tokens whose rows fit a wave's tile: their time is that of reading the cache.
bool few(const SpanArgs &a) { return a.max_new > 0 && (int64_t)a.max_new * a.group <= 32; }

size_t workspace_bytes(const SpanArgs &a) { return few(a) ? span_few_workspace(a) : span_tile_workspace(a); }

int32_t run(const SpanArgs &a, void *workspace, size_t ws_bytes, void *stream) {
    const size_t need = workspace_bytes(a);
    if (ws_bytes < need)
        return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes < %zu needed", ws_bytes, need);
    SVDQ_TRY(need_ptr(workspace, "workspace"));
    SVDQ_TRY(check_device());
    hipStream_t s = (hipStream_t)stream;
    return hip_status(few(a) ? launch_span_few(a, workspace, s) : launch_span_tiles(a, workspace, s),
                      "attention launch");
}

}  // namespace

extern "C" {

size_t svdq_packed_attention_workspace_bytes(const svdq_packed_shape *shape) {
    SpanArgs a;
    return read_shape(shape, true, a) == SVDQ_OK && !empty(a) ? workspace_bytes(a) : 0;
}

int32_t svdq_packed_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                              const int32_t *q_starts, const int32_t *k_starts,
                              const svdq_packed_shape *shape, float scale, uint16_t *out,
                              void *workspace, size_t ws_bytes, void *stream) {
    g_last_error[0] = 0;
    SpanArgs a;
    SVDQ_TRY(read_shape(shape, k_starts != nullptr, a));
    SVDQ_TRY(read_scale(scale, a));
    if (empty(a)) return SVDQ_OK;
    SVDQ_TRY(need_ptr(q, "q"));
    if (a.Tk > 0) {                                  // without keys k and v are not read
        SVDQ_TRY(need_ptr(k, "k"));
        SVDQ_TRY(need_ptr(v, "v"));
    }
    SVDQ_TRY(need_index(q_starts, "q_starts"));
    if (k_starts) SVDQ_TRY(need_index(k_starts, "k_starts"));
    SVDQ_TRY(need_ptr(out, "out"));
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_starts = q_starts;
    a.k_starts = k_starts ? k_starts : q_starts;
    a.out = out;
    return run(a, workspace, ws_bytes, stream);
}

size_t svdq_paged_attention_workspace_bytes(const svdq_paged_shape *shape) {
    SpanArgs a;
    return read_shape(shape, a) == SVDQ_OK && !empty(a) ? workspace_bytes(a) : 0;
}

int32_t svdq_paged_attention(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                             const int32_t *tables, const int32_t *q_starts,
                             const int32_t *kv_len, const svdq_paged_shape *shape, float scale,
                             uint16_t *out, void *workspace, size_t ws_bytes, void *stream) {
    g_last_error[0] = 0;
    SpanArgs a;
    SVDQ_TRY(read_shape(shape, a));
    SVDQ_TRY(read_scale(scale, a));
    if (empty(a)) return SVDQ_OK;
    SVDQ_TRY(need_ptr(q, "q"));
    if (a.pages > 0) {                               // without pages the cache is not read
        SVDQ_TRY(need_ptr(k_cache, "k_cache"));
        SVDQ_TRY(need_ptr(v_cache, "v_cache"));
    }
    if (a.width > 0) SVDQ_TRY(need_index(tables, "tables"));
    SVDQ_TRY(need_index(q_starts, "q_starts"));
    SVDQ_TRY(need_index(kv_len, "kv_len"));
    SVDQ_TRY(need_ptr(out, "out"));
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.tables = tables;
    a.q_starts = q_starts;
    a.kv_len = kv_len;
    a.out = out;
    return run(a, workspace, ws_bytes, stream);
}

int32_t svdq_page_tables(const int32_t *cached, const int32_t *added, const int32_t *free_pages,
                         const svdq_table_shape *e, int32_t *tables, int32_t *q_starts,
                         int32_t *kv_len, int32_t *slots, int32_t *positions, int32_t *counts,
                         void *stream) {
    g_last_error[0] = 0;
    if (!e) return fail(SVDQ_ERR_INVALID_ARG, "shape must not be NULL");
    TableArgs a = {};
    SVDQ_TRY(check_rows(e->tokens, "tokens"));
    SVDQ_TRY(check_count(e->free_count, "free_count"));
    SVDQ_TRY(check_count(e->requests, "requests"));
    if (e->requests > SVDQ_MAX_REQUESTS)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "requests = %d exceeds the limit %d", e->requests,
                    SVDQ_MAX_REQUESTS);
    SVDQ_TRY(read_pages(e->page, e->pages, e->width, a.page_shift));
    if (e->requests > 0) {
        SVDQ_TRY(need_index(cached, "cached"));
        SVDQ_TRY(need_index(added, "added"));
        SVDQ_TRY(need_index(kv_len, "kv_len"));
        if (e->width > 0) SVDQ_TRY(need_index(tables, "tables"));
    }
    if (e->free_count > 0) SVDQ_TRY(need_index(free_pages, "free_pages"));
    SVDQ_TRY(need_index(q_starts, "q_starts"));
    if (e->tokens > 0) {
        SVDQ_TRY(need_index(slots, "slots"));
        SVDQ_TRY(need_index(positions, "positions"));
    }
    SVDQ_TRY(need_index(counts, "counts"));
    SVDQ_TRY(check_device());
    a.cached = cached;
    a.added = added;
    a.free_pages = free_pages;
    a.tables = tables;
    a.q_starts = q_starts;
    a.kv_len = kv_len;
    a.slots = slots;
    a.positions = positions;
    a.counts = counts;
    a.T = e->tokens;
    a.pages = e->pages;
    a.free_count = e->free_count;
    a.B = e->requests;
    a.width = e->width;
    return hip_status(launch_page_tables(a, (hipStream_t)stream), "page_tables launch");
}

int32_t svdq_qkv_norm_rope_cache(const uint16_t *qkv, const svdq_cache_epilogue *e, void *stream) {
    g_last_error[0] = 0;
    if (!e) return fail(SVDQ_ERR_INVALID_ARG, "epi must not be NULL");
    CacheArgs a = {};
    SVDQ_TRY(check_rows(e->tokens, "tokens"));
    SVDQ_TRY(read_heads(e->heads, e->kv_heads, e->head_dim));
    SVDQ_TRY(check_rows(((int64_t)e->heads + 2 * (int64_t)e->kv_heads) * e->head_dim,
                        "(heads + 2 kv_heads) head_dim"));
    SVDQ_TRY(read_pages(e->page, e->pages, 0, a.page_shift));
    if (e->rotary < 16 || e->rotary > e->head_dim || e->rotary % 16 != 0)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "rotary must be a multiple of 16, 16 .. head_dim = %d (got %d)",
                    e->head_dim, e->rotary);
    SVDQ_TRY(check_flag(e->half, "half"));
    if (e->table_rows < 1)
        return fail(SVDQ_ERR_INVALID_ARG, "table_rows must be >= 1 (got %lld)", (long long)e->table_rows);
    SVDQ_TRY(check_rows(e->table_rows, "table_rows"));
    if (!(e->eps >= 0.0f) || e->eps > 3.0e38f)
        return fail(SVDQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (e->tokens == 0) return SVDQ_OK;
    if (e->gamma_q) SVDQ_TRY(need_ptr(e->gamma_q, "gamma_q"));
    if (e->gamma_k) SVDQ_TRY(need_ptr(e->gamma_k, "gamma_k"));
    SVDQ_TRY(need_ptr(e->cos_t, "cos_t"));
    SVDQ_TRY(need_ptr(e->sin_t, "sin_t"));
    SVDQ_TRY(need_index(e->positions, "positions"));
    SVDQ_TRY(need_index(e->slots, "slots"));
    SVDQ_TRY(need_ptr(e->q, "q"));
    if (e->pages > 0) {
        SVDQ_TRY(need_ptr(e->k_cache, "k_cache"));
        SVDQ_TRY(need_ptr(e->v_cache, "v_cache"));
    }
    SVDQ_TRY(need_ptr(qkv, "qkv"));
    a.qkv = qkv;
    a.gq = e->gamma_q;
    a.gk = e->gamma_k;
    a.cos_t = e->cos_t;
    a.sin_t = e->sin_t;
    a.positions = e->positions;
    a.slots = e->slots;
    a.q = e->q;
    a.k_cache = e->k_cache;
    a.v_cache = e->v_cache;
    a.T = e->tokens;
    a.P = e->table_rows;
    a.pages = e->pages;
    a.H = e->heads;
    a.G = e->kv_heads;
    a.D = e->head_dim;
    a.R = e->rotary;
    a.half = e->half;
    a.eps = e->eps;
    SVDQ_TRY(check_grid(cache_rope_groups(a), 256, "the norm and turn"));
    SVDQ_TRY(check_device());
    return hip_status(launch_cache_rope(a, (hipStream_t)stream), "qkv_norm_rope_cache launch");
}

}  // extern "C"
