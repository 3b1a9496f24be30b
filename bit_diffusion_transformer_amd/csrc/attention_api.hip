// attention_api.hip -- the C ABI of include/svdq_attention.h: argument
// validation, workspace carving and launches.  Arguments are checked first
// (no device call), then the device, then the launches follow.
#include <cmath>

#include "attention_internal.h"
#include "svdq_checks.h"

using namespace svdq;

namespace {

int32_t read_axes(const svdq_rope_axes *e, RopeAxes &out, int &pairs) {
    if (!e) return fail(SVDQ_ERR_INVALID_ARG, "axes must not be NULL");
    if (e->axes < 1 || e->axes > SVDQ_ROPE_MAX_AXES)
        return fail(SVDQ_ERR_INVALID_ARG, "axes must be 1 .. %d (got %d)", SVDQ_ROPE_MAX_AXES,
                    e->axes);
    int64_t D = 0;
    out = RopeAxes{};
    out.axes = e->axes;
    for (int a = 0; a < e->axes; ++a) {
        if (e->dims[a] < 2 || e->dims[a] % 2 != 0)
            return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "dims[%d] must be even and >= 2 (got %d)", a,
                        e->dims[a]);
        if (!(e->theta[a] > 0.0) || !std::isfinite(e->theta[a]))
            return fail(SVDQ_ERR_INVALID_ARG, "theta[%d] must be finite and > 0", a);
        D += e->dims[a];
        out.dims[a] = e->dims[a];
        out.log_theta[a] = std::log(e->theta[a]);
    }
    if (D % 8 != 0 || D > SVDQ_ROPE_MAX_DIM)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE,
                    "the dims must add up to a multiple of 8 of at most %d (got %lld)",
                    SVDQ_ROPE_MAX_DIM, (long long)D);
    pairs = (int)(D / 2);
    return SVDQ_OK;
}

int32_t read_shape(const svdq_attention_shape *e, AttnShape &a) {
    if (!e) return fail(SVDQ_ERR_INVALID_ARG, "shape must not be NULL");
    SVDQ_TRY(check_rows(e->batch, "batch"));
    SVDQ_TRY(check_rows(e->seq_q, "seq_q"));
    if (e->seq_k < 1 || e->seq_k > SVDQ_MAX_KEYS)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "seq_k must be 1 .. %d (got %lld)", SVDQ_MAX_KEYS,
                    (long long)e->seq_k);
    if (e->heads < 1) return fail(SVDQ_ERR_INVALID_ARG, "heads must be >= 1 (got %d)", e->heads);
    if (e->kv_heads < 1 || e->heads % e->kv_heads != 0)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "kv_heads = %d must divide heads = %d", e->kv_heads,
                    e->heads);
    if (e->head_dim != 64 && e->head_dim != 128)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "head_dim must be 64 or 128 (got %d)",
                    e->head_dim);
    if (e->keep < 1 || e->keep > SVDQ_MAX_KEYS / SVDQ_KEY_BLOCK)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "keep must be 1 .. %d (got %d)",
                    SVDQ_MAX_KEYS / SVDQ_KEY_BLOCK, e->keep);
    if (e->first < 0 || e->first > e->keep)
        return fail(SVDQ_ERR_INVALID_ARG, "first must be 0 .. keep = %d (got %d)", e->keep,
                    e->first);
    a.B = e->batch;
    a.seq_q = e->seq_q;
    a.seq_k = e->seq_k;
    a.H = e->heads;
    a.G = e->kv_heads;
    a.D = e->head_dim;
    a.keep = e->keep;
    a.first = e->first;
    a.nq = (a.seq_q + SVDQ_QUERY_BLOCK - 1) / SVDQ_QUERY_BLOCK;
    a.nk = (a.seq_k + SVDQ_KEY_BLOCK - 1) / SVDQ_KEY_BLOCK;
    a.planes_q = a.B * a.H;
    a.planes_k = a.B * a.G;
    SVDQ_TRY(check_rows(a.planes_q, "batch * heads"));
    // the means (one workgroup per block), the choice (fewer than one of 512 per
    // query block), the attention, the join
    SVDQ_TRY(check_grid(a.planes_q * a.nq + a.planes_k * a.nk, 512, "the block selection"));
    SVDQ_TRY(check_grid(a.planes_q * a.nq * attention_splits(a), 256, "the block attention"));
    return SVDQ_OK;
}

bool empty(const AttnShape &a) { return a.planes_q == 0 || a.seq_q == 0; }

// 2^127 at most: the kernels take scale log2(e), which has to be finite.
int32_t check_scale(float scale) {
    if (!(scale > 0.0f) || scale > 0x1p127f)
        return fail(SVDQ_ERR_INVALID_ARG, "scale must be > 0 and at most 2^127");
    return SVDQ_OK;
}

int32_t check_workspace(const void *ws, size_t ws_bytes, size_t need) {
    if (ws_bytes < need)
        return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes < %zu needed", ws_bytes,
                    need);
    return need == 0 ? SVDQ_OK : need_ptr(ws, "workspace");
}

// svdq_sparse_attention: the selection's means, or afterwards the attention's
// partial results, and the lists.
size_t list_bytes(const AttnShape &a) {
    return a.every() ? 0 : align256((size_t)(a.planes_q * a.nq) * (size_t)a.keep * 4);
}
size_t step_bytes(const AttnShape &a) {
    const size_t s = select_workspace(a), t = attention_workspace(a);
    return s > t ? s : t;
}

}  // namespace

extern "C" {

int32_t svdq_rope_tables(const float *pos, int64_t S, const svdq_rope_axes *axes, float *cos_t,
                         float *sin_t, void *stream) {
    g_last_error[0] = 0;
    SVDQ_TRY(check_rows(S, "S"));
    RopeAxes ax;
    int pairs = 0;
    SVDQ_TRY(read_axes(axes, ax, pairs));
    if (S == 0) return SVDQ_OK;
    SVDQ_TRY(need_ptr(pos, "pos"));
    SVDQ_TRY(need_ptr(cos_t, "cos_t"));
    SVDQ_TRY(need_ptr(sin_t, "sin_t"));
    SVDQ_TRY(check_device());
    return hip_status(launch_rope_tables(pos, S, ax, pairs, cos_t, sin_t, (hipStream_t)stream),
                      "rope_tables launch");
}

int32_t svdq_qkv_norm_rope(const uint16_t *qkv, int64_t M, const svdq_qkv_epilogue *e,
                           void *stream) {
    g_last_error[0] = 0;
    SVDQ_TRY(check_rows(M, "M"));
    SVDQ_TRY(validate_qkv(e, M, false));
    SVDQ_TRY(check_rows(3 * (int64_t)e->heads * e->head_dim, "3 heads head_dim"));
    if (M == 0) return SVDQ_OK;
    SVDQ_TRY(check_grid(qkv_norm_rope_groups(M, e->heads, e->head_dim), 256, "the norm and turn"));
    SVDQ_TRY(need_ptr(qkv, "qkv"));
    SVDQ_TRY(check_device());
    return hip_status(launch_qkv_norm_rope(qkv, M, qkv_args(e), (hipStream_t)stream),
                      "qkv_norm_rope launch");
}

size_t svdq_select_blocks_workspace_bytes(const svdq_attention_shape *shape) {
    AttnShape a;
    return read_shape(shape, a) == SVDQ_OK && !empty(a) ? select_workspace(a) : 0;
}

int32_t svdq_select_blocks(const uint16_t *q, const uint16_t *k, const int32_t *kv_len,
                           const svdq_attention_shape *shape, int32_t *blocks, void *workspace,
                           size_t ws_bytes, void *stream) {
    g_last_error[0] = 0;
    AttnShape a;
    SVDQ_TRY(read_shape(shape, a));
    if (empty(a)) return SVDQ_OK;
    SVDQ_TRY(need_ptr(q, "q"));
    SVDQ_TRY(need_ptr(k, "k"));
    if (kv_len) SVDQ_TRY(need_ptr(kv_len, "kv_len"));
    SVDQ_TRY(need_ptr(blocks, "blocks"));
    SVDQ_TRY(check_workspace(workspace, ws_bytes, select_workspace(a)));
    SVDQ_TRY(check_device());
    return hip_status(launch_select_blocks(q, k, kv_len, a, blocks, workspace, (hipStream_t)stream),
                      "select_blocks launch");
}

size_t svdq_block_attention_workspace_bytes(const svdq_attention_shape *shape) {
    AttnShape a;
    return read_shape(shape, a) == SVDQ_OK && !empty(a) ? attention_workspace(a) : 0;
}

int32_t svdq_block_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                             const int32_t *kv_len, const svdq_attention_shape *shape,
                             float scale, const int32_t *blocks, uint16_t *out, void *workspace,
                             size_t ws_bytes, void *stream) {
    g_last_error[0] = 0;
    AttnShape a;
    SVDQ_TRY(read_shape(shape, a));
    SVDQ_TRY(check_scale(scale));
    if (empty(a)) return SVDQ_OK;
    SVDQ_TRY(need_ptr(q, "q"));
    SVDQ_TRY(need_ptr(k, "k"));
    SVDQ_TRY(need_ptr(v, "v"));
    if (kv_len) SVDQ_TRY(need_ptr(kv_len, "kv_len"));
    SVDQ_TRY(need_ptr(blocks, "blocks"));
    SVDQ_TRY(need_ptr(out, "out"));
    SVDQ_TRY(check_workspace(workspace, ws_bytes, attention_workspace(a)));
    SVDQ_TRY(check_device());
    return hip_status(launch_block_attention(q, k, v, kv_len, a, scale, blocks, nullptr, out, workspace,
                                             (hipStream_t)stream),
                      "block_attention launch");
}

size_t svdq_sparse_attention_workspace_bytes(const svdq_attention_shape *shape) {
    AttnShape a;
    return read_shape(shape, a) == SVDQ_OK && !empty(a) ? step_bytes(a) + list_bytes(a) : 0;
}

int32_t svdq_sparse_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                              const int32_t *kv_len, const svdq_attention_shape *shape,
                              float scale, int32_t *blocks, uint16_t *out, void *workspace,
                              size_t ws_bytes, void *stream) {
    g_last_error[0] = 0;
    AttnShape a;
    SVDQ_TRY(read_shape(shape, a));
    SVDQ_TRY(check_scale(scale));
    if (empty(a)) return SVDQ_OK;
    SVDQ_TRY(need_ptr(q, "q"));
    SVDQ_TRY(need_ptr(k, "k"));
    SVDQ_TRY(need_ptr(v, "v"));
    if (kv_len) SVDQ_TRY(need_ptr(kv_len, "kv_len"));
    if (blocks) SVDQ_TRY(need_ptr(blocks, "blocks"));
    SVDQ_TRY(need_ptr(out, "out"));
    SVDQ_TRY(check_workspace(workspace, ws_bytes, step_bytes(a) + list_bytes(a)));
    SVDQ_TRY(check_device());
    hipStream_t s = (hipStream_t)stream;
    if (a.every())                                   // nothing to select
        return hip_status(launch_block_attention(q, k, v, kv_len, a, scale, nullptr, blocks, out,
                                                 workspace, s),
                          "block_attention launch");
    int32_t *lists = blocks ? blocks
                            : reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + step_bytes(a));
    SVDQ_TRY(hip_status(launch_select_blocks(q, k, kv_len, a, lists, workspace, s),
                        "select_blocks launch"));
    return hip_status(launch_block_attention(q, k, v, kv_len, a, scale, lists, nullptr, out, workspace,
                                             s),
                      "block_attention launch");
}

}  // extern "C"
