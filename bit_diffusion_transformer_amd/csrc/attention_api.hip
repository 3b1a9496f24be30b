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

}  // extern "C"
