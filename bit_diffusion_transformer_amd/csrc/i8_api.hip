// i8_api.hip -- the C ABI of include/svdq_i8.h: argument validation, workspace
// carving and launches, in the order of the other entry points (arguments,
// device, launches).
#include "i8_internal.h"
#include "svdq_checks.h"

using namespace svdq;

namespace {

int32_t check_k_i8(int64_t K) {
    SVDQ_TRY(check_k(K));
    if (K > SVDQ_I8_MAX_K)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "K = %lld exceeds the limit %d of exact 8-bit sums",
                    (long long)K, SVDQ_I8_MAX_K);
    return SVDQ_OK;
}

int32_t check_quantizer(int64_t rows, int64_t K, const char *what) {
    return check_grid(i8_quantize_groups(rows, K), i8_quantize_threads(K), what);
}

int32_t check_shape(int32_t act, int64_t M, int64_t N, int64_t K) {
    SVDQ_TRY(check_rows(M, "M"));
    if (act != SVDQ_ACT_NONE && act != SVDQ_ACT_GELU)
        return fail(SVDQ_ERR_INVALID_ARG, "unknown activation %d", act);
    SVDQ_TRY(check_n(N));
    SVDQ_TRY(check_k_i8(K));
    if (M == 0) return SVDQ_OK;
    SVDQ_TRY(check_grid(i8_gemm_groups(M, N), 512, "the 8-bit GEMM"));
    return check_quantizer(M, K, "the 8-bit quantizer");
}

int32_t check_workspace(const void *ws, size_t ws_bytes, size_t need) {
    if (ws_bytes < need)
        return fail(SVDQ_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes < %zu needed", ws_bytes,
                    need);
    return need == 0 ? SVDQ_OK : need_ptr(ws, "workspace");
}

struct Workspace {
    int8_t *qa;
    float *sa;
    size_t bytes;
};

Workspace carve(void *base, int64_t M, int64_t K) {
    char *p = static_cast<char *>(base);
    Workspace w{};
    size_t off = 0;
    w.qa = reinterpret_cast<int8_t *>(p + off);
    off += align256((size_t)M * (size_t)K);
    w.sa = reinterpret_cast<float *>(p + off);
    off += align256((size_t)M * 4);
    w.bytes = off;
    return w;
}

// svdq_i8_linear's: a few tokens need none, their codes stay on the chip.
size_t linear_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N < 0 || K <= 0 || i8_few_tokens(M, N, K)) return 0;
    return carve(nullptr, M, K).bytes;
}

}  // namespace

extern "C" {

int32_t svdq_i8_pack_weights(const float *W, int64_t N, int64_t K, int8_t *qw, float *sw,
                             void *stream) {
    g_last_error[0] = 0;
    SVDQ_TRY(check_rows(N, "N"));
    SVDQ_TRY(check_k_i8(K));
    if (N == 0) return SVDQ_OK;
    SVDQ_TRY(check_quantizer(N, K, "the 8-bit packer"));
    SVDQ_TRY(need_ptr(W, "W"));
    SVDQ_TRY(need_ptr(qw, "qw"));
    SVDQ_TRY(need_ptr(sw, "sw"));
    SVDQ_TRY(check_device());
    return hip_status(launch_i8_quantize(W, true, nullptr, N, K, qw, sw, (hipStream_t)stream),
                      "i8_pack_weights launch");
}

int32_t svdq_i8_quantize_act(const uint16_t *X, const float *lambda, int64_t M, int64_t K,
                             int8_t *qa, float *sa, void *stream) {
    g_last_error[0] = 0;
    SVDQ_TRY(check_rows(M, "M"));
    SVDQ_TRY(check_k_i8(K));
    if (M == 0) return SVDQ_OK;
    SVDQ_TRY(check_quantizer(M, K, "the 8-bit quantizer"));
    SVDQ_TRY(need_ptr(X, "X"));
    if (lambda) SVDQ_TRY(need_ptr(lambda, "lambda"));
    SVDQ_TRY(need_ptr(qa, "qa"));
    SVDQ_TRY(need_ptr(sa, "sa"));
    SVDQ_TRY(check_device());
    return hip_status(launch_i8_quantize(X, false, lambda, M, K, qa, sa, (hipStream_t)stream),
                      "i8_quantize_act launch");
}

size_t svdq_i8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    (void)M, (void)N, (void)K;
    return 0;
}

int32_t svdq_i8_gemm(const int8_t *qa, const float *sa, const int8_t *qw, const float *sw,
                     const uint16_t *bias, int32_t act, int64_t M, int64_t N, int64_t K,
                     uint16_t *Y, void *workspace, size_t ws_bytes, void *stream) {
    g_last_error[0] = 0;
    SVDQ_TRY(check_shape(act, M, N, K));
    if (M == 0) return SVDQ_OK;
    SVDQ_TRY(need_ptr(qa, "qa"));
    SVDQ_TRY(need_ptr(sa, "sa"));
    SVDQ_TRY(need_ptr(qw, "qw"));
    SVDQ_TRY(need_ptr(sw, "sw"));
    SVDQ_TRY(need_ptr(Y, "Y"));
    if (bias) SVDQ_TRY(need_ptr(bias, "bias"));
    SVDQ_TRY(check_device());
    (void)workspace, (void)ws_bytes;
    return hip_status(launch_i8_gemm(qa, sa, qw, sw, bias, act, M, N, K, Y, (hipStream_t)stream),
                      "i8_gemm launch");
}

size_t svdq_i8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    return linear_workspace(M, N, K);
}

int32_t svdq_i8_linear(const uint16_t *X, const float *lambda, const int8_t *qw, const float *sw,
                       const uint16_t *bias, int32_t act, int64_t M, int64_t N, int64_t K,
                       uint16_t *Y, void *workspace, size_t ws_bytes, void *stream) {
    g_last_error[0] = 0;
    SVDQ_TRY(check_shape(act, M, N, K));
    if (M == 0) return SVDQ_OK;
    SVDQ_TRY(need_ptr(X, "X"));
    if (lambda) SVDQ_TRY(need_ptr(lambda, "lambda"));
    SVDQ_TRY(need_ptr(qw, "qw"));
    SVDQ_TRY(need_ptr(sw, "sw"));
    SVDQ_TRY(need_ptr(Y, "Y"));
    if (bias) SVDQ_TRY(need_ptr(bias, "bias"));
    SVDQ_TRY(check_workspace(workspace, ws_bytes, linear_workspace(M, N, K)));
    SVDQ_TRY(check_device());
    hipStream_t s = (hipStream_t)stream;
    if (i8_few_tokens(M, N, K))
        return hip_status(launch_i8_few(X, lambda, qw, sw, bias, act, M, N, K, Y, s),
                          "i8_linear launch");
    const Workspace w = carve(workspace, M, K);
    SVDQ_TRY(hip_status(launch_i8_quantize(X, false, lambda, M, K, w.qa, w.sa, s),
                        "i8_quantize_act launch"));
    return hip_status(launch_i8_gemm(w.qa, w.sa, qw, sw, bias, act, M, N, K, Y, s),
                      "i8_gemm launch");
}

}  // extern "C"
