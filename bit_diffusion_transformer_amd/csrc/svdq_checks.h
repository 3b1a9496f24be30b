// svdq_checks.h -- argument checks, the device check and the error text shared
// by the entry points (internal; not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "svdq.h"
#include "svdq_internal.h"

namespace svdq {

extern thread_local char g_last_error[512];   // detail of the thread's last error

inline int32_t fail(int32_t status, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return status;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Per-device cache of the architecture check: 0 unknown, 1 gfx950, 2 other.
constexpr int kMaxDevices = 64;
extern std::atomic<int> g_arch_ok[kMaxDevices];

inline int32_t check_device() {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || dev < 0)
        return fail(SVDQ_ERR_UNSUPPORTED_DEVICE, "no HIP device available (%s)",
                    hipGetErrorString(e));
    if (dev < kMaxDevices) {
        int v = g_arch_ok[dev].load(std::memory_order_relaxed);
        if (v == 1) return SVDQ_OK;
        if (v == 2) return fail(SVDQ_ERR_UNSUPPORTED_DEVICE, "device %d is not gfx950", dev);
    }
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess)
        return fail(SVDQ_ERR_UNSUPPORTED_DEVICE, "hipGetDeviceProperties failed: %s",
                    hipGetErrorString(e));
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < kMaxDevices) g_arch_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    if (!ok)
        return fail(SVDQ_ERR_UNSUPPORTED_DEVICE,
                    "device %d is %s; this library is built for gfx950 (MI355X) only", dev,
                    prop.gcnArchName);
    return SVDQ_OK;
}

inline int32_t hip_status(hipError_t e, const char *what) {
    if (e == hipSuccess) return SVDQ_OK;
    return fail(SVDQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline int32_t check_k(int64_t K) {
    if (K < SVDQ_GROUP || K % SVDQ_GROUP != 0)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "K must be a positive multiple of 64 (got %lld)",
                    (long long)K);
    if (K > SVDQ_MAX_K)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "K = %lld exceeds the limit %d", (long long)K,
                    SVDQ_MAX_K);
    return SVDQ_OK;
}

// Token and output-row counts: >= 0 (0: nothing to do) and within the limit.
inline int32_t check_rows(int64_t n, const char *name) {
    if (n < 0) return fail(SVDQ_ERR_INVALID_ARG, "%s must be >= 0 (got %lld)", name, (long long)n);
    if (n > SVDQ_MAX_ROWS)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "%s = %lld exceeds the limit %d", name,
                    (long long)n, SVDQ_MAX_ROWS);
    return SVDQ_OK;
}

// The MXFP4 variant: whole stages of two groups (128 values) along K.
inline int32_t check_k_mx(int64_t K) {
    if (K < 128 || K % 128 != 0)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE,
                    "K must be a positive multiple of 128 for MXFP4 (got %lld)", (long long)K);
    return check_k(K);
}

inline int32_t check_r(int32_t r) {
    if (r < 0 || r > SVDQ_MAX_RANK || r % 16 != 0)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE,
                    "rank r must be a multiple of 16 in [0, %d] (got %d)", SVDQ_MAX_RANK, r);
    return SVDQ_OK;
}

inline int32_t check_n(int64_t N) {
    if (N < 8 || N % 8 != 0)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "N must be a positive multiple of 8 (got %lld)",
                    (long long)N);
    return check_rows(N, "N");
}

// A launch's work-items (workgroups x threads) must fit the 32-bit grid size
// of a dispatch.  Shapes inside the row and K limits can still exceed it
// (e.g. 2^28 tokens with a wide N); they are rejected here rather than
// launched with a truncated grid.
inline int32_t check_grid(int64_t workgroups, int64_t threads, const char *what) {
    if (workgroups > (int64_t)0xFFFFFFFF / threads)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE,
                    "%s would need %lld workgroups of %lld threads, more than 2^32 - 1 work-items",
                    what, (long long)workgroups, (long long)threads);
    return SVDQ_OK;
}

#define SVDQ_TRY(expr)                       \
    do {                                     \
        int32_t _s = (expr);                 \
        if (_s != SVDQ_OK) return _s;        \
    } while (0)

inline int32_t need_ptr(const void *p, const char *name) {
    if (!p) return fail(SVDQ_ERR_INVALID_ARG, "%s must not be NULL", name);
    if (!aligned16(p)) return fail(SVDQ_ERR_MISALIGNED, "%s is not 16-byte aligned", name);
    return SVDQ_OK;
}

// need_gamma: the norm weights must be given (otherwise each may be NULL).
inline int32_t validate_qkv(const svdq_qkv_epilogue *e, int64_t M, bool need_gamma = true) {
    if (!e) return fail(SVDQ_ERR_INVALID_ARG, "epi must not be NULL");
    if (e->heads < 1) return fail(SVDQ_ERR_INVALID_ARG, "heads must be >= 1 (got %d)", e->heads);
    if (e->head_dim != 64 && e->head_dim != 128)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "head_dim must be 64 or 128 (got %d)",
                    e->head_dim);
    if (((int64_t)e->heads * e->head_dim) % 128 != 0)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "heads * head_dim must be a multiple of 128");
    if (e->seq < 1) return fail(SVDQ_ERR_INVALID_ARG, "seq must be >= 1");
    if (M % e->seq != 0)
        return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "M = %lld is not a multiple of seq = %lld",
                    (long long)M, (long long)e->seq);
    if (!(e->eps >= 0.0f) || e->eps > 3.0e38f)
        return fail(SVDQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (M == 0) return SVDQ_OK;
    if (need_gamma || e->gamma_q) SVDQ_TRY(need_ptr(e->gamma_q, "gamma_q"));
    if (need_gamma || e->gamma_k) SVDQ_TRY(need_ptr(e->gamma_k, "gamma_k"));
    SVDQ_TRY(need_ptr(e->cos_t, "cos_t"));
    SVDQ_TRY(need_ptr(e->sin_t, "sin_t"));
    SVDQ_TRY(need_ptr(e->q, "q"));
    SVDQ_TRY(need_ptr(e->k, "k"));
    return need_ptr(e->v, "v");
}

inline QkvArgs qkv_args(const svdq_qkv_epilogue *e) {
    QkvArgs a;
    a.H = e->heads;
    a.D = e->head_dim;
    a.S = e->seq;
    a.gq = e->gamma_q;
    a.gk = e->gamma_k;
    a.eps = e->eps;
    a.cos_t = e->cos_t;
    a.sin_t = e->sin_t;
    a.Q = e->q;
    a.K = e->k;
    a.V = e->v;
    return a;
}

}  // namespace svdq
