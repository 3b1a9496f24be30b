// svdq_wave.h -- device helpers of the 8-bit GEMM and the attention kernels
// (internal; not part of the ABI).
#pragma once

#include "svdq_device.h"

namespace svdq {

// Consecutive workgroups go to the 8 XCDs in turn.  The b-th of n, mapped so that
// each XCD gets a contiguous range, whose operands its L2 then holds.
__device__ __forceinline__ int64_t xcd_range(int64_t b, int64_t n) {
    const int64_t x = b & 7, q = n >> 3, r = n & 7;
    return x * q + (x < r ? x : r) + (b >> 3);
}

// 16 bytes per lane from global memory straight into LDS: lane l's bytes go to
// dst + 16 l (dst uniform).  (A function of its own, not a template: the host
// pass drops a kernel template that names this builtin.)
__device__ __forceinline__ void copy16_to_lds(const void *src, void *dst) {
    __builtin_amdgcn_global_load_lds(src, (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

// Workgroup barrier without a memory fence: copies into other buffers stay in
// flight across it.  The clobber keeps LDS accesses on their side.
__device__ __forceinline__ void wave_barrier_all() { asm volatile("s_barrier" ::: "memory"); }

// At most `n` vector-memory instructions of this wave in flight, and all its
// LDS reads returned (gfx9 s_waitcnt: vmcnt[3:0], expcnt[6:4], lgkmcnt[11:8],
// vmcnt[5:4] << 14).
template <int n>
__device__ __forceinline__ void wait_loads() {
    static_assert(n >= 0 && n < 64, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt((n & 0xF) | ((n >> 4) << 14) | (0x7 << 4));
}

// GELU, erf form, with one hardware exponential and no reciprocal:
//   GELU(x) = max(x, 0) - |x| h(|x|),  h(a) = erfc(a / sqrt 2) / 2 = 2^P(a).
// log2 h is smooth (it falls like -a^2 log2(e) / 2 with a slowly varying rest),
// so a polynomial of degree 6 with P(0) = -1, fitted for the least absolute
// error of h over 0 .. 6.5, leaves |error| <= 1.5e-7 |x| (evaluated in fp32
// against the 64-bit form over -9 .. 9), below that of the rational erf at two
// thirds of its issue cycles.  Past |x| = 8, where h < 2^-50, |x| is held there.
__device__ __forceinline__ float gelu_exp2(float x) {
    const float a = __builtin_elementwise_minimum(fabsf(x), 8.0f);   // a NaN stays one
    float p = __builtin_fmaf(a, 1.7755859516910277e-05f, -0.0006477624410763383f);
    p = __builtin_fmaf(a, p, 0.0077240546233952045f);
    p = __builtin_fmaf(a, p, -0.05292674899101257f);
    p = __builtin_fmaf(a, p, -0.4590827226638794f);
    p = __builtin_fmaf(a, p, -1.1511168479919434f);
    p = __builtin_fmaf(a, p, -1.0f);
    return __builtin_fmaf(-a, __builtin_amdgcn_exp2f(p), fmaxf(x, 0.0f));
}

}  // namespace svdq
