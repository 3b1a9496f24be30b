// i8_device.h -- device helpers of the 8-bit linear's kernels (internal; not part
// of the ABI): the matrix instruction and its LDS layout, the row quantization.
#pragma once

#include "svdq_device.h"

namespace svdq {

namespace i8 {

constexpr int kRow = 128;        // bytes of a row per stage

typedef int i32x16 __attribute__((ext_vector_type(16)));

// 32x32 output tile, K = 32 int8 per call: lane l supplies 16 bytes of row /
// column l % 32, k half l / 32; output element i of lane l is row
// 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32.
__device__ __forceinline__ i32x16 mfma_i8_32x32x32(i32x4 a, i32x4 b, i32x16 c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

// The 16-byte segment s of a row sits at slot s ^ swz(row): any 8 consecutive
// rows of one segment touch 8 distinct slots (all banks of a 128-byte pass),
// any 16 consecutive rows 16 distinct 16-byte groups of 256 bytes.
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Eight consecutive values of a row as they are loaded (16 bytes of bf16, 32 of
// fp32), and as fp32.
template <bool F32>
struct Raw {
    u32x4 w[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw<F32> load_raw(const void *X, int64_t at) {
    Raw<F32> r;
    const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const char *>(X) + at * (F32 ? 4 : 2));
    r.w[0] = p[0];
    if (F32) r.w[F32 ? 1 : 0] = p[1];
    return r;
}

template <bool F32>
__device__ __forceinline__ void values(const Raw<F32> &r, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (F32) {
            v[j] = __uint_as_float(r.w[0][j]);
            v[4 + j] = __uint_as_float(r.w[F32 ? 1 : 0][j]);
        } else {
            v[2 * j] = bf16_lo(r.w[0][j]);
            v[2 * j + 1] = bf16_hi(r.w[0][j]);
        }
    }
}

__device__ __forceinline__ void load_inv(const float *lam, int k, float (&inv)[8]) {
    const f32x4 *p = reinterpret_cast<const f32x4 *>(lam + k);
    const f32x4 x = p[0], y = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        inv[j] = 1.0f / x[j];
        inv[4 + j] = 1.0f / y[j];
    }
}

// rint(fl32(v inv)) as the low byte of v inv + 1.5 * 2^23 (the addition rounds
// to the nearest integer, ties to even, for |v inv| < 2^22).
__device__ __forceinline__ uint32_t code8(float v, float inv) {
    return __float_as_uint(v * inv + 12582912.0f);
}

__device__ __forceinline__ u32x2 codes8(const float (&v)[8], float inv) {
    u32x2 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t ab = __builtin_amdgcn_perm(code8(v[4 * h + 1], inv), code8(v[4 * h], inv), 0x0C0C0400);
        const uint32_t cd = __builtin_amdgcn_perm(code8(v[4 * h + 3], inv), code8(v[4 * h + 2], inv), 0x04000C0C);
        out[h] = ab | cd;
    }
    return out;
}

// The larger of two magnitudes; a NaN stays one (and the row's outputs with it).
__device__ __forceinline__ float larger(float x, float y) { return __builtin_elementwise_maximum(x, y); }

// The largest x of the wave, every lane getting it: lane exchanges within 16
// lanes, then the swaps with the lanes 16 and 32 away.
__device__ __forceinline__ float wave_max(float x) {
    auto with = [&](int y) { x = larger(x, __int_as_float(y)); };
    with(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xF, 0xF, true));    // lane ^ 1
    with(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xF, 0xF, true));    // lane ^ 2
    with(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x141, 0xF, 0xF, true));   // 7 - lane
    with(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x140, 0xF, 0xF, true));   // 15 - lane
    const uint32_t u = __float_as_uint(x);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    x = larger(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const uint32_t v = __float_as_uint(x);
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return larger(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// A NaN or an infinity in the row: not finite either, with all-zero codes (inv is 0,
// and a NaN's code8 is 0), so the outputs are 0 times the scale, NaN.
__device__ __forceinline__ float scale_of(float amax, float &inv) {
    const float s = amax / 127.0f;
    inv = 0.0f;
    if (s != 0.0f) {
        const float t = 1.0f / s;
        inv = __builtin_isfinite(t) ? t : 0.0f;
    }
    return s;
}

}  // namespace i8

}  // namespace svdq
