// i8_quantize.hip -- 8-bit row quantization: the activations' step (with
// optional smoothing) and the offline packing of the weights.
#include "i8_internal.h"
#include "svdq_device.h"

namespace svdq {

namespace {

constexpr int kThreads = 256;

// Eight consecutive values of a row, as fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void *X, int64_t at, float (&v)[8]) {
    if (F32) {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(static_cast<const float *>(X) + at);
        const f32x4 a = p[0], b = p[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
        const u32x4 x = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(X) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_lo(x[j]);
            v[2 * j + 1] = bf16_hi(x[j]);
        }
    }
}

__device__ __forceinline__ void load_inv(const float *lam, int k, float (&inv)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) inv[j] = lam ? 1.0f / lam[k + j] : 1.0f;
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

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor(x, d));
    return x;
}

// The largest of `x` over the workgroup; `slot` alternates between calls, so
// that one barrier a call is enough.
__device__ __forceinline__ float group_max(float x, float (*part)[kThreads / 64], int slot) {
    x = wave_max(x);
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = x;
    __syncthreads();
    return fmaxf(fmaxf(part[slot][0], part[slot][1]), fmaxf(part[slot][2], part[slot][3]));
}

__device__ __forceinline__ float scale_of(float amax, float &inv) {
    const float s = amax / 127.0f;
    inv = 0.0f;
    if (s != 0.0f) {
        const float t = 1.0f / s;
        inv = __builtin_isfinite(t) ? t : 0.0f;
    }
    return s;
}

// One workgroup per `rows` consecutive rows; thread t holds the pieces of 8
// values at 8 (t + 256 c), c < CH, of the row at hand in registers, so each
// row is read once, and the reciprocals of its smoothing factors across the
// rows (a correctly rounded division costs about as much as everything else
// here together).  The next row is loaded before the current one is reduced.
// Bound by memory: 2 bytes read and 1 written per element (4 and 1 for W).
template <int CH, bool F32>
__global__ void __launch_bounds__(kThreads)
i8_quantize_kernel(const void *__restrict__ X, const float *__restrict__ lam, int64_t M, int64_t K,
                   int rows, int8_t *__restrict__ q, float *__restrict__ s) {
    __shared__ float part[2][kThreads / 64];
    const int64_t m0 = (int64_t)blockIdx.x * rows;
    const int64_t m1 = m0 + rows < M ? m0 + rows : M;
    float inv[CH][8], next[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int k = 8 * ((int)threadIdx.x + kThreads * c);
        if (k < K) {
            load8<F32>(X, m0 * K + k, next[c]);
            if (!F32) load_inv(lam, k, inv[c]);
        }
    }
    for (int64_t m = m0; m < m1; ++m) {
        float v[CH][8], amax = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * ((int)threadIdx.x + kThreads * c);
            if (k < K) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[c][j] = F32 ? next[c][j] : next[c][j] * inv[c][j];
                    amax = fmaxf(amax, fabsf(v[c][j]));
                }
                if (m + 1 < m1) load8<F32>(X, (m + 1) * K + k, next[c]);
            }
        }
        amax = group_max(amax, part, (int)(m - m0) & 1);
        float r;
        const float scale = scale_of(amax, r);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * ((int)threadIdx.x + kThreads * c);
            if (k < K) *reinterpret_cast<u32x2 *>(q + m * K + k) = codes8(v[c], r);
        }
        if (threadIdx.x == 0) s[m] = scale;
    }
}

// Rows too long for the registers: the row is read twice (the second time
// mostly from the caches).
template <bool F32>
__global__ void __launch_bounds__(kThreads)
i8_quantize_long_kernel(const void *__restrict__ X, const float *__restrict__ lam, int64_t K,
                        int8_t *__restrict__ q, float *__restrict__ s) {
    __shared__ float part[1][kThreads / 64];
    const int64_t m = blockIdx.x;
    float amax = 0.0f, v[8], inv[8];
    for (int k = 8 * (int)threadIdx.x; k < K; k += 8 * kThreads) {
        load8<F32>(X, m * K + k, v);
        if (!F32) load_inv(lam, k, inv);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(F32 ? v[j] : v[j] * inv[j]));
    }
    amax = group_max(amax, part, 0);
    float r;
    const float scale = scale_of(amax, r);
    for (int k = 8 * (int)threadIdx.x; k < K; k += 8 * kThreads) {
        load8<F32>(X, m * K + k, v);
        if (!F32) {
            load_inv(lam, k, inv);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= inv[j];
        }
        *reinterpret_cast<u32x2 *>(q + m * K + k) = codes8(v, r);
    }
    if (threadIdx.x == 0) s[m] = scale;
}

// Rows per workgroup: the divisions of the smoothing are shared by up to four
// rows once there are workgroups enough to fill the chip without.
int rows_per_group(int64_t M) { return M >= 4096 ? 4 : M >= 2048 ? 2 : 1; }

template <bool F32>
hipError_t launch(const void *X, const float *lam, int64_t M, int64_t K, int8_t *q, float *s,
                  hipStream_t stream) {
    const int pieces = (int)((K / 8 + kThreads - 1) / kThreads);
    if (pieces > 8) {
        i8_quantize_long_kernel<F32><<<(unsigned)M, kThreads, 0, stream>>>(X, lam, K, q, s);
        return hipGetLastError();
    }
    const int rows = rows_per_group(M);
    const unsigned grid = (unsigned)((M + rows - 1) / rows);
    if (pieces == 1)
        i8_quantize_kernel<1, F32><<<grid, kThreads, 0, stream>>>(X, lam, M, K, rows, q, s);
    else if (pieces == 2)
        i8_quantize_kernel<2, F32><<<grid, kThreads, 0, stream>>>(X, lam, M, K, rows, q, s);
    else if (pieces <= 4)
        i8_quantize_kernel<4, F32><<<grid, kThreads, 0, stream>>>(X, lam, M, K, rows, q, s);
    else
        i8_quantize_kernel<8, F32><<<grid, kThreads, 0, stream>>>(X, lam, M, K, rows, q, s);
    return hipGetLastError();
}

}  // namespace

int64_t i8_quantize_groups(int64_t M, int64_t K) { return M; }

hipError_t launch_i8_quantize(const void *X, bool fp32, const float *lambda, int64_t M, int64_t K,
                              int8_t *q, float *s, hipStream_t stream) {
    return fp32 ? launch<true>(X, nullptr, M, K, q, s, stream)
                : launch<false>(X, lambda, M, K, q, s, stream);
}

}  // namespace svdq
