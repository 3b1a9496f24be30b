// i8_quantize.hip -- 8-bit row quantization: the activations' step (with
// optional smoothing) and the offline packing of the weights.
#include "i8_device.h"
#include "i8_internal.h"

namespace svdq {

using namespace i8;

namespace {

// The largest of `x` over the workgroup; `slot` alternates between calls, so
// that one barrier a call is enough.
template <int WAVES>
__device__ __forceinline__ float group_max(float x, float (*part)[WAVES], int slot) {
    x = wave_max(x);
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) x = larger(x, part[slot][w]);
    return x;
}

// One workgroup per `rows` consecutive rows; thread t holds the pieces of 8
// values at 8 (t + THREADS c), c < CH, of the row at hand in registers, so each
// row is read once, and the reciprocals of its smoothing factors across the
// rows (a correctly rounded division costs about as much as everything else
// here together).  The next row is loaded before the current one is reduced.
// Bound by memory: 2 bytes read and 1 written per element (4 and 1 for W).
// 4608 x 12288 with smoothing: 36 us, 4.7 TB/s; 333 x 4096: 3.5 us; weights of 16384 x
// 4096: 66 us, 5.1 TB/s.
template <int THREADS, int CH, bool F32, bool SMOOTH>
__global__ void __launch_bounds__(THREADS)
i8_quantize_kernel(const void *__restrict__ X, const float *__restrict__ lam, int64_t M, int64_t K,
                   int rows, int8_t *__restrict__ q, float *__restrict__ s) {
    __shared__ float part[2][THREADS / 64];
    const int64_t m0 = (int64_t)blockIdx.x * rows;
    const int64_t m1 = m0 + rows < M ? m0 + rows : M;
    Raw<F32> next[CH];
    float inv[SMOOTH ? CH : 1][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int k = 8 * ((int)threadIdx.x + THREADS * c);
        if (k < K) next[c] = load_raw<F32>(X, m0 * K + k);
    }
    if (SMOOTH)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * ((int)threadIdx.x + THREADS * c);
            if (k < K) load_inv(lam, k, inv[SMOOTH ? c : 0]);
        }
    for (int64_t m = m0; m < m1; ++m) {
        float v[CH][8], amax = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * ((int)threadIdx.x + THREADS * c);
            if (k < K) {
                values<F32>(next[c], v[c]);
                if (m + 1 < m1) next[c] = load_raw<F32>(X, (m + 1) * K + k);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (SMOOTH) v[c][j] *= inv[SMOOTH ? c : 0][j];
                    amax = larger(amax, fabsf(v[c][j]));
                }
            }
        }
        amax = group_max<THREADS / 64>(amax, part, (int)(m - m0) & 1);
        float r;
        const float scale = scale_of(amax, r);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = 8 * ((int)threadIdx.x + THREADS * c);
            if (k < K) *reinterpret_cast<u32x2 *>(q + m * K + k) = codes8(v[c], r);
        }
        if (threadIdx.x == 0) s[m] = scale;
    }
}

// Rows too long for the registers: the row is read twice (the second time mostly
// from the caches).
constexpr int kMaxRegisters = 16384;
constexpr int kLong = 512;

template <bool F32>
__global__ void __launch_bounds__(kLong)
i8_quantize_long_kernel(const void *__restrict__ X, const float *__restrict__ lam, int64_t K,
                        int8_t *__restrict__ q, float *__restrict__ s) {
    __shared__ float part[1][kLong / 64];
    const int64_t m = blockIdx.x;
    float amax = 0.0f, v[8], inv[8];
    auto load = [&](int k) {
        values<F32>(load_raw<F32>(X, m * K + k), v);
        if (lam) {
            load_inv(lam, k, inv);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= inv[j];
        }
    };
    for (int k = 8 * (int)threadIdx.x; k < K; k += 8 * kLong) {
        load(k);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = larger(amax, fabsf(v[j]));
    }
    amax = group_max<kLong / 64>(amax, part, 0);
    float r;
    const float scale = scale_of(amax, r);
    for (int k = 8 * (int)threadIdx.x; k < K; k += 8 * kLong) {
        load(k);
        *reinterpret_cast<u32x2 *>(q + m * K + k) = codes8(v, r);
    }
    if (threadIdx.x == 0) s[m] = scale;
}

// Rows per workgroup: the divisions of the smoothing are shared by up to four
// rows once there are workgroups enough to fill the chip without.
int rows_per_group(int64_t M) { return M >= 4096 ? 4 : M >= 2048 ? 2 : 1; }

template <int THREADS, int CH, bool F32>
void start(const void *X, const float *lam, int64_t M, int64_t K, int8_t *q, float *s,
           hipStream_t stream) {
    const int rows = rows_per_group(M);
    const unsigned grid = (unsigned)((M + rows - 1) / rows);
    if (!F32 && lam)
        i8_quantize_kernel<THREADS, CH, F32, !F32><<<grid, THREADS, 0, stream>>>(X, lam, M, K, rows, q, s);
    else
        i8_quantize_kernel<THREADS, CH, F32, false><<<grid, THREADS, 0, stream>>>(X, lam, M, K, rows, q, s);
}

// 256 threads up to K = 4096, then 512 (three pieces at K = 12288: the
// registers of a thread leave room for two workgroups per SIMD's waves).
template <bool F32>
hipError_t launch(const void *X, const float *lam, int64_t M, int64_t K, int8_t *q, float *s,
                  hipStream_t stream) {
    if (K <= 2048) start<256, 1, F32>(X, lam, M, K, q, s, stream);
    else if (K <= 4096) start<256, 2, F32>(X, lam, M, K, q, s, stream);
    else if (K <= 8192) start<512, 2, F32>(X, lam, M, K, q, s, stream);
    else if (K <= 12288) start<512, 3, F32>(X, lam, M, K, q, s, stream);
    else if (K <= kMaxRegisters) start<512, 4, F32>(X, lam, M, K, q, s, stream);
    else i8_quantize_long_kernel<F32><<<(unsigned)M, kLong, 0, stream>>>(X, lam, K, q, s);
    return hipGetLastError();
}

}  // namespace

int64_t i8_quantize_groups(int64_t M, int64_t K) {
    const int rows = K > kMaxRegisters ? 1 : rows_per_group(M);
    return (M + rows - 1) / rows;
}
int64_t i8_quantize_threads(int64_t K) { return K <= 4096 ? 256 : 512; }

hipError_t launch_i8_quantize(const void *X, bool fp32, const float *lambda, int64_t M, int64_t K,
                              int8_t *q, float *s, hipStream_t stream) {
    return fp32 ? launch<true>(X, nullptr, M, K, q, s, stream)
                : launch<false>(X, lambda, M, K, q, s, stream);
}

}  // namespace svdq
