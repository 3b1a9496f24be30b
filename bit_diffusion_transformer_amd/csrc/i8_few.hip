// i8_few.hip -- the whole 8-bit linear in one launch for a few tokens: each
// workgroup quantizes the tokens itself and streams its own rows of weights.
//
// For a few tokens the layer is the weights' bytes and the time to start: a
// quantizer's launch and its codes' way through memory cost more than its work,
// which every workgroup can do while its first weights are on their way.  Bound by
// the weights' bytes: 1 token, 4096 -> 24576: 20.3 us (quantizer and GEMM in two
// launches: 24.7), 5.0 TB/s; 4096 -> 4096: 7.7 (10.1); 1024 -> 1024: 3.8 (7.2).
// 12 KB of a wave's ring leave room for three workgroups per compute unit (16 KB:
// 22.9 us, 8 KB: 19.9 but 17.1 instead of 16.2 for 4096 -> 16384).
#include "i8_device.h"
#include "i8_internal.h"
#include "svdq_wave.h"

namespace svdq {

namespace i8 {

constexpr int kFewWaves = 4;                     // share K, a stage each in turn
constexpr int kFewPieces = 8;                    // of 8 values, that a thread quantizes, at most
constexpr int kFewThreads = 64 * kFewWaves;

// A workgroup's channels; a wave's stages in flight at most, and their copies.
template <int ROWS_>
struct Few {
    static constexpr int ROWS = ROWS_;
    static constexpr int RING = 96 / ROWS;
    static constexpr int COPIES = ROWS / 8;      // 1 KB each
    static constexpr int STAGE = ROWS * kRow;
};

// LDS: a ring per wave, of as many stages as it has up to RING (4 KB at least, for
// its sums); codes [M][K up to whole stages]; the pieces' maxima.
__host__ __device__ inline int few_stages(int64_t K) { return (int)((K + kRow - 1) / kRow); }
template <class T>
__host__ __device__ inline int few_ring(int64_t K) {
    const int n = (few_stages(K) + kFewWaves - 1) / kFewWaves;
    return n < T::RING ? n : T::RING;
}
template <class T>
__host__ __device__ inline int few_ring_bytes(int64_t K) {
    const int n = few_ring<T>(K) * T::STAGE;
    return n > 4096 ? n : 4096;
}
template <class T>
inline size_t few_lds(int64_t M, int64_t K) {
    return (size_t)kFewWaves * few_ring_bytes<T>(K) + (size_t)M * few_stages(K) * kRow +
           kFewPieces * kFewWaves * 4;
}

// Waits until at most `younger` stages (up to N) of a wave are in flight.
template <int N, int COPIES>
__device__ __forceinline__ void wait_stage(int younger) {
    if (N == 0 || younger >= N) wait_loads<N * COPIES>();
    else wait_stage<(N > 0 ? N - 1 : 0), COPIES>(younger);
}

// Channels are the rows of one 32 x 32 block (rows past ROWS repeat the first
// ones), tokens its columns (those past M repeat the last one).  A wave's ring
// holds its own stages of the weights: no barrier in the loop over K, only waits
// for its own copies.
template <class T, bool SMOOTH, int PIECES>
__global__ void __launch_bounds__(kFewThreads)
i8_few_kernel(const uint16_t *__restrict__ X, const float *__restrict__ lam,
              const int8_t *__restrict__ qw, const float *__restrict__ sw,
              const uint16_t *__restrict__ bias, int act, int M, int64_t N, int K,
              uint16_t *__restrict__ Y) {
    extern __shared__ __align__(1024) uint8_t few[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * T::ROWS;
    const int depth = few_ring<T>(K), ring_bytes = few_ring_bytes<T>(K);
    const int row_bytes = few_stages(K) * kRow;
    uint8_t *const ring = few + wave * ring_bytes;
    uint8_t *const codes = few + kFewWaves * ring_bytes;
    float *const part = reinterpret_cast<float *>(codes + M * row_bytes);   // [piece][wave]

    // What the first wave scales its sums with, then the tokens' pieces (P of 8
    // values a row and thread), then the weights: loads return in order.
    const int h = lane >> 5;
    f32x4 ch_scale[T::COPIES];
    u32x2 ch_bias[T::COPIES];
    if (wave == 0)
#pragma unroll
        for (int q = 0; q < T::COPIES; ++q) {                // N % 8 == 0: four channels in or out
            int64_t n = n0 + 8 * q + 4 * h;
            n = n < N ? n : N - 4;
            ch_scale[q] = *reinterpret_cast<const f32x4 *>(sw + n);
            ch_bias[q] = bias ? *reinterpret_cast<const u32x2 *>(bias + n) : u32x2{};
        }
    const int P = (K + 8 * kFewThreads - 1) / (8 * kFewThreads);
    const int pieces = M * P;                        // <= kFewPieces
    // f(c, row, k) over the thread's pieces: values k .. k + 7 of row.  Pieces past
    // the count repeat the last one, values past K are zero.
    auto each = [&](auto f) __attribute__((always_inline)) {
        int row = 0, at = 0;
#pragma unroll
        for (int c = 0; c < PIECES; ++c) {
            f(c, row, 8 * ((int)threadIdx.x + kFewThreads * at));
            if (c + 1 < pieces && ++at == P) at = 0, ++row;
        }
    };
    Raw<false> raw[PIECES];
    Raw<true> factors[SMOOTH ? PIECES : 1];
    each([&](int c, int row, int k) __attribute__((always_inline)) {
        const int in = k < K ? k : 0;
        raw[c] = load_raw<false>(X, (int64_t)row * K + in);
        if (SMOOTH) factors[SMOOTH ? c : 0] = load_raw<true>(lam, in);
    });
    asm volatile("" ::: "memory");                   // the copies stay behind them

    // Copies of a stage: 8 rows each, lane l carries row l / 8 into slot l % 8.
    // Rows past N re-read the last one (never stored); the second half of a stage
    // of 64 bytes re-reads the first (left out below).
    const int nf = K / kRow, ns = nf + ((K & 64) ? 1 : 0);
    const int8_t *w0 = qw + n0 * K;
    const int64_t left = N - n0;
    auto issue = [&](int s, int slot) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < T::COPIES; ++i) {
            const int row = 8 * i + lane / 8;
            int seg = (lane & 7) ^ swz(row);
            if (s == nf) seg &= 3;
            const int r = row < left ? row : (int)left - 1;
            copy16_to_lds(w0 + (int64_t)r * K + (int64_t)s * kRow + 16 * seg,
                          ring + slot * T::STAGE + i * 1024);
        }
    };
#pragma unroll
    for (int i = 0; i < T::RING; ++i) {              // past the end: the last one, not used
        const int s = wave + kFewWaves * i;
        if (i < depth) issue(s < ns ? s : ns - 1, i);
    }

    // Values, their maxima, the codes
    auto value = [&](int c, float (&v)[8]) __attribute__((always_inline)) {
        values<false>(raw[c], v);
        if (SMOOTH) {
            float f[8];
            values<true>(factors[SMOOTH ? c : 0], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= 1.0f / f[j];
        }
    };
    float v[SMOOTH ? PIECES : 1][8], top[PIECES];
    each([&](int c, int, int k) __attribute__((always_inline)) {
        value(c, v[SMOOTH ? c : 0]);
        top[c] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top[c] = larger(top[c], fabsf(v[SMOOTH ? c : 0][j]));
        top[c] = wave_max(k < K ? top[c] : 0.0f);
    });
    if (lane == 0)
#pragma unroll
        for (int c = 0; c < PIECES; ++c) part[c * kFewWaves + wave] = top[c];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // copies stay in flight
    auto row_scale = [&](int row, float &inv) __attribute__((always_inline)) {
        float top = 0.0f;
        for (int i = row * P; i < (row + 1) * P; ++i) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(part + i * kFewWaves);
            top = larger(larger(larger(x.x, x.y), larger(x.z, x.w)), top);
        }
        return scale_of(top, inv);
    };
    float inv = 0.0f;
    int of = -1;                                     // the row that `inv` is of
    each([&](int c, int row, int k) __attribute__((always_inline)) {
        if (row != of) row_scale(row, inv), of = row;
        if (k < K) {
            if (!SMOOTH) value(c, v[0]);
            *reinterpret_cast<u32x2 *>(codes + row * row_bytes + k / kRow * kRow +
                                       16 * ((k / 16 % 8) ^ swz(row)) + k % 16) =
                codes8(v[SMOOTH ? c : 0], inv);
        }
    });
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

    const int token = (lane & 31) < M ? lane & 31 : M - 1;
    const int channel = lane & (T::ROWS - 1);
    const uint8_t *const b_row = codes + token * row_bytes, *const a_row = ring + channel * kRow;
    const int a_swz = swz(channel), b_swz = swz(token);
    i32x16 acc = {};
    for (int slot = 0, s = wave; s < ns; slot = slot + 1 < depth ? slot + 1 : 0, s += kFewWaves) {
        // this stage has landed when at most the younger ones remain in flight
        const int younger = (ns - 1 - s) / kFewWaves;
        wait_stage<T::RING - 1, T::COPIES>(younger);
        asm volatile("" ::: "memory");
        const uint8_t *a_st = a_row + slot * T::STAGE, *b_st = b_row + s * kRow;
        i32x4 a[4], b[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            a[kk] = *reinterpret_cast<const i32x4 *>(a_st + 16 * ((2 * kk + h) ^ a_swz));
            b[kk] = *reinterpret_cast<const i32x4 *>(b_st + 16 * ((2 * kk + h) ^ b_swz));
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the slot is refilled
        if (younger >= T::RING) issue(s + kFewWaves * T::RING, slot);
        acc = mfma_i8_32x32x32(a[0], b[0], acc);
        acc = mfma_i8_32x32x32(a[1], b[1], acc);
        if (s < nf) {
            acc = mfma_i8_32x32x32(a[2], b[2], acc);
            acc = mfma_i8_32x32x32(a[3], b[3], acc);
        }
    }
    // The waves' sums, through their own rings (a wave without a stage still has its
    // first copies on their way there); the first wave scales and stores.
    wait_loads<0>();
    asm volatile("" ::: "memory");
    if (wave > 0)
#pragma unroll
        for (int q = 0; q < T::COPIES; ++q)
            *reinterpret_cast<i32x4 *>(ring + q * 1024 + lane * 16) =
                i32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    __syncthreads();
    if (wave > 0) return;
    const float sa = row_scale(token, inv);
#pragma unroll
    for (int q = 0; q < T::COPIES; ++q) {
        const int64_t n = n0 + 8 * q + 4 * h;
        i32x4 sum = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w)
            sum += *reinterpret_cast<const i32x4 *>(ring + w * ring_bytes + q * 1024 + lane * 16);
        if ((lane & 31) < M && n < N) {
            const float add[4] = {bf16_lo(ch_bias[q].x), bf16_hi(ch_bias[q].x), bf16_lo(ch_bias[q].y),
                                  bf16_hi(ch_bias[q].y)};
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = (float)sum[e] * (sa * ch_scale[q][e]) + add[e];
                if (act) y[e] = gelu_exp2(y[e]);
            }
            *reinterpret_cast<u32x2 *>(Y + token * N + n) =
                u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
        }
    }
}

}  // namespace i8

using namespace i8;

static int64_t few_pieces(int64_t M, int64_t K) {
    return M * ((K + 8 * kFewThreads - 1) / (8 * kFewThreads));
}

// Up to two pieces a thread, or four while there are few channels to repeat them
// for: 4 tokens, 2048 -> 4096: 7.0 us here, 8.2 in two launches, but 1024 -> 24576 with
// smoothing 11.9 and 11.1.  Eight pieces where few channels meet a long K, whose
// codes are long in a second launch: 2 tokens, 8192 -> 4096: 12.1 and 14.6, but 8
// tokens, 2048 -> 4096: 9.2 and 8.5.
bool i8_few_tokens(int64_t M, int64_t N, int64_t K) {
    return few_pieces(M, K) <= (N > 8192 ? 2 : N <= 4096 && K > 4096 ? kFewPieces : 4);
}

template <class T, int PIECES>
static void start_few(const uint16_t *X, const float *lambda, const int8_t *qw, const float *sw,
                      const uint16_t *bias, int act, int64_t M, int64_t N, int64_t K, uint16_t *Y,
                      hipStream_t stream) {
    const unsigned grid = (unsigned)((N + T::ROWS - 1) / T::ROWS);
    auto *f = lambda ? i8_few_kernel<T, true, PIECES> : i8_few_kernel<T, false, PIECES>;
    f<<<grid, kFewThreads, few_lds<T>(M, K), stream>>>(X, lambda, qw, sw, bias, act, (int)M, N, (int)K, Y);
}

hipError_t launch_i8_few(const uint16_t *X, const float *lambda, const int8_t *qw, const float *sw,
                         const uint16_t *bias, int act, int64_t M, int64_t N, int64_t K,
                         uint16_t *Y, hipStream_t stream) {
    const int64_t pieces = few_pieces(M, K);
    auto go = [&](auto t) {
        typedef decltype(t) T;
        auto *f = pieces == 1 ? start_few<T, 1> : pieces == 2 ? start_few<T, 2> : start_few<T, 4>;
        f(X, lambda, qw, sw, bias, act, M, N, K, Y, stream);
        return hipGetLastError();
    };
    if (pieces > 4) {
        start_few<Few<16>, kFewPieces>(X, lambda, qw, sw, bias, act, M, N, K, Y, stream);
        return hipGetLastError();
    }
    // A compute unit streams at most 24 GB/s from memory, so few channels are spread
    // over more of them; more workgroups repeat the quantization, and more pieces of
    // it.  One token, 8 | 16 | 32 channels a workgroup: 1024 -> 1024 3.8 | 4.1 | 4.8 us,
    // 8192 -> 2048 10.5 | 9.4 | 9.7, 8192 -> 4096 13.6 | 10.7 | 13.3, 4096 -> 12288 17.6 |
    // 15.1 | 13.6; 8192 -> 8192 24.2 | 16.1 | 18.8; four tokens, 320 -> 8192 10.1 | 7.4 | 6.4.
    if (N <= 2048 && K <= 2048) return go(Few<8>());
    return N <= (pieces <= 2 || K > 4096 ? 8192 : 4096) ? go(Few<16>()) : go(Few<32>());
}

}  // namespace svdq
