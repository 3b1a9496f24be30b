// i8_few.hip -- the whole 8-bit linear in one launch for a few tokens: each
// workgroup quantizes the tokens itself and streams its own rows of weights.
//
// For a few tokens the layer is the weights' bytes and the time to start: a
// quantizer's launch and its codes' way through memory cost more than its work,
// which every workgroup can do while its first weights are on their way.  Bound by
// the weights' bytes: 1 token, 4096 -> 24576: 20.3 us (quantizer and GEMM in two
// launches: 24.7), 5.0 TB/s; 4096 -> 4096: 7.7 (10.1); 1472 -> 4528: 5.7 (7.9).
// Three stages of the ring leave room for three workgroups per compute unit (four:
// 22.9 us, two: 19.9 but 17.1 instead of 16.2 for 4096 -> 16384).
#include "i8_device.h"
#include "i8_internal.h"
#include "svdq_wave.h"

namespace svdq {

namespace i8 {

constexpr int kFewRows = 32;                     // channels per workgroup
constexpr int kFewWaves = 4;                     // share K, a stage each in turn
constexpr int kFewRing = 3;                      // stages of a wave in flight, at most
constexpr int kFewStage = kFewRows * kRow;       // 4 KB: four copies
constexpr int kFewPieces = 4;                    // of 8 values, that a thread quantizes, at most
constexpr int kFewThreads = 64 * kFewWaves;

// LDS: a ring per wave, of as many stages as it has up to kFewRing; codes [M][K up
// to whole stages]; the pieces' maxima.
__host__ __device__ inline int few_stages(int64_t K) { return (int)((K + kRow - 1) / kRow); }
__host__ __device__ inline int few_ring(int64_t K) {
    const int n = (few_stages(K) + kFewWaves - 1) / kFewWaves;
    return n < kFewRing ? n : kFewRing;
}
__host__ __device__ inline int few_codes_at(int64_t K) { return kFewWaves * few_ring(K) * kFewStage; }
inline size_t few_lds(int64_t M, int64_t K) {
    return (size_t)few_codes_at(K) + (size_t)M * few_stages(K) * kRow + kFewPieces * kFewWaves * 4;
}

// Tokens are the columns of one 32 x 32 block (columns past M repeat the last
// one).  A wave's ring holds its own stages of the weights: no barrier in the
// loop over K, only waits for its own copies.
template <bool SMOOTH, int PIECES>
__global__ void __launch_bounds__(kFewThreads)
i8_few_kernel(const uint16_t *__restrict__ X, const float *__restrict__ lam,
              const int8_t *__restrict__ qw, const float *__restrict__ sw,
              const uint16_t *__restrict__ bias, int act, int M, int64_t N, int K,
              uint16_t *__restrict__ Y) {
    extern __shared__ __align__(1024) uint8_t few[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * kFewRows;
    const int depth = few_ring(K), row_bytes = few_stages(K) * kRow;
    uint8_t *const ring = few + wave * depth * kFewStage;
    uint8_t *const codes = few + few_codes_at(K);
    float *const part = reinterpret_cast<float *>(codes + M * row_bytes);   // [piece][wave]

    // What the first wave scales its sums with, then the tokens' pieces (P of 8
    // values a row and thread), then the weights: loads return in order.
    const int h = lane >> 5;
    f32x4 ch_scale[4];
    u32x2 ch_bias[4];
    if (wave == 0)
#pragma unroll
        for (int q = 0; q < 4; ++q) {                // N % 8 == 0: four channels in or out
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
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + lane / 8;
            int seg = (lane & 7) ^ swz(row);
            if (s == nf) seg &= 3;
            const int r = row < left ? row : (int)left - 1;
            copy16_to_lds(w0 + (int64_t)r * K + (int64_t)s * kRow + 16 * seg,
                          ring + slot * kFewStage + i * 1024);
        }
    };
#pragma unroll
    for (int i = 0; i < kFewRing; ++i) {             // past the end: the last one, not used
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
        for (int j = 0; j < 8; ++j) top[c] = fmaxf(top[c], fabsf(v[SMOOTH ? c : 0][j]));
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
            top = fmaxf(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)), top);
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
    const uint8_t *const b_row = codes + token * row_bytes, *const a_row = ring + (lane & 31) * kRow;
    const int a_swz = swz(lane & 31), b_swz = swz(token);
    i32x16 acc = {};
    for (int slot = 0, s = wave; s < ns; slot = slot + 1 < depth ? slot + 1 : 0, s += kFewWaves) {
        // this stage has landed when at most the younger ones remain in flight
        const int younger = (ns - 1 - s) / kFewWaves;
        if (younger >= 2) wait_loads<8>();
        else if (younger == 1) wait_loads<4>();
        else wait_loads<0>();
        asm volatile("" ::: "memory");
        const uint8_t *a_st = a_row + slot * kFewStage, *b_st = b_row + s * kRow;
        i32x4 a[4], b[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            a[kk] = *reinterpret_cast<const i32x4 *>(a_st + 16 * ((2 * kk + h) ^ a_swz));
            b[kk] = *reinterpret_cast<const i32x4 *>(b_st + 16 * ((2 * kk + h) ^ b_swz));
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the slot is refilled
        if (younger >= kFewRing) issue(s + kFewWaves * kFewRing, slot);
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
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<i32x4 *>(ring + q * 1024 + lane * 16) =
                i32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    __syncthreads();
    if (wave > 0) return;
    const float sa = row_scale(token, inv);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + 8 * q + 4 * h;
        i32x4 sum = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w)
            sum += *reinterpret_cast<const i32x4 *>(ring + w * depth * kFewStage + q * 1024 + lane * 16);
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

// Up to two pieces a thread, or four while every compute unit has one workgroup at
// most: 4 tokens, 1024 -> 8192: 7.0 us here, 8.0 in two launches, but -> 24576 with
// smoothing 11.9 and 11.1; eight pieces, 8 tokens, 2048 -> 4096: 9.2 and 8.5.
bool i8_few_tokens(int64_t M, int64_t N, int64_t K) {
    return few_pieces(M, K) <= (N <= 8192 ? kFewPieces : 2);
}

template <int PIECES>
static void start_few(const uint16_t *X, const float *lambda, const int8_t *qw, const float *sw,
                      const uint16_t *bias, int act, int64_t M, int64_t N, int64_t K, uint16_t *Y,
                      hipStream_t stream) {
    const unsigned grid = (unsigned)((N + kFewRows - 1) / kFewRows);
    auto *f = lambda ? i8_few_kernel<true, PIECES> : i8_few_kernel<false, PIECES>;
    f<<<grid, kFewThreads, few_lds(M, K), stream>>>(X, lambda, qw, sw, bias, act, (int)M, N, (int)K, Y);
}

hipError_t launch_i8_few(const uint16_t *X, const float *lambda, const int8_t *qw, const float *sw,
                         const uint16_t *bias, int act, int64_t M, int64_t N, int64_t K,
                         uint16_t *Y, hipStream_t stream) {
    const int64_t pieces = few_pieces(M, K);
    auto *f = pieces == 1 ? start_few<1> : pieces == 2 ? start_few<2> : start_few<4>;
    f(X, lambda, qw, sw, bias, act, M, N, K, Y, stream);
    return hipGetLastError();
}

}  // namespace svdq
