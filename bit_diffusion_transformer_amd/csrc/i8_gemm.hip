// i8_gemm.hip -- Y = act(diag(sa) (qa qw^T) diag(sw) + bias) on the 8-bit
// integer matrix instruction (v_mfma_i32_32x32x32_i8).
//
// Output tiles are computed transposed, D[n][m] = S[m][n]: the weight codes
// are the A operand and the activation codes the B operand, so that an output
// lane holds four consecutive n of one token row.  Both operands are [rows,
// K] bytes, and a stage of the K loop is 128 of them: one cache line per row.
// Lines go straight into a ring in LDS (global_load_lds, no registers), each
// wave reads its fragments with 16-byte LDS reads (XOR-swizzled, no bank
// conflicts), and the integer sums stay in registers over the whole K loop
// (exact: K <= 2^17).  The epilogue scales in fp32, adds the bias, applies
// the activation and rounds once.
#include "i8_internal.h"
#include "svdq_wave.h"

#include <type_traits>

namespace svdq {

namespace i8 {

constexpr int kRow = 128;        // bytes of a row per stage
constexpr int kGroupM = 8;       // m tiles per raster group (L2 reuse of weights)

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

template <int BM_, int BN_, int WM_, int WN_, int NBUF_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_;          // tokens, output channels
    static constexpr int WM = WM_, WN = WN_;          // waves along each
    static constexpr int NBUF = NBUF_;                // stages in the ring
    static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    static constexpr int MB = BM / WM / 32, NB = BN / WN / 32;   // 32 x 32 blocks per wave
    static constexpr int STAGE = (BM + BN) * kRow;
    static constexpr int CW = BN / 8 / WAVES;                    // copies per wave and stage, W
    static constexpr int LOADS = CW + BM / 8 / WAVES;            // and both operands
    static constexpr int SEGS = NB * 4;               // 16-byte segments of a staged output row
    static constexpr int OUT = MB * 32 * SEGS * 16;   // a wave's staged output
    static constexpr int LDS = NBUF * STAGE > WAVES * OUT ? NBUF * STAGE : WAVES * OUT;
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "whole copies per wave");
    static_assert((SEGS & (SEGS - 1)) == 0, "the staging swizzle");
};

template <class T>
__global__ void __launch_bounds__(T::THREADS, T::WAVES == 8 ? 2 : 1)
i8_gemm_kernel(const int8_t *__restrict__ qa, const float *__restrict__ sa,
               const int8_t *__restrict__ qw, const float *__restrict__ sw,
               const uint16_t *__restrict__ bias, int act, int64_t M, int64_t N, int64_t K,
               uint16_t *__restrict__ Y) {
    __shared__ __align__(1024) uint8_t lds[T::LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t nbm = (M + T::BM - 1) / T::BM, nbn = (N + T::BN - 1) / T::BN;
    int64_t m0, n0;
    {
        const int64_t id = xcd_range(blockIdx.x, nbm * nbn);
        const int64_t per = kGroupM * nbn, g = id / per;
        const int64_t gm = nbm - g * kGroupM < kGroupM ? nbm - g * kGroupM : kGroupM;
        const int64_t in = id - g * per;
        m0 = (g * kGroupM + in % gm) * T::BM;
        n0 = in / gm * T::BN;
    }

    // Copies of a stage: 1 KB each, 8 rows; lane l carries row l / 8 into slot
    // l % 8.  Copy i of wave w: weight rows 8 (w + WAVES i) for i < CW, then token
    // rows.  Rows past the matrix re-read its last row (never stored).  The
    // second half of a stage that holds only 64 bytes re-reads the first (its
    // products are left out).
    uint32_t off[T::LOADS];
    const int row0 = 8 * wave + lane / 8;            // of copy 0; later ones 8 WAVES further
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) {
        const int row = row0 + 8 * T::WAVES * (i < T::CW ? i : i - T::CW);
        const int64_t left = i < T::CW ? N - n0 : M - m0;
        const uint32_t r = row < left ? row : (uint32_t)left - 1;
        off[i] = r * (uint32_t)K + 16 * ((lane & 7) ^ swz(row));
    }
    const int8_t *w0 = qw + n0 * K, *x0 = qa + m0 * K;
    const int nf = (int)(K / kRow);                  // whole stages
    const bool half = (K & 64) != 0;                 // then one of 64 bytes
    const int ns = nf + (half ? 1 : 0);
    auto issue = [&](int s) {
        uint8_t *st = lds + (s % T::NBUF) * T::STAGE + wave * 1024;
        const int64_t g = (int64_t)s * kRow;
        const bool last = s == nf;
#pragma unroll
        for (int i = 0; i < T::LOADS; ++i) {
            uint32_t o = off[i];
            if (last) {                              // segment seg -> seg % 4
                const int row = row0 + 8 * T::WAVES * (i < T::CW ? i : i - T::CW);
                o -= 16 * (((lane & 7) ^ swz(row)) & 4);
            }
            copy16_to_lds((i < T::CW ? w0 : x0) + g + o, st + i * T::WAVES * 1024);
        }
    };

    const int wn = wave / T::WM, wm = wave % T::WM;
    int a_at[4], b_at[4];                            // k step kk: bytes 32 kk .. of a row
    {
        const int ar = wn * T::NB * 32 + (lane & 31), br = T::BN + wm * T::MB * 32 + (lane & 31);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int seg = 2 * kk + (lane >> 5);
            a_at[kk] = ar * kRow + 16 * (seg ^ swz(ar));
            b_at[kk] = br * kRow + 16 * (seg ^ swz(br));
        }
    }
    i32x16 acc[T::NB][T::MB];
#pragma unroll
    for (int i = 0; i < T::NB; ++i)
#pragma unroll
        for (int j = 0; j < T::MB; ++j) acc[i][j] = i32x16{};

    // Fragments of one k step, double-buffered: step kk + 1 is read while the
    // products of step kk run.  The barrier that hands a stage's buffer back sits
    // before its last step's products, whose operands are in registers by then:
    // they cover the barrier and the first reads of the next stage.
    struct Frags {
        i32x4 a[T::NB], b[T::MB];
    } f[2];
    auto load = [&](Frags &x, const uint8_t *st, int kk) {
#pragma unroll
        for (int i = 0; i < T::NB; ++i)
            x.a[i] = *reinterpret_cast<const i32x4 *>(st + a_at[kk] + i * 32 * kRow);
#pragma unroll
        for (int j = 0; j < T::MB; ++j)
            x.b[j] = *reinterpret_cast<const i32x4 *>(st + b_at[kk] + j * 32 * kRow);
    };
    auto mul = [&](const Frags &x) {
#pragma unroll
        for (int i = 0; i < T::NB; ++i)
#pragma unroll
            for (int j = 0; j < T::MB; ++j) acc[i][j] = mfma_i8_32x32x32(x.a[i], x.b[j], acc[i][j]);
    };

#pragma unroll
    for (int s = 0; s < T::NBUF; ++s)
        if (s < ns) issue(s);
    if (ns >= T::NBUF) wait_loads<(T::NBUF - 1) * T::LOADS>();
    else wait_loads<0>();
    wave_barrier_all();
    load(f[0], lds, 0);
    for (int s = 0; s < nf; ++s) {
        const uint8_t *st = lds + (s % T::NBUF) * T::STAGE;
        load(f[1], st, 1);
        mul(f[0]);
        load(f[0], st, 2);
        mul(f[1]);
        load(f[1], st, 3);
        mul(f[0]);
        // stage s + 1 has landed when at most the younger stages remain in flight
        if (s + T::NBUF <= ns) wait_loads<(T::NBUF - 2) * T::LOADS>();
        else wait_loads<0>();
        wave_barrier_all();
        if (s + T::NBUF < ns) issue(s + T::NBUF);
        if (s + 1 < ns) load(f[0], lds + ((s + 1) % T::NBUF) * T::STAGE, 0);
        mul(f[1]);
    }
    if (half) {
        load(f[1], lds + (nf % T::NBUF) * T::STAGE, 1);
        mul(f[0]);
        mul(f[1]);
    }
    wait_loads<0>();
    wave_barrier_all();                              // the ring becomes the output staging

    // Epilogue: lane l holds, of token column l % 32 of each block, channels
    // 8 q + 4 (l / 32) .. + 3 for q = 0 .. 3.  The wave stages [token][channel]
    // bf16 rows in its own part of the LDS and stores them as 16-byte segments.
    uint8_t *out = lds + wave * T::OUT;
    const int64_t nw = n0 + wn * T::NB * 32, mw = m0 + wm * T::MB * 32;
    const int h = lane >> 5;
#pragma unroll
    for (int j = 0; j < T::MB; ++j) {
        const int row = 32 * j + (lane & 31);
        const int64_t m = mw + row;
        const float a = m < M ? sa[m] : 0.0f;
#pragma unroll
        for (int i = 0; i < T::NB; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t n = nw + 32 * i + 8 * q + 4 * h;
                f32x4 w = {};
                u32x2 c = {};
                if (n < N) {                          // N % 8 == 0: four in or four out
                    w = *reinterpret_cast<const f32x4 *>(sw + n);
                    if (bias) c = *reinterpret_cast<const u32x2 *>(bias + n);
                }
                const float b[4] = {bf16_lo(c.x), bf16_hi(c.x), bf16_lo(c.y), bf16_hi(c.y)};
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = (float)acc[i][j][4 * q + e] * (a * w[e]) + b[e];
                    if (act) y[e] = gelu_exp2(y[e]);
                }
                const int seg = (4 * i + q) ^ (row & (T::SEGS - 1));
                *reinterpret_cast<u32x2 *>(out + (row * T::SEGS + seg) * 16 + 8 * h) =
                    u32x2{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
            }
        }
    }
    __builtin_amdgcn_wave_barrier();
    constexpr int ROWS = 64 / T::SEGS;               // rows per store instruction
#pragma unroll
    for (int it = 0; it < T::MB * 32 / ROWS; ++it) {
        const int row = it * ROWS + lane / T::SEGS, sl = lane % T::SEGS;
        const u32x4 y = *reinterpret_cast<const u32x4 *>(out + (row * T::SEGS + (sl ^ (row & (T::SEGS - 1)))) * 16);
        const int64_t m = mw + row, n = nw + 8 * sl;
        if (m < M && n < N)   // not read again here: past the L2, whose room the operands use
            __builtin_nontemporal_store(y, reinterpret_cast<u32x4 *>(Y + m * N + n));
    }
}

// Tall tiles: 256 channels x 64 MB tokens, eight waves 2 (tokens) x 4
// (channels), 32 MB x 64 each; one workgroup per compute unit.
template <int BM>
using Tall = Tile<BM, 256, 2, 4, 2>;
typedef Tile<128, 128, 2, 2, 2> Mid;
typedef Tile<64, 64, 2, 2, 4> Small;

template <class T>
int64_t tiles(int64_t M, int64_t N) {
    return (M + T::BM - 1) / T::BM * ((N + T::BN - 1) / T::BN);
}

}  // namespace i8

using namespace i8;

int64_t i8_gemm_groups(int64_t M, int64_t N) { return tiles<Small>(M, N); }
size_t i8_gemm_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_i8_gemm(const int8_t *qa, const float *sa, const int8_t *qw, const float *sw,
                          const uint16_t *bias, int act, int64_t M, int64_t N, int64_t K,
                          uint16_t *Y, void *workspace, hipStream_t stream) {
    (void)workspace;
    const int64_t cus = wg_slots() / 2;
    auto run = [&](auto t) {
        typedef decltype(t) T;
        i8_gemm_kernel<T><<<(unsigned)tiles<T>(M, N), T::THREADS, 0, stream>>>(
            qa, sa, qw, sw, bias, act, M, N, K, Y);
        return hipGetLastError();
    };
    if (tiles<Tall<256>>(M, N) >= cus) {
        // The height with the shortest time for the whole rounds of compute
        // units that its tiles take, a tile's time taken as its height + 16.
        int best = 0;
        int64_t least = 0;
        for (int bm = 128; bm <= 320; bm += 64) {
            const int64_t n = (M + bm - 1) / bm * ((N + 255) / 256);
            const int64_t cost = (n + cus - 1) / cus * (bm + 16);
            if (!best || cost < least) best = bm, least = cost;
        }
        if (best == 128) return run(Tall<128>());
        if (best == 192) return run(Tall<192>());
        if (best == 256) return run(Tall<256>());
        return run(Tall<320>());
    }
    if (tiles<Mid>(M, N) >= cus) return run(Mid());
    return run(Small());
}

}  // namespace svdq
