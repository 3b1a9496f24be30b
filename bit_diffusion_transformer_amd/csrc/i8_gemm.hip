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
//
// Measured by calls in a row with inputs that change (operations: two per code
// product).  4096 x 4096 -> 16384 with GELU: 260-263 us, 2.1 POP/s; 4608 x 12288 ->
// 4096: 200-206 us, 2.25-2.3 POP/s.  Bound by power: all-zero codes take 211 and 169
// us, in as many cycles at 2.45 GHz that random ones get at 1.9.  333 tokens, 4096 ->
// 4096: 14.5 us, of which 4 are a launch with one stage; every further stage of 128
// costs 0.35 us (two workgroups' barrier, 32 KB of copies, 64 KB of fragment reads),
// whether its operands are in the L2s or not.
#include "i8_device.h"
#include "i8_internal.h"
#include "svdq_wave.h"

#include <type_traits>

namespace svdq {

namespace i8 {

constexpr int kGroupM = 8;       // m tiles per raster group (L2 reuse of weights)

// WM x WN waves cover a tile; KS such groups share its stages of K in turn (stage
// s goes to group s % KS), each with a ring of its own, and add their sums at
// the end.
template <int BM_, int BN_, int WM_, int WN_, int NBUF_, int KS_ = 1>
struct Tile {
    static constexpr int BM = BM_, BN = BN_;          // tokens, output channels
    static constexpr int WM = WM_, WN = WN_;          // waves along each
    static constexpr int NBUF = NBUF_;                // stages in the ring
    static constexpr int KS = KS_;                    // groups along K
    static constexpr int WAVES = WM * WN;             // of a group
    static constexpr int THREADS = 64 * WAVES * KS;
    static constexpr int MB = BM / WM / 32, NB = BN / WN / 32;   // 32 x 32 blocks per wave
    static constexpr int STAGE = (BM + BN) * kRow;
    static constexpr int CW = BN / 8 / WAVES;                    // copies per wave and stage, W
    static constexpr int LOADS = CW + BM / 8 / WAVES;            // and both operands
    static constexpr int SEGS = NB * 4;               // 16-byte segments of a staged output row
    static constexpr int OUT = MB * 32 * SEGS * 16;   // a wave's staged output
    static constexpr int SUMS = (KS - 1) * BM * BN * 4;          // the other groups' sums
    static constexpr int RING = NBUF * STAGE;                    // of a group
    static constexpr int LDS = KS * RING > SUMS + WAVES * OUT ? KS * RING : SUMS + WAVES * OUT;
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "whole copies per wave");
    static_assert((SEGS & (SEGS - 1)) == 0, "the staging swizzle");
};

template <class T>
__global__ void __launch_bounds__(T::THREADS, T::WAVES == 8 ? 2 : T::KS * T::WAVES / 4 > 1 ? T::KS * T::WAVES / 4 : 1)
i8_gemm_kernel(const int8_t *__restrict__ qa, const float *__restrict__ sa,
               const int8_t *__restrict__ qw, const float *__restrict__ sw,
               const uint16_t *__restrict__ bias, int act, int64_t M, int64_t N, int64_t K,
               uint16_t *__restrict__ Y) {
    __shared__ __align__(1024) uint8_t lds[T::LDS];
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = wid % T::WAVES, group = wid / T::WAVES;
    uint8_t *const ring = lds + group * T::RING;
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
    auto issue = [&](int s, int slot) {
        uint8_t *st = ring + slot * T::STAGE + wave * 1024;
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

    // The group's i-th stage is stage group + KS i; every group runs `turns` of
    // them, so that all meet at every barrier.
    const int turns = (ns + T::KS - 1) / T::KS;
    auto stage = [&](int i) { return T::KS * i + group; };
#pragma unroll
    for (int i = 0; i < T::NBUF; ++i)
        if (stage(i) < ns) issue(stage(i), i);
    if (stage(T::NBUF - 1) < ns) wait_loads<(T::NBUF - 1) * T::LOADS>();
    else wait_loads<0>();
    wave_barrier_all();
    if (T::KS == 1 || group < ns) load(f[0], ring, 0);
    for (int i = 0; T::KS == 1 ? i < nf : i < turns; ++i) {
        const uint8_t *st = ring + (i % T::NBUF) * T::STAGE;
        if (T::KS == 1 || stage(i) < nf) {
            load(f[1], st, 1);
            mul(f[0]);
            load(f[0], st, 2);
            mul(f[1]);
            load(f[1], st, 3);
            mul(f[0]);
        } else if (stage(i) < ns) {                  // the 64-byte stage
            load(f[1], st, 1);
            mul(f[0]);
        }
        // the next stage has landed when at most the younger ones remain in flight
        if (stage(i + T::NBUF - 1) < ns) wait_loads<(T::NBUF - 2) * T::LOADS>();
        else wait_loads<0>();
        wave_barrier_all();
        if (stage(i + T::NBUF) < ns) issue(stage(i + T::NBUF), i % T::NBUF);
        if (stage(i + 1) < ns) load(f[0], ring + ((i + 1) % T::NBUF) * T::STAGE, 0);
        if (T::KS == 1 || stage(i) < ns) mul(f[1]);
    }
    if (T::KS == 1 && half) {
        load(f[1], ring + (nf % T::NBUF) * T::STAGE, 1);
        mul(f[0]);
        mul(f[1]);
    }
    wait_loads<0>();
    wave_barrier_all();                              // the rings become sums and output staging
    if (T::KS > 1) {
        auto part = [&](int g, int i, int j, int q) {
            return reinterpret_cast<i32x4 *>(
                lds + ((((g - 1) * T::WAVES + wave) * T::NB + i) * T::MB + j) * 4096 + q * 1024 + lane * 16);
        };
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < T::NB; ++i)
#pragma unroll
                for (int j = 0; j < T::MB; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *part(group, i, j, q) = i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                      acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        }
        wait_loads<0>();
        wave_barrier_all();
        if (group > 0) return;
        for (int g = 1; g < T::KS; ++g)
#pragma unroll
            for (int i = 0; i < T::NB; ++i)
#pragma unroll
                for (int j = 0; j < T::MB; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const i32x4 x = *part(g, i, j, q);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += x[e];
                    }
    }

    // Epilogue: lane l holds, of token column l % 32 of each block, channels
    // 8 q + 4 (l / 32) .. + 3 for q = 0 .. 3.  The wave stages [token][channel]
    // bf16 rows in its own part of the LDS and stores them as 16-byte segments.
    uint8_t *out = lds + T::SUMS + wave * T::OUT;
    const int64_t nw = n0 + wn * T::NB * 32, mw = m0 + wm * T::MB * 32;
    const int h = lane >> 5;
    // Every scale and bias first, in one batch of loads (N % 8 == 0: four channels
    // are in or out together; those past N re-read the last four, never stored).
    f32x4 w[T::NB][4];
    u32x2 c[T::NB][4];
    float a[T::MB];
#pragma unroll
    for (int i = 0; i < T::NB; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            int64_t n = nw + 32 * i + 8 * q + 4 * h;
            n = n < N ? n : N - 4;
            w[i][q] = *reinterpret_cast<const f32x4 *>(sw + n);
            c[i][q] = bias ? *reinterpret_cast<const u32x2 *>(bias + n) : u32x2{};
        }
#pragma unroll
    for (int j = 0; j < T::MB; ++j) {
        const int64_t m = mw + 32 * j + (lane & 31);
        a[j] = sa[m < M ? m : M - 1];
    }
#pragma unroll
    for (int j = 0; j < T::MB; ++j) {
        const int row = 32 * j + (lane & 31);
#pragma unroll
        for (int i = 0; i < T::NB; ++i) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float b[4] = {bf16_lo(c[i][q].x), bf16_hi(c[i][q].x), bf16_lo(c[i][q].y),
                                    bf16_hi(c[i][q].y)};
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = (float)acc[i][j][4 * q + e] * (a[j] * w[i][q][e]) + b[e];
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
typedef Tile<128, 128, 2, 2, 4> Mid;          // one per compute unit, three stages ahead
typedef Tile<128, 64, 2, 2, 3> Half;          // two per compute unit
typedef Tile<64, 64, 2, 2, 4> Small;          // two per compute unit
typedef Tile<32, 64, 1, 2, 3, 4> Few;         // few tiles: K shared by four groups
typedef Tile<32, 32, 1, 1, 4, 4> Fewest;

template <class T>
int64_t tiles(int64_t M, int64_t N) {
    return (M + T::BM - 1) / T::BM * ((N + T::BN - 1) / T::BN);
}

}  // namespace i8

using namespace i8;

int64_t i8_gemm_groups(int64_t M, int64_t N) { return tiles<Small>(M, N); }

hipError_t launch_i8_gemm(const int8_t *qa, const float *sa, const int8_t *qw, const float *sw,
                          const uint16_t *bias, int act, int64_t M, int64_t N, int64_t K,
                          uint16_t *Y, hipStream_t stream) {
    const int64_t cus = wg_slots() / 2;
    auto run = [&](auto t) {
        typedef decltype(t) T;
        i8_gemm_kernel<T><<<(unsigned)tiles<T>(M, N), T::THREADS, 0, stream>>>(
            qa, sa, qw, sw, bias, act, M, N, K, Y);
        return hipGetLastError();
    };
    // The smaller tiles while they fit the compute units once (K shared by four
    // groups of waves) or twice; then larger ones, whose operands are read less
    // often.  Measured with K = 4096 and N = 4096 in us, at M = 1, 64, 128, 333,
    // 512, 777, 1024: Fewest 7.3, 8.2, 14, ..; Few 8.8, 9.4, 9.9, 26, ..; Small 11,
    // 11, 12, 15, 17, 33, 38; Half 17, 17, 17, 18, 19, 25, 30; Mid 22, 22, 22, 23,
    // 24, 27, 28.
    if (tiles<Fewest>(M, N) <= cus) return run(Fewest());
    if (tiles<Few>(M, N) <= cus) return run(Few());
    if (tiles<Small>(M, N) <= 2 * cus) return run(Small());
    if (4 * tiles<Mid>(M, N) < 3 * cus) return run(Half());
    if (tiles<Mid>(M, N) <= cus) return run(Mid());
    if (tiles<Half>(M, N) <= 2 * cus) return run(Half());   // 4128 x 960 x 3584: 23.5, Tall 30.0
    // Tall tiles: the height with the shortest time for the whole rounds of
    // compute units that its tiles take; a round costs its rows and, for filling
    // the ring and the epilogue, as much as 112 rows at K = 4096.
    int best = 0;
    int64_t least = 0;
    for (int bm = 128; bm <= 320; bm += 64) {
        const int64_t n = (M + bm - 1) / bm * ((N + 255) / 256);
        const int64_t cost = (n + cus - 1) / cus * (bm * K + 112 * 4096);
        if (!best || cost < least) best = bm, least = cost;
    }
    if (best == 128) return run(Tall<128>());
    if (best == 192) return run(Tall<192>());
    if (best == 256) return run(Tall<256>());
    return run(Tall<320>());
}

}  // namespace svdq
