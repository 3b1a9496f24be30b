// span_attention.hip -- attention of packed sequences and of new tokens over a
// paged cache, on the bf16 matrix instruction (v_mfma_f32_32x32x16_bf16).
//
// A tile is 128 or 256 rows of one sequence and key head: row r is head r % group
// of token r / group, so that the heads that share a key head share its tiles, and
// a few tokens fill more of one.  Four or eight waves of 32 rows go over the tile's
// blocks of 64 keys with the score and weight layouts of the block-sparse
// kernel: S^T = K Q^T, the softmax within a lane, O^T = V^T P^T, K and V copied
// into LDS a block ahead.  What a workgroup does is a piece of the line of all
// tiles (span_plan.h).  A request of at most 32 rows beside longer ones ("narrow") would
// leave all waves but one idle: there every wave has the same rows and keys of its own.
//
// What bounds it.  Long sequences: power.  16384 causal tokens, 32 heads on 8 of 128, take 2.0 ms
// (1.1 PFLOP/s, the matrix units busy 54 % of the cycles at about 1.9 GHz); with all inputs zero
// the same work takes 1.54 ms.  Four images of 777 to 4096 tokens, 24 heads: 310 us, with zeros 246.
// Two streams of 1560 rows over 32760 keys, 12 heads: 670 us, 0.89 PFLOP/s, with zeros 515.  (On the
// slowest card seen 2.16 ms, 333 and 721 us.)  Short ones: a tile's start and end (the queries, the
// first copies, the partial results; about 4 us), which other workgroups of the compute unit fill
// in part: twelve prompts of 1 to 2000 tokens 100 us, 0.66 PFLOP/s (90 with zeros).  Two waves a
// SIMD, D = 64 too: with four (and 128 registers) its pass spills, 1000 causal tokens of 16 heads
// 29.7 us against 22.2, 4000 80 against 66.  Narrow: 31 decoding requests of up to 6000 keys beside
// 512 new tokens over 4608, 28 heads of 64 on 4, in tiles of 256 rows: 48 us, 54 with wide tiles for
// all; the 31 alone 20 and 26.
#include "attention_tile.h"
#include "span_plan.h"

#include <type_traits>

namespace svdq {

namespace span {

using namespace attn;

template <int D, bool PAGED, int WAVES>
struct Lds {
    static constexpr int TILE = kKeys * D * 2;     // bytes of a K or V block
    static constexpr int OWN = 32 * D * 2;         // of a narrow tile's unit, a wave's own
    static constexpr int BYTES = PAGED && 2 * WAVES * OWN > 4 * TILE ? 2 * WAVES * OWN : 4 * TILE;
    uint8_t kv[BYTES];                             // K [2], V [2]; narrow: a wave's K and V, wave after wave
    Seq seqs[WAVES][64];                           // a wave each: they are not in step
    f32x2 stat[PAGED ? WAVES : 1][32];             // narrow: maximum and sum of each wave's rows
};

template <int D, bool PAGED, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 2)
span_attention_kernel(SpanArgs a, Shared *__restrict__ shared, float *__restrict__ part,
                      float *__restrict__ stat) {
    constexpr int kRows = 32 * WAVES;
    constexpr int DB = D / 32, DK = D / 16;        // 32-wide blocks and 16-wide steps of D
    constexpr int RPT = 512 / D;                   // rows per 1 KB copy
    constexpr int SEGS = D / 8;                    // 16-byte segments of a row
    constexpr int PART = kKeys / WAVES, COPIES = PART / RPT;   // rows and copies per wave
    typedef Lds<D, PAGED, WAVES> L;
    __shared__ __align__(1024) L lds;
    uint8_t *const lds_v0 = lds.kv + 2 * L::TILE;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h2 = lane >> 5, col = lane & 31;

    const int w = (int)xcd_range(blockIdx.x, gridDim.x);
    if (threadIdx.x == 0) shared[2 * w].parts = shared[2 * w + 1].parts = 0;
    Piece<kRows> piece;
    if (!piece.open(a, lds.seqs[wave], w, (int)gridDim.x)) return;
    Place<kRows> &at = piece.at;

    // Within the 16 or 8 rows that this wave copies of a block: bytes of a row from the first.
    const int cp_row = lane / SEGS, cp_slot = lane % SEGS;
    const int64_t k_row = PAGED ? D * 2 : a.k_stride * 2, v_row = PAGED ? D * 2 : a.v_stride * 2;
    uint32_t k_at[COPIES], v_at[COPIES];
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
        const int r = c * RPT + cp_row, row = PART * wave + r;
        k_at[c] = (uint32_t)(r * k_row) + 16 * (cp_slot ^ swz_k<D>(row));
        v_at[c] = (uint32_t)(r * v_row) + 16 * (cp_slot ^ swz_v<D>(row));
    }
    // LDS offsets (of buffer 0): K row `col` (and 32 further), segment 2 t + h2 of
    // step t; V: lane i of a 16-lane group supplies row i / 4 of four keys, 4
    // columns from 4 (i % 4) of the group's 16, and gets column i of the four
    // rows; a step of 16 keys is 16 rows further (the same swizzle).
    const uint8_t *k_rd[DK], *v_rd[DB];
#pragma unroll
    for (int t = 0; t < DK; ++t)
        k_rd[t] = lds.kv + col * (D * 2) + 16 * ((2 * t + h2) ^ swz_k<D>(col));
    {
        const int i = lane & 15, row = 4 * h2 + (i >> 2);
        const int sub = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);     // segment of a 32-wide block
#pragma unroll
        for (int d = 0; d < DB; ++d)
            v_rd[d] = lds_v0 + row * (D * 2) + 16 * ((4 * d + sub) ^ swz_v<D>(row)) + 8 * (lane & 1);
    }
    const uint32_t lds_k = lds_address(lds.kv) + wave * COPIES * 1024, lds_v = lds_k + 2 * L::TILE;
    const float scale_log2 = a.scale_log2;

    for (;; ) {
        // ---- one tile, or the part of it that this piece of the line has
        const int first = piece.first, last = piece.last;
        const int64_t row0 = (int64_t)at.t * kRows, rows_left = (int64_t)at.s.nq * a.group - row0;
        if (rows_left <= 0) return;                // (lengths that changed under the call)
        const int rows = rows_left < kRows ? (int)rows_left : kRows;
        const int tok0 = token_of(a, (double)row0), rem0 = (int)(row0 - (int64_t)tok0 * a.group);
        const int nk = at.s.nk;
        const bool narrow = PAGED && Place<kRows>::narrow(a, at.s);
        const int mine = narrow ? col : 32 * wave + col;
        const bool active = 32 * wave < rows;      // uniform over the wave
        const int row = mine < rows ? mine : rows - 1;   // rows past the last: never stored
        const int ahead = token_of(a, rem0 + row), tok = tok0 + ahead, sub = rem0 + row - ahead * a.group;
        // keys that the row sees: no more than the rows behind it
        int limit = a.causal ? nk - at.s.nq + 1 + tok : nk;
        limit = limit < 0 ? 0 : limit < nk ? limit : nk;
        const int low = __builtin_amdgcn_readlane(limit, 0), high = __builtin_amdgcn_readlane(limit, 31);

        const uint8_t *kb, *vb;
        int pages = -1;                            // lane l: page of block i0 + l / 4, rows 16 (l % 4) on
        uint32_t bad = 0, bad_next = 0;            // 16-row parts of a block without a page
        uint64_t bad16 = 0;
        if (PAGED) {
            kb = reinterpret_cast<const uint8_t *>(a.k);
            vb = reinterpret_cast<const uint8_t *>(a.v);
        } else {
            kb = reinterpret_cast<const uint8_t *>(a.k + at.s.k0 * a.k_stride + (int64_t)at.g * D);
            vb = reinterpret_cast<const uint8_t *>(a.v + at.s.k0 * a.v_stride + (int64_t)at.g * D);
        }
        const int32_t *table = PAGED ? a.tables + (int64_t)at.b * a.width : nullptr;
        auto read_pages = [&](int i0) __attribute__((always_inline)) {            // of 16 blocks
            const int n = i0 * kKeys + 16 * lane;
            int p = -1;
            if (n < nk) p = table[n >> a.page_shift];
            const bool good = p >= 0 && p < a.pages;
            pages = good ? p : -1;
            bad16 = __ballot(!good && n < nk);
        };
        // Rows at or past the sequence's keys, and those without a page, are not read: K is left
        // as it is (its scores are masked, whatever they are), V is zero (the weights are
        // zero, and zero times what is not finite would be NaN).
        auto issue = [&](int i, auto buffer) __attribute__((always_inline)) {
            constexpr int BUF = decltype(buffer)::value;
            const int n0 = i * kKeys + PART * wave;
            int left = nk - n0;
            const uint8_t *k0, *v0;
            if (PAGED) {
                if ((i & 15) == 0 || i == first) read_pages(i & ~15);
                const int page = __builtin_amdgcn_readlane(pages, 4 * (i & 15) + wave * PART / 16);
                bad_next = (uint32_t)(bad16 >> (4 * (i & 15))) & 15u;
                if (page < 0) left = 0;
                const int64_t r = ((((int64_t)page * a.G + at.g) << a.page_shift) +
                                   (n0 & ((1 << a.page_shift) - 1))) * (D * 2);
                k0 = kb + r;
                v0 = vb + r;
            } else {
                k0 = kb + n0 * k_row;
                v0 = vb + n0 * v_row;
            }
            const uint32_t kd = lds_k + BUF * L::TILE, vd = lds_v + BUF * L::TILE;
            if (__builtin_expect(left >= PART, 1)) {
                copies_in_flight(k0, k_at, kd);
                copies_in_flight(v0, v_at, vd);
            } else {
#pragma unroll
                for (int c = 0; c < COPIES; ++c) {
                    if (c * RPT + cp_row < left) {
                        copy_in_flight(k0, k_at[c], kd + c * 1024);
                        copy_in_flight(v0, v_at[c], vd + c * 1024);
                    } else {
                        *reinterpret_cast<u32x4 *>(lds_v0 + BUF * L::TILE + (wave * COPIES + c) * 1024 + lane * 16) = u32x4{};
                    }
                }
            }
        };

        // A narrow tile: every wave has all its rows and goes over units of 32 keys of its own, the
        // wave-th, then every WAVES-th; K and V of a unit lie in LDS of its own, K of the next one
        // is copied as soon as the scores are there, V as soon as it has been used.
        constexpr int NC = 16 / RPT;               // copies of 16 keys
        const int u0 = 2 * first + wave, seen = (high + 31) / 32, u1 = 2 * last < seen ? 2 * last : seen;
        const uint32_t own = (uint32_t)wave * (2 * L::OWN);
        uint32_t nk_at[NC], nv_at[NC];             // bytes from the first of 16 keys
        bool full = false, full_next = false;      // every copy of the unit was issued
        auto issue_unit = [&](int u, auto which) __attribute__((always_inline)) {
            constexpr bool V = decltype(which)::value;
            const int j = (u - u0) / WAVES;
            if (!V && (j & 31) == 0) {             // lane l: 16 keys of this wave's unit j + l / 2
                const int n = 16 * (2 * (u + WAVES * (lane >> 1)) + (lane & 1));
                const int p = n < nk ? table[n >> a.page_shift] : -1;
                const bool good = p >= 0 && p < a.pages;
                pages = good ? p : -1;
                bad16 = __ballot(!good && n < nk);
            }
            if (!V) {
                bad_next = (uint32_t)(bad16 >> (2 * (j & 31))) & 3u;
                full_next = true;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n0 = 32 * u + 16 * h, page = __builtin_amdgcn_readlane(pages, 2 * (j & 31) + h);
                const int left = page < 0 ? 0 : nk - n0;
                const int64_t r = ((((int64_t)page * a.G + at.g) << a.page_shift) +
                                   (n0 & ((1 << a.page_shift) - 1))) * (D * 2);
                const uint32_t to = own + (V ? L::OWN : 0) + h * 16 * D * 2;
                const uint32_t (&off)[NC] = V ? nv_at : nk_at;
                if (__builtin_expect(left >= 16, 1)) {
                    copies_in_flight((V ? vb : kb) + r, off, lds_address(lds.kv) + to);
                } else {
                    full_next = false;
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        if (c * RPT + cp_row < left)
                            copy_in_flight((V ? vb : kb) + r, off[c], lds_address(lds.kv) + to + c * 1024);
                        else if (V)
                            *reinterpret_cast<u32x4 *>(lds.kv + to + c * 1024 + lane * 16) = u32x4{};
                }
            }
        };
        auto start_units = [&]() __attribute__((always_inline)) {
            if (u0 >= u1) return;
            issue_unit(u0, std::false_type());
            issue_unit(u0, std::true_type());
        };

        u32x4 qf[DK];
        {
            const uint16_t *p = a.q + (int64_t)(at.s.q0 + tok) * a.q_stride +
                                (int64_t)(at.g * a.group + sub) * D + 8 * h2;
#pragma unroll
            for (int s = 0; s < DK; ++s) qf[s] = *reinterpret_cast<const u32x4 *>(p + 16 * s);
            if (narrow) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int r = c * RPT + cp_row;
                    nk_at[c] = r * (D * 2) + 16 * (cp_slot ^ swz_k<D>(r));
                    nv_at[c] = r * (D * 2) + 16 * (cp_slot ^ swz_v<D>(r));
                }
                start_units();
            } else if (first < last) {
                issue(first, std::integral_constant<int, 0>());
            }
            // A row with a value that is not finite becomes a row of NaN: scores of minus
            // infinity alone would look like keys that it does not see.
            uint32_t odd = 0;
#pragma unroll
            for (int s = 0; s < DK; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) odd |= not_finite(qf[s][j]);
            const uint64_t rows_odd = __ballot(odd != 0);
            if (rows_odd && ((rows_odd >> col | rows_odd >> (col + 32)) & 1))
#pragma unroll
                for (int s = 0; s < DK; ++s) qf[s] = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
        }

        f32x16 o[DB];
        float m, l;
        // A v that is not finite, of a key that only some rows of a block see, would reach the
        // others as zero times it.  That shows as a result that is not finite, and the part is
        // gone over once more with such values taken out of the blocks that have a mask, and a
        // NaN put where a row sees one of them, whatever its weight: in the blocks without a
        // mask a weight of zero gives one too.
        bool masked = false;
        auto pass = [&](auto mode) __attribute__((always_inline)) {
            constexpr bool careful = decltype(mode)::value;
#pragma unroll
            for (int d = 0; d < DB; ++d) o[d] = f32x16{};
            m = -__builtin_inff();
            l = 0.0f;
            auto block = [&](int i, auto buffer) __attribute__((always_inline)) {
                constexpr int BUF = decltype(buffer)::value, AT = BUF * L::TILE;
                const int n0 = i * kKeys;
                wait_loads<0>();
                wave_barrier_all();
                bad = bad_next;
                if (i + 1 < last) issue(i + 1, std::integral_constant<int, 1 - BUF>());
                if (!active || n0 >= high) return;
                f32x16 s[2] = {f32x16{}, f32x16{}};
                {
                    // fragments two steps ahead of the products that use them
                    u32x4 kf[3][2];
                    auto load = [&](int t) __attribute__((always_inline)) {
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk)
                            kf[t % 3][kk] = *reinterpret_cast<const u32x4 *>(k_rd[t] + AT + 32 * kk * (D * 2));
                    };
                    load(0);
                    load(1);
#pragma unroll
                    for (int t = 0; t < DK; ++t) {
                        if (t + 2 < DK) load(t + 2);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) s[kk] = mfma_bf16_32x32x16(kf[t % 3][kk], qf[t], s[kk]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                // V fragments of a step of 16 keys (kk, t): keys 0 .. 3 and 8 .. 11 past
                // 4 h2, every 32-wide block of columns
                u32x4 vf[2][DB];
                auto load_v = [&](int st) __attribute__((always_inline)) {
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const u32x2 y = read_transposed(v_rd[d] + AT + (16 * st + 8 * u) * (D * 2));
                            vf[st & 1][d][2 * u] = y.x;
                            vf[st & 1][d][2 * u + 1] = y.y;
                        }
                };
                load_v(0);
                __builtin_amdgcn_sched_barrier(0);
                const bool edge = n0 + kKeys > low || (PAGED && bad != 0);
                if (edge) {
                    masked = true;
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int n = n0 + 32 * kk + 8 * (e / 4) + 4 * h2 + e % 4;
                            if (n >= limit || (PAGED && (bad >> (2 * kk + e / 8) & 1)))
                                s[kk][e] = -__builtin_inff();
                        }
                }
                float top = s[0][0];
#pragma unroll
                for (int e = 1; e < 16; ++e) top = fmaxf(top, s[0][e]);
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, s[1][e]);
                top = max_both_halves(top);
                // The running maximum moves only when a score passes it by more than 8
                // in the exponent of two: the weights stay below 2^8, and most blocks
                // leave the sums as they are.
                if (__any((top - m) * scale_log2 > 8.0f)) {
                    const float m1 = fmaxf(m, top);
                    const float f = m == m1 ? 1.0f : __builtin_amdgcn_exp2f((m - m1) * scale_log2);
                    m = m1;
                    l *= f;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[d][e] *= f;
                }
                // A weight's exponent is s c - fl(m c), c = scale log2 e, in one operation: off
                // by the rounding of m c, which all keys of a row share: at most 2^-15 up to
                // |m c| = 2^10.  Past that the difference s - m is taken first (exact where a
                // weight counts).  A row without a key so far has m = -inf and no offset.
                float off = m * scale_log2;
                const bool far = fabsf(off) > 1024.0f;
                if (__any(far)) {
                    const float by = far && m > -__builtin_inff() ? m : 0.0f;
                    off = far ? 0.0f : off;
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int e = 0; e < 16; ++e) s[kk][e] -= by;
                }
                // [kk][step of 16 keys]: weights, rounded to bf16, the type of the matrix
                // instruction's operand beside V; the same values go into their sum, so a
                // row's weights still add up to one.
                u32x4 p[2][2];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        s[kk][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kk][e], scale_log2, -off));
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            p[kk][t][x] = pack_bf16x2(s[kk][8 * t + 2 * x], s[kk][8 * t + 2 * x + 1]);
                            l = add_pair(p[kk][t][x], l);
                        }
                }
                if (careful && edge) {
#pragma unroll 1
                    for (int st = 0; st < 4; ++st) {
                        u32x4 ps = p[0][0];
                        if (st == 1) ps = p[0][1];
                        if (st == 2) ps = p[1][0];
                        if (st == 3) ps = p[1][1];
                        const int lim = PAGED && (bad >> st & 1) ? 0 : limit;
                        u32x4 seen;
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            seen[x] = seen_pair(n0 + 16 * st + 8 * (x >> 1) + 4 * h2 + 2 * (x & 1), lim);
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            u32x4 x, odd;
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const u32x2 y = read_transposed(v_rd[d] + AT + (16 * st + 8 * u) * (D * 2));
                                x[2 * u] = y.x;
                                x[2 * u + 1] = y.y;
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t f = not_finite(x[j]);     // 0x8000 of each half
                                odd[j] = (f >> 15) * 0x3F80u;
                                x[j] &= ~((f >> 15) * 0xFFFFu);
                            }
                            o[d] = mfma_bf16_32x32x16(x, ps, o[d]);
                            const f32x16 c = mfma_bf16_32x32x16(odd, seen, f32x16{});
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (c[e] > 0.0f) o[d][e] = __builtin_nanf("");
                        }
                    }
                    return;
                }
#pragma unroll
                for (int st = 0; st < 4; ++st) {
                    if (st < 3) load_v(st + 1);
#pragma unroll
                    for (int d = 0; d < DB; ++d) o[d] = mfma_bf16_32x32x16(vf[st & 1][d], p[st >> 1][st & 1], o[d]);
                }
            };
            if (careful && first < last) issue(first, std::integral_constant<int, 0>());
            for (int i = first; i < last; i += 2) {
                block(i, std::integral_constant<int, 0>());
                if (i + 1 < last) block(i + 1, std::integral_constant<int, 1>());
            }
        };
        if (PAGED && narrow) {
            auto units = [&](auto mode) __attribute__((always_inline)) {
                constexpr bool careful = decltype(mode)::value;
#pragma unroll
                for (int d = 0; d < DB; ++d) o[d] = f32x16{};
                m = -__builtin_inff();
                l = 0.0f;
                for (int u = u0; u < u1; u += WAVES) {
                    const int n0 = 32 * u;
                    bad = bad_next;
                    full = full_next;
                    if (full)
                        wait_loads<2 * NC>();      // all but this unit's V
                    else
                        wait_loads<0>();
                    asm volatile("" ::: "memory");
                    f32x16 s = {};
#pragma unroll
                    for (int t = 0; t < DK; ++t)
                        s = mfma_bf16_32x32x16(*reinterpret_cast<const u32x4 *>(k_rd[t] + own), qf[t], s);
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    const bool more = u + WAVES < u1;
                    if (more) issue_unit(u + WAVES, std::false_type());
                    const bool edge = n0 + 32 > low || bad != 0;
                    if (edge) {
                        masked = true;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int n = n0 + 8 * (e / 4) + 4 * h2 + e % 4;
                            if (n >= limit || (bad >> (e / 8) & 1)) s[e] = -__builtin_inff();
                        }
                    }
                    float top = s[0];
#pragma unroll
                    for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
                    top = max_both_halves(top);
                    if (__any((top - m) * scale_log2 > 8.0f)) {
                        const float m1 = fmaxf(m, top);
                        const float f = m == m1 ? 1.0f : __builtin_amdgcn_exp2f((m - m1) * scale_log2);
                        m = m1;
                        l *= f;
#pragma unroll
                        for (int d = 0; d < DB; ++d)
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[d][e] *= f;
                    }
                    float off = m * scale_log2;
                    const bool far = fabsf(off) > 1024.0f;
                    if (__any(far)) {
                        const float by = far && m > -__builtin_inff() ? m : 0.0f;
                        off = far ? 0.0f : off;
#pragma unroll
                        for (int e = 0; e < 16; ++e) s[e] -= by;
                    }
                    u32x4 p[2];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], scale_log2, -off));
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            p[t][x] = pack_bf16x2(s[8 * t + 2 * x], s[8 * t + 2 * x + 1]);
                            l = add_pair(p[t][x], l);
                        }
                    if (more && full_next)
                        wait_loads<2 * NC>();      // all but the next unit's K
                    else
                        wait_loads<0>();
                    asm volatile("" ::: "memory");
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            u32x4 x, odd = {};
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const u32x2 y = read_transposed(v_rd[d] + own + L::OWN - 2 * L::TILE + (16 * t + 8 * h) * (D * 2));
                                x[2 * h] = y.x;
                                x[2 * h + 1] = y.y;
                            }
                            if (careful && edge)
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const uint32_t f = not_finite(x[j]);
                                    odd[j] = (f >> 15) * 0x3F80u;
                                    x[j] &= ~((f >> 15) * 0xFFFFu);
                                }
                            o[d] = mfma_bf16_32x32x16(x, p[t], o[d]);
                            if (careful && edge) {
                                const int lim = bad >> t & 1 ? 0 : limit;
                                u32x4 seen;
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    seen[y] = seen_pair(n0 + 16 * t + 8 * (y >> 1) + 4 * h2 + 2 * (y & 1), lim);
                                const f32x16 c = mfma_bf16_32x32x16(odd, seen, f32x16{});
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if (c[e] > 0.0f) o[d][e] = __builtin_nanf("");
                            }
                        }
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    if (more) issue_unit(u + WAVES, std::true_type());
                }
            };
            units(std::false_type());
            float z = 0.0f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) z = __builtin_fmaf(o[d][e], 0.0f, z);
            if (__builtin_expect(__any(masked && z != z), 0)) {
                start_units();
                units(std::true_type());
            }
            // The waves' results, each in its own LDS, then their sums, four columns at a time.
            l = sum_both_halves(l);
            f32x4 *const mine_o = reinterpret_cast<f32x4 *>(lds.kv + own) + lane;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mine_o[64 * (4 * d + e)] = f32x4{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
            if (h2 == 0) lds.stat[wave][col] = f32x2{m, l};
            const int slot = share(piece, row0, rows, shared);
            __syncthreads();
            for (int i = wave; i < 4 * DB; i += WAVES) {
                Joined sum = Joined::none();
#pragma unroll
                for (int x = 0; x < WAVES; ++x) {
                    const f32x2 s = lds.stat[x][col];
                    sum.add(s.x, s.y, reinterpret_cast<const f32x4 *>(lds.kv + x * (2 * L::OWN))[64 * i + lane], scale_log2);
                }
                if (slot >= 0) {
                    *reinterpret_cast<f32x4 *>(part + (int64_t)slot * WAVES * (32 * D) + 256 * i + 4 * lane) = sum.o;
                    if (i == 0 && h2 == 0) {
                        const int64_t r = (int64_t)slot * kRows + col;
                        stat[2 * r] = sum.m;
                        stat[2 * r + 1] = sum.l;
                    }
                } else if (col < rows) {
                    const float inv = sum.l > 0.0f ? 1.0f / sum.l : 0.0f;
                    *reinterpret_cast<u32x2 *>(a.out + ((int64_t)(at.s.q0 + tok) * a.H + at.g * a.group + sub) * D +
                                               8 * i + 4 * h2) =
                        u32x2{pack_bf16x2(sum.o.x * inv, sum.o.y * inv), pack_bf16x2(sum.o.z * inv, sum.o.w * inv)};
                }
            }
            __syncthreads();
            if (!piece.next(a)) return;
            continue;
        }
        pass(std::false_type());
        float z = 0.0f;                            // NaN where something is not finite
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) z = __builtin_fmaf(o[d][e], 0.0f, z);
        // (every wave has left the buffers behind these barriers)
        if (__builtin_expect(__syncthreads_or(masked && z != z), 0)) {
            pass(std::true_type());
            __syncthreads();
        }

        l = sum_both_halves(l);
        const int slot = share(piece, row0, rows, shared);
        if (slot >= 0) {
            // Unnormalized sums, as the lanes hold them: [slot][wave][8 columns][lane][4] fp32, and
            // maximum and sum of the weights [slot][row][2].
            float *p = part + ((int64_t)slot * WAVES + wave) * (32 * D) + 4 * lane;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<f32x4 *>(p + (4 * d + e) * 256) =
                        f32x4{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
            if (h2 == 0) {
                const int64_t r = (int64_t)slot * kRows + mine;
                stat[2 * r] = m;
                stat[2 * r + 1] = l;
            }
        } else {
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            // A lane holds d = 32 db + 8 e + 4 h2 + (0 .. 3) of its row; the swap of
            // the lane halves gives each eight consecutive ones: 16-byte stores.
            uint16_t *dst = a.out + ((int64_t)(at.s.q0 + tok) * a.H + at.g * a.group + sub) * D;
            const bool in = mine < rows;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    u32x2 x[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        x[u] = u32x2{pack_bf16x2(o[d][4 * (e + u)] * inv, o[d][4 * (e + u) + 1] * inv),
                                     pack_bf16x2(o[d][4 * (e + u) + 2] * inv, o[d][4 * (e + u) + 3] * inv)};
                    const auto s0 = __builtin_amdgcn_permlane32_swap(x[0].x, x[1].x, false, false);
                    const auto s1 = __builtin_amdgcn_permlane32_swap(x[0].y, x[1].y, false, false);
                    if (in)
                        *reinterpret_cast<u32x4 *>(dst + 32 * d + 8 * (e + h2)) =
                            u32x4{(uint32_t)s0[0], (uint32_t)s1[0], (uint32_t)s0[1], (uint32_t)s1[1]};
                }
        }
        if (!piece.next(a)) return;
    }
}

// Joins the shared tiles: a workgroup per slot.  A tile is WAVES x D / 32 items of 32 rows
// and 32 columns, of which the i-th of P parts takes the i-th of P ranges; 128 threads
// an item, which read whole kilobytes of a part as its wave wrote them.  Tiles of 256 rows,
// which seldom have many parts: four items at once, since an item's loads wait for the one
// before (57 MB 15.4 us; two at once 18.5, eight 15.4).  Tiles of 128: two (9.6 us, as four) and
// four parts at once: tiles of 64 parts take 41 us with their attention, 48 one at a time.
template <int WAVES>
constexpr int kJoinThreads = 64 * WAVES;

template <int D, int WAVES>
__global__ void __launch_bounds__(kJoinThreads<WAVES>)
join_tiles_kernel(SpanArgs a, const Shared *__restrict__ shared, const float *__restrict__ part,
                  const float *__restrict__ stat) {
    constexpr int DB = D / 32, ITEMS = WAVES * DB;
    const Shared sh = shared[blockIdx.x];
    if (sh.parts == 0) return;
    const int i0 = ITEMS * sh.index / sh.parts, i1 = ITEMS * (sh.index + 1) / sh.parts;
    const int col = threadIdx.x & 31, e = (threadIdx.x >> 5) & 3;
    const int64_t w = (blockIdx.x >> 1) - sh.index;         // the piece with part 0
    for (int item = i0 + (threadIdx.x >> 7); item < i1; item += kJoinThreads<WAVES> / 128) {
        const int wave = item / DB, db = item % DB, r = 32 * wave + col;
        if (r >= sh.rows) continue;
        Joined lo = Joined::none(), hi = Joined::none();    // 4 columns each
#pragma unroll 4
        for (int i = 0; i < sh.parts; ++i) {
            const int64_t slot = i == 0 ? 2 * w + 1 : 2 * (w + i);
            const f32x2 s = *reinterpret_cast<const f32x2 *>(stat + 2 * (slot * (32 * WAVES) + r));
            const float *p = part + (slot * WAVES + wave) * (32 * D) + (4 * db + e) * 256 + 4 * col;
            lo.add(s.x, s.y, *reinterpret_cast<const f32x4 *>(p), a.scale_log2);
            hi.add(s.x, s.y, *reinterpret_cast<const f32x4 *>(p + 128), a.scale_log2);
        }
        const float inv = lo.l > 0.0f ? 1.0f / lo.l : 0.0f;
        *reinterpret_cast<u32x4 *>(joined_row<D>(a, sh, r) + 32 * db + 8 * e) =
            u32x4{pack_bf16x2(lo.o.x * inv, lo.o.y * inv), pack_bf16x2(lo.o.z * inv, lo.o.w * inv),
                  pack_bf16x2(hi.o.x * inv, hi.o.y * inv), pack_bf16x2(hi.o.z * inv, hi.o.w * inv)};
    }
}

// Workers: as many workgroups as the compute units hold at once, two waves to a SIMD, or fewer
// where even the most keys that the shape allows make fewer pieces.
template <int D, int WAVES>
int workers(const SpanArgs &a) { return span_workers<32 * WAVES>(a, 2048 / WAVES); }

// Tiles of 256 rows read K and V half as often as tiles of 128, and fill less well.  128 | 256, us:
// Packed, with many pairs of a row and a key (half of them seen with `causal`), 256.  D = 128: 32
// heads on 8, causal, one prompt of 1000 39.8 | 43.5, 2000 67 | 68, 4000 174 | 171, 8000 530 | 515;
// twelve of 1 to 2000 103 | 107; 24 heads, four images of 777 to 4096 342 | 317.
// Paged, where the call does not know how many keys there are, with many rows.  D = 128: 12 heads,
// 2 x 1560 rows over 32760 734 | 677; 32 heads on 8, 40 over 4000 28.0 | 31.2, 512 over 4608 65.9 |
// 65.9, 48 decoding requests and 1000 new 82 | 78; D = 64: 28 heads on 4, 512 over 4608 beside
// 31 decoding requests 46 | 49, 48 decoding and 1000 new 31 | 37; 12 heads, 2 x 1560 over 32760
// 425 | 406; 32 on 4, 2048 over 20000 406 | 373.
// The lengths are the device's alone, so the rule for packed ones takes their mean, and a long sequence
// among many short or empty ones gets tiles of 128: 16384 tokens beside 40 of one token 2160 | 1960,
// 8192 beside them 566 | 522, the four images beside 28 empty ones 335 | 306 (beside 8 of 500 tokens
// 16384 pass the rule).
bool wide(const SpanArgs &a) {
    if (a.max_new > 0) return (double)a.T * a.H * a.D >= 0x1p21;
    const double pairs = (double)a.T * (double)a.Tk / a.B * a.H;
    return pairs >= (a.causal ? 0x1p28 : 0x1p27);
}

template <int D>
size_t bytes(const SpanArgs &a) {
    return wide(a) ? Workspace<D, 256>::bytes(workers<D, 8>(a)) : Workspace<D, 128>::bytes(workers<D, 4>(a));
}

template <int D, bool PAGED, int WAVES>
hipError_t launch(const SpanArgs &a, void *ws, hipStream_t stream) {
    constexpr int R = 32 * WAVES;
    const int n = workers<D, WAVES>(a);
    const Workspace<D, R> s(ws, n);
    span_attention_kernel<D, PAGED, WAVES><<<n, 64 * WAVES, 0, stream>>>(a, s.shared, s.part, s.stat);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || n == 1 || !may_share<R>(a)) return e;
    join_tiles_kernel<D, WAVES><<<2 * n, kJoinThreads<WAVES>, 0, stream>>>(a, s.shared, s.part, s.stat);
    return hipGetLastError();
}

template <int D>
hipError_t launch(const SpanArgs &a, void *ws, hipStream_t stream) {
    if (a.kv_len) return wide(a) ? launch<D, true, 8>(a, ws, stream) : launch<D, true, 4>(a, ws, stream);
    return wide(a) ? launch<D, false, 8>(a, ws, stream) : launch<D, false, 4>(a, ws, stream);
}

}  // namespace span

size_t span_tile_workspace(const SpanArgs &a) { return a.D == 64 ? span::bytes<64>(a) : span::bytes<128>(a); }

hipError_t launch_span_tiles(const SpanArgs &a, void *ws, hipStream_t stream) {
    return a.D == 64 ? span::launch<64>(a, ws, stream) : span::launch<128>(a, ws, stream);
}

}  // namespace svdq
