// span_few.hip -- attention of few new tokens over a paged cache: at most 16 or 32
// rows of a request and key head (row r: head r % group of token r / group), on
// the bf16 matrix instruction (v_mfma_f32_16x16x32_bf16).
//
// Bound by reading the cache once.  A workgroup is one wave, and goes over its piece of
// the line of all tiles (span_plan.h) in units of 32 keys: K and V go from global
// memory straight into the wave's own two LDS buffers, so a unit or two of each wave
// are in flight at any time and no wave waits for another.  Scores are computed
// transposed, S^T = K Q^T: a lane holds eight keys of one row, the maximum takes two
// lane exchanges, and the weights come out as the operand of O^T = V^T P^T.
//
// 32 heads on 8 of 128: one token over 65537 keys 50 us and 6.5 for the join (268 MB, 5.4 TB/s
// while it reads), 64 tokens over 9 to 8192 keys 62 and 5 (328 MB, 5.3 TB/s).  With workgroups of
// four waves that share blocks of 64 keys the calls took 76 and 78 us where the first form of
// this kernel took 63 and 72: a barrier waits for the slowest copy.
#include "attention_tile.h"
#include "span_plan.h"

#include <type_traits>

namespace svdq {

namespace few {

using namespace attn;

constexpr int kUnit = 32;                          // keys

template <int D>
struct Lds {
    static constexpr int TILE = kUnit * D * 2;     // bytes of K or V of a unit
    uint8_t k[2][TILE];
    uint8_t v[2][TILE];
    Seq seqs[64];
};

// Both other 16-lane groups' and the other half's: the largest of the four lanes of a row.
__device__ __forceinline__ float max_of_row(float x) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max_both_halves(fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])));
}
__device__ __forceinline__ float sum_of_row(float x) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return sum_both_halves(__uint_as_float(p[0]) + __uint_as_float(p[1]));
}

// LDS layout of V: the eight rows and two 16-byte segments that 32 lanes of the
// transposing read touch lie in different banks.
template <int D>
__device__ __forceinline__ int swz_few(int row) {
    return D == 128 ? 2 * (row & 7) : 2 * ((row >> 1) & 3);
}

template <int D, int NR>
__global__ void __launch_bounds__(64, D == 64 ? 2 : 1)
few_attention_kernel(SpanArgs a, Shared *__restrict__ shared, float *__restrict__ part, float *__restrict__ stat) {
    constexpr int R = 16 * NR, DK = D / 32, DT = D / 16;
    constexpr int RPT = 512 / D, SEGS = D / 8;     // rows per 1 KB copy, 16-byte segments of a row
    constexpr int COPIES = 16 / RPT;               // of 16 keys, K and V each
    __shared__ __align__(1024) Lds<D> lds;
    const int lane = threadIdx.x, g4 = lane >> 4, c16 = lane & 15;
    const int w = blockIdx.x;
    if (lane == 0) shared[2 * w].parts = shared[2 * w + 1].parts = 0;
    Piece<R> piece;
    if (!piece.open(a, lds.seqs, w, (int)gridDim.x)) return;
    Place<R> &at = piece.at;

    const int cp_row = lane / SEGS, cp_slot = lane % SEGS;
    uint32_t k_at[COPIES], v_at[COPIES];           // bytes from the first of 16 keys
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
        const int row = c * RPT + cp_row;
        k_at[c] = row * (D * 2) + 16 * (cp_slot ^ swz_k<D>(row));
        v_at[c] = row * (D * 2) + 16 * (cp_slot ^ swz_few<D>(row));
    }
    const uint8_t *k_rd[DK], *v_rd[DT];
#pragma unroll
    for (int s = 0; s < DK; ++s) k_rd[s] = lds.k[0] + c16 * (D * 2) + 16 * ((4 * s + g4) ^ swz_k<D>(c16));
    {
        const int row = 4 * g4 + (c16 >> 2);
#pragma unroll
        for (int d = 0; d < DT; ++d)
            v_rd[d] = lds.v[0] + row * (D * 2) + 16 * ((2 * d + ((c16 & 3) >> 1)) ^ swz_few<D>(row)) + 8 * (c16 & 1);
    }
    const uint32_t lds_k = lds_address(lds.k), lds_v = lds_address(lds.v);
    const float scale_log2 = a.scale_log2;
    const uint8_t *kb = reinterpret_cast<const uint8_t *>(a.k), *vb = reinterpret_cast<const uint8_t *>(a.v);

    for (;;) {
        const int64_t row0 = (int64_t)at.t * R, rows_left = (int64_t)at.s.nq * a.group - row0;
        if (rows_left <= 0) return;                // (lengths that changed under the call)
        const int rows = rows_left < R ? (int)rows_left : R;
        const int tok0 = token_of(a, (double)row0), rem0 = (int)(row0 - (int64_t)tok0 * a.group);
        const int nk = at.s.nk;
        int limit[NR], to_tok[NR], to_sub[NR];
        u32x4 qf[NR][DK];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = 16 * r + c16 < rows ? 16 * r + c16 : rows - 1;   // past the last: never stored
            const int ahead = token_of(a, rem0 + row);
            to_tok[r] = tok0 + ahead;
            to_sub[r] = rem0 + row - ahead * a.group;
            // keys that the row sees: no more than the rows behind it
            const int n = a.causal ? nk - at.s.nq + 1 + to_tok[r] : nk;
            limit[r] = n < 0 ? 0 : n < nk ? n : nk;
            const uint16_t *p = a.q + (int64_t)(at.s.q0 + to_tok[r]) * a.q_stride +
                                (int64_t)(at.g * a.group + to_sub[r]) * D + 8 * g4;
#pragma unroll
            for (int s = 0; s < DK; ++s) qf[r][s] = *reinterpret_cast<const u32x4 *>(p + 32 * s);
        }
        const int low = __builtin_amdgcn_readlane(limit[0], 0), high = __builtin_amdgcn_readlane(limit[NR - 1], 15);

        const int first = 2 * piece.first, seen = (high + kUnit - 1) / kUnit;
        const int last = 2 * piece.last < seen ? 2 * piece.last : seen;   // units
        const int32_t *table = a.tables + (int64_t)at.b * a.width;
        // Lane l: the page of 16 keys, window 64 i0 + l.
        int pages = -1, pages_next = -1;
        uint64_t bad16 = 0;
        auto read_pages = [&](int i0) __attribute__((always_inline)) {
            const int n = (64 * i0 + lane) * 16;
            return n < nk ? table[n >> a.page_shift] : -1;
        };
        auto take_pages = [&](int i0, int p) __attribute__((always_inline)) {
            const bool good = p >= 0 && p < a.pages;
            pages = good ? p : -1;
            bad16 = __ballot(!good && (64 * i0 + lane) * 16 < nk);
        };
        bool full[2];                              // the buffer's copies were all issued
        uint32_t bad[2];
        // Rows at or past the sequence's keys, and those without a page, are not read: K is left as
        // it is (its scores are masked, whatever they are), V is zero (the weights are zero,
        // and zero times what is not finite would be NaN).
        auto issue = [&](int u, auto buffer) __attribute__((always_inline)) {
            constexpr int BUF = decltype(buffer)::value;
            if (u == first) {
                take_pages(u >> 5, read_pages(u >> 5));
                pages_next = read_pages((u >> 5) + 1);
            } else if ((u & 31) == 0) {
                take_pages(u >> 5, pages_next);
                pages_next = read_pages((u >> 5) + 1);
            }
            bad[BUF] = (uint32_t)(bad16 >> (2 * (u & 31))) & 3u;
            full[BUF] = true;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n0 = u * kUnit + 16 * h;
                const int page = __builtin_amdgcn_readlane(pages, 2 * (u & 31) + h);
                const int left = page < 0 ? 0 : nk - n0;
                const int64_t r = ((((int64_t)page * a.G + at.g) << a.page_shift) +
                                   (n0 & ((1 << a.page_shift) - 1))) * (D * 2);
                const uint8_t *k0 = kb + r, *v0 = vb + r;
                const uint32_t kd = lds_k + BUF * Lds<D>::TILE + h * 16 * D * 2;
                const uint32_t vd = lds_v + BUF * Lds<D>::TILE + h * 16 * D * 2;
                if (__builtin_expect(left >= 16, 1)) {
                    copies_in_flight(k0, k_at, kd);
                    copies_in_flight(v0, v_at, vd);
                } else {
                    full[BUF] = false;
#pragma unroll
                    for (int c = 0; c < COPIES; ++c) {
                        if (c * RPT + cp_row < left) {
                            copy_in_flight(k0, k_at[c], kd + c * 1024);
                            copy_in_flight(v0, v_at[c], vd + c * 1024);
                        } else {
                            *reinterpret_cast<u32x4 *>(lds.v[BUF] + h * 16 * D * 2 + c * 1024 + lane * 16) = u32x4{};
                        }
                    }
                }
            }
        };

        auto start = [&]() __attribute__((always_inline)) {
            if (first < last) issue(first, std::integral_constant<int, 0>());
            if (first + 1 < last) issue(first + 1, std::integral_constant<int, 1>());
        };
        start();
        // A row with a value that is not finite becomes a row of NaN: scores of minus infinity
        // alone would look like keys that it does not see.
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            uint32_t odd = 0;
#pragma unroll
            for (int s = 0; s < DK; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) odd |= not_finite(qf[r][s][j]);
            uint64_t odds = __ballot(odd != 0);
            odds |= odds >> 32;
            if (odds && ((odds >> c16 | odds >> (c16 + 16)) & 1))
#pragma unroll
                for (int s = 0; s < DK; ++s)
                    qf[r][s] = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
        }

        f32x4 o[DT][NR];
        float m[NR], l[NR];
        bool masked = false;
        // CAREFUL: once more, with values of v that are not finite taken out of the units that
        // have a mask (zero times such a value would reach the rows that do not see its key),
        // and a NaN put where a row sees one of them, whatever its weight: in the units
        // without a mask a weight of zero gives one too.
        auto pass = [&](auto mode) __attribute__((always_inline)) {
            constexpr bool careful = decltype(mode)::value;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                m[r] = -__builtin_inff();
                l[r] = 0.0f;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[d][r] = f32x4{};
            }
            auto unit = [&](int u, auto buffer) __attribute__((always_inline)) {
                constexpr int BUF = decltype(buffer)::value, AT = BUF * Lds<D>::TILE;
                const int n0 = u * kUnit;
                // this unit's copies: all but the other buffer's, which follow them
                if (u + 1 < last && full[1 - BUF])
                    wait_loads<4 * COPIES>();
                else
                    wait_loads<0>();
                asm volatile("" ::: "memory");
                f32x4 s[2][NR];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < NR; ++r) s[t][r] = f32x4{};
#pragma unroll
                for (int x = 0; x < DK; ++x)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const u32x4 kf = *reinterpret_cast<const u32x4 *>(k_rd[x] + AT + t * 16 * D * 2);
#pragma unroll
                        for (int r = 0; r < NR; ++r) s[t][r] = mfma_bf16_16x16x32(kf, qf[r][x], s[t][r]);
                    }
                const bool edge = n0 + kUnit > low || bad[BUF] != 0;
                if (edge) {
                    masked = true;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int n = n0 + 16 * t + 4 * g4 + e;
#pragma unroll
                            for (int r = 0; r < NR; ++r)
                                if (n >= limit[r] || (bad[BUF] >> t & 1)) s[t][r][e] = -__builtin_inff();
                        }
                }
                u32x4 p[NR], seen[NR];
                if (careful && edge)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            seen[r][x] = seen_pair(n0 + 16 * (x / 2) + 4 * g4 + 2 * (x & 1),
                                                   bad[BUF] >> (x / 2) & 1 ? 0 : limit[r]);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float top = s[0][r][0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e / 4][r][e % 4]);
                    top = max_of_row(top);
                    // The running maximum moves only when a score passes it by more than 8 in the
                    // exponent of two.
                    if (__any((top - m[r]) * scale_log2 > 8.0f)) {
                        const float m1 = fmaxf(m[r], top);
                        const float f = m[r] == m1 ? 1.0f : __builtin_amdgcn_exp2f((m[r] - m1) * scale_log2);
                        m[r] = m1;
                        l[r] *= f;
#pragma unroll
                        for (int d = 0; d < DT; ++d) o[d][r] *= f;
                    }
                    // A weight's exponent is (s - m) c where |m c| is large (exact where a weight
                    // counts), otherwise s c - fl(m c) in one operation.  A row without a key so
                    // far has m = -inf and no offset.
                    float off = m[r] * scale_log2;
                    const bool far = fabsf(off) > 1024.0f;
                    if (__any(far)) {
                        const float by = far && m[r] > -__builtin_inff() ? m[r] : 0.0f;
                        off = far ? 0.0f : off;
#pragma unroll
                        for (int e = 0; e < 8; ++e) s[e / 4][r][e % 4] -= by;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        s[e / 4][r][e % 4] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e / 4][r][e % 4], scale_log2, -off));
                    // weights rounded to bf16, the operand beside V; the same go into their sum
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        p[r][x] = pack_bf16x2(s[x / 2][r][2 * (x & 1)], s[x / 2][r][2 * (x & 1) + 1]);
                        l[r] = add_pair(p[r][x], l[r]);
                    }
                }
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    u32x4 vf;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const u32x2 y = read_transposed(v_rd[d] + AT + 16 * x * (D * 2));
                        vf[2 * x] = y.x;
                        vf[2 * x + 1] = y.y;
                    }
                    u32x4 odd = {};
                    if (careful && edge)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t f = not_finite(vf[j]);        // 0x8000 of each half
                            odd[j] = (f >> 15) * 0x3F80u;
                            vf[j] &= ~((f >> 15) * 0xFFFFu);
                        }
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        o[d][r] = mfma_bf16_16x16x32(vf, p[r], o[d][r]);
                        if (careful && edge) {
                            const f32x4 c = mfma_bf16_16x16x32(odd, seen[r], f32x4{});
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (c[e] > 0.0f) o[d][r][e] = __builtin_nanf("");
                        }
                    }
                }
                // the buffer has been read: the unit after the next may go there
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                if (u + 2 < last) issue(u + 2, buffer);
            };
            if (careful) start();
            for (int u = first; u < last; u += 2) {
                unit(u, std::integral_constant<int, 0>());
                if (u + 1 < last) unit(u + 1, std::integral_constant<int, 1>());
            }
        };
        pass(std::false_type());
        float z = 0.0f;                            // NaN where something is not finite
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) z = __builtin_fmaf(o[d][r][e], 0.0f, z);
        if (__builtin_expect(__any(masked && z != z), 0)) pass(std::true_type());

        const int slot = share(piece, row0, rows, shared);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = 16 * r + c16;
            const float sum = sum_of_row(l[r]);
            if (row >= rows) continue;
            if (slot < 0) {
                const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
                uint16_t *dst = a.out + ((int64_t)(at.s.q0 + to_tok[r]) * a.H + at.g * a.group + to_sub[r]) * D + 4 * g4;
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    *reinterpret_cast<u32x2 *>(dst + 16 * d) =
                        u32x2{pack_bf16x2(o[d][r][0] * inv, o[d][r][1] * inv), pack_bf16x2(o[d][r][2] * inv, o[d][r][3] * inv)};
            } else {
                const int64_t x = (int64_t)slot * R + row;
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    *reinterpret_cast<f32x4 *>(part + x * D + 16 * d + 4 * g4) = o[d][r];
                if (g4 == 0) {
                    stat[2 * x] = m[r];
                    stat[2 * x + 1] = sum;
                }
            }
        }
        if (!piece.next(a)) return;
    }
}

// Joins the shared tiles: a workgroup per slot, the i-th of a tile's P parts taking the
// i-th of P ranges of its rows, so that the parts' rows are spread over as many.  D / 4
// lanes per row; where a range has fewer rows than there are such groups of lanes
// (a row of hundreds of parts), several groups take a row's parts in turn and are
// joined through LDS.
template <int D, int R>
__global__ void __launch_bounds__(256)
join_rows_kernel(SpanArgs a, const Shared *__restrict__ shared, const float *__restrict__ part,
                 const float *__restrict__ stat) {
    constexpr int LANES = D / 4, GROUPS = 256 / LANES;
    __shared__ Joined sums[GROUPS][LANES];
    const Shared sh = shared[blockIdx.x];
    if (sh.parts == 0) return;
    const int r0 = (int)((int64_t)sh.rows * sh.index / sh.parts), r1 = (int)((int64_t)sh.rows * (sh.index + 1) / sh.parts);
    const int grp = threadIdx.x / LANES, c = threadIdx.x % LANES;
    const int64_t w = (blockIdx.x >> 1) - sh.index;         // the piece with part 0
    int ways = 1;
    while (2 * ways * (r1 - r0) <= GROUPS && 2 * ways <= GROUPS) ways *= 2;
    for (int row = r0; row < r1; row += GROUPS / ways) {    // (once, where ways > 1)
        const int r = row + grp / ways;
        Joined j = Joined::none();
        if (r < r1) {
            for (int i = grp % ways; i < sh.parts; i += 8 * ways) {
                f32x2 s[8];
                f32x4 o[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {               // (8 parts in flight; the last again behind it)
                    const int k = i + u * ways < sh.parts ? i + u * ways : i;
                    const int64_t x = (k == 0 ? 2 * w + 1 : 2 * (w + k)) * R + r;
                    s[u] = *reinterpret_cast<const f32x2 *>(stat + 2 * x);
                    o[u] = *reinterpret_cast<const f32x4 *>(part + x * D + 4 * c);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (i + u * ways < sh.parts) j.add(s[u].x, s[u].y, o[u], a.scale_log2);
            }
        }
        if (ways > 1) {
            sums[grp][c] = j;
            __syncthreads();
            if (grp % ways != 0) return;
            for (int i = 1; i < ways; ++i) {
                const Joined &x = sums[grp + i][c];
                j.add(x.m, x.l, x.o, a.scale_log2);
            }
        }
        if (r >= r1) continue;
        const float inv = j.l > 0.0f ? 1.0f / j.l : 0.0f;
        *reinterpret_cast<u32x2 *>(joined_row<D>(a, sh, r) + 4 * c) =
            u32x2{pack_bf16x2(j.o.x * inv, j.o.y * inv), pack_bf16x2(j.o.z * inv, j.o.w * inv)};
    }
}

// Workers: two to a compute unit (four at D = 64), which keep enough copies in flight, or
// twice as many where there is a tile for each.  D = 128, 512 | 1024 workers, us with the join:
// one token over 65537 keys 58 | 63, 64 over 9 to 8192 72 | 74, 256 over 1000 197 | 192, 256 over
// 4000 723 | 708; D = 64, 1024 | 2048: one over 65537 37 | 43.
template <int D, int NR>
int workers(const SpanArgs &a) {
    const int64_t tiles = (a.B < a.T ? a.B : a.T) * (int64_t)a.G;
    const int most = D == 64 ? 1024 : 512;
    return span_workers<16 * NR>(a, tiles < 2 * most ? most : 2 * most);
}

template <int D, int NR>
hipError_t launch(const SpanArgs &a, void *ws, hipStream_t stream) {
    constexpr int R = 16 * NR;
    const int n = workers<D, NR>(a);
    const Workspace<D, R> s(ws, n);
    few_attention_kernel<D, NR><<<n, 64, 0, stream>>>(a, s.shared, s.part, s.stat);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || n == 1 || !may_share<R>(a)) return e;
    join_rows_kernel<D, R><<<2 * n, 256, 0, stream>>>(a, s.shared, s.part, s.stat);
    return hipGetLastError();
}

}  // namespace few

size_t span_few_workspace(const SpanArgs &a) {
    const bool one = (int64_t)a.max_new * a.group <= 16;
    if (a.D == 64)
        return one ? Workspace<64, 16>::bytes(few::workers<64, 1>(a)) : Workspace<64, 32>::bytes(few::workers<64, 2>(a));
    return one ? Workspace<128, 16>::bytes(few::workers<128, 1>(a)) : Workspace<128, 32>::bytes(few::workers<128, 2>(a));
}

hipError_t launch_span_few(const SpanArgs &a, void *ws, hipStream_t stream) {
    const bool one = (int64_t)a.max_new * a.group <= 16;
    if (a.D == 64) return one ? few::launch<64, 1>(a, ws, stream) : few::launch<64, 2>(a, ws, stream);
    return one ? few::launch<128, 1>(a, ws, stream) : few::launch<128, 2>(a, ws, stream);
}

}  // namespace svdq
