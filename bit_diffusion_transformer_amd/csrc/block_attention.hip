// block_attention.hip -- attention of blocks of 128 queries over lists of key
// blocks of 64, on the bf16 matrix instruction (v_mfma_f32_32x32x16_bf16).
//
// One workgroup of four waves per query block and head, 32 queries a wave.
// Scores are computed transposed, S^T = K Q^T, so that a lane holds the scores
// of one query (column l % 32, half of the block's keys; lane l ^ 32 the other
// half): the running maximum and sum of the softmax stay within the lane but
// for one exchange, and the weights P^T come out in the lane layout that the
// second product, O^T = V^T P^T, takes as its operand, without a pass through
// LDS (its order of keys within a step is that of the score tile's rows, and
// the V operand is read in the same order).  K and V blocks go from global
// memory straight into LDS (two buffers, the next block's copies in flight
// while the current one is used); K is read in 16-byte pieces, V through the
// transposing 8-byte LDS read.
//
// Calls in a row, on two cards.  12 heads of 32760 queries, 64 of 512 blocks each, D =
// 128: 854-870 us, 0.95-0.97 PFLOP/s (a faster card takes 5 % less with its selection);
// 48 heads of 4608, 24 of 72 blocks: 198-204 us; 24 heads of 16384, 32 of 256 blocks,
// D = 64: 248-252 us.  Bound by power: all-zero inputs take 637 us for the first of
// these, in as many cycles (1.5 million) at 2.4 GHz that random ones get at 1.85.  The
// parts add up: on a card where the whole takes 800 us, the two products and their LDS
// reads alone take 609, the softmax 111 more, the copies (32 KB per 128 x 64 scores)
// the rest.  Two waves share a SIMD; a wave's key block costs it 790 cycles to issue
// copies, 770 for S, 1190 for the softmax, 1130 for the second product and 130 at the
// barrier.
#include "attention_internal.h"
#include "svdq_wave.h"

#include <type_traits>

namespace svdq {

namespace attn {

constexpr int kQB = SVDQ_QUERY_BLOCK, kKB = SVDQ_KEY_BLOCK;
constexpr int kMaxList = SVDQ_MAX_KEYS / SVDQ_KEY_BLOCK;

typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// c plus the two bf16 values of x (products with one): the sum of the weights as
// they enter the second product, rounded, in half the instructions.
__device__ __forceinline__ float add_pair(uint32_t x, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x),
                                           __builtin_bit_cast(bf16x2, 0x3F803F80u), c, false);
}
__device__ __forceinline__ float max_both_halves(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float sum_both_halves(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// LDS layout of a K or V block: rows of D values, 16-byte segments XORed by a
// function of the row.  K: eight (sixteen) consecutive rows of one segment hit
// different banks.  V: four consecutive rows of four neighbouring segments do
// (what 32 lanes of the transposing read touch).
template <int D>
__device__ __forceinline__ int swz_k(int row) {
    return D == 128 ? row & 15 : (row & 7) ^ ((row >> 3) & 1);
}
template <int D>
__device__ __forceinline__ int swz_v(int row) {
    return D == 128 ? 4 * (row & 3) : 2 * (row & 3);
}

// Transposing LDS read: within each 16 lanes, lane i supplies 8 bytes (4 columns)
// of row i / 4 and receives column i of the four rows.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t *p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p));
}

template <int D>
struct Lds {
    static constexpr int TILE = kKB * D * 2;      // bytes of a K or V block
    uint8_t k[2][TILE];
    uint8_t v[2][TILE];
    uint16_t list[kMaxList];
    // The list's length, until the first copies into this buffer (after the first
    // key block's barrier): at D = 64 four workgroups' LDS are 160 KB exactly.
    __device__ int *count() { return reinterpret_cast<int *>(v[1]); }
};

// The list's usable entries, in order: not negative, below `valid`, above every
// entry before them; without a list, 0 .. valid - 1, which goes to `made` (keep
// entries) if that is given.  By the first wave.
__device__ __forceinline__ void read_list(const int32_t *__restrict__ blocks, int keep, int valid,
                                          uint16_t *list, int *count, int32_t *made) {
    const int lane = threadIdx.x & 63;
    if (!blocks) {
        for (int i = lane; i < valid; i += 64) list[i] = (uint16_t)i;
        if (made)
            for (int i = lane; i < keep; i += 64) made[i] = i < valid ? i : -1;
        if (lane == 0) *count = valid;
        return;
    }
    int n = 0, top = -1;
    for (int i0 = 0; i0 < keep; i0 += 64) {
        const int e = i0 + lane < keep ? blocks[i0 + lane] : -1;
        int best = e;                              // inclusive running maximum
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(best, d);
            if (lane >= d) best = o > best ? o : best;
        }
        int before = __shfl_up(best, 1);
        before = lane == 0 || before < top ? top : before;
        const bool take = e >= 0 && e < valid && e > before;
        const uint64_t taken = __ballot(take);
        if (take) list[n + __popcll(taken & ((1ull << lane) - 1))] = (uint16_t)e;
        n += __popcll(taken);
        const int last = __shfl(best, 63);
        top = last > top ? last : top;
    }
    if (lane == 0) *count = n;
}

// Two workgroups per compute unit at D = 128 (LDS and registers); four at D = 64
// (24 heads of 16384, 32 blocks each: 262 us, three take 270).
template <int D, bool SPLIT>
__global__ void __launch_bounds__(256, D == 64 ? 4 : 2)
block_attention_kernel(const uint16_t *__restrict__ q, const uint16_t *__restrict__ k,
                       const uint16_t *__restrict__ v, const int32_t *__restrict__ kv_len,
                       AttnShape a, float scale_log2, const int32_t *__restrict__ blocks,
                       int32_t *__restrict__ made, uint16_t *__restrict__ out, int splits,
                       float *__restrict__ part, float *__restrict__ stat) {
    constexpr int DB = D / 32, DK = D / 16;        // 32-wide blocks and 16-wide steps of D
    constexpr int RPT = 512 / D;                   // rows per 1 KB copy
    constexpr int SEGS = D / 8;                    // 16-byte segments of a row
    constexpr int COPIES = kKB / RPT / 4;          // copies per wave, K and V each
    __shared__ __align__(1024) Lds<D> lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h2 = lane >> 5, col = lane & 31;

    // contiguous query blocks per XCD: their lists share key blocks in its L2
    int64_t id = xcd_range(blockIdx.x, a.planes_q * a.nq * (SPLIT ? splits : 1));
    const int piece = SPLIT ? (int)(id % splits) : 0;
    if (SPLIT) id /= splits;
    const int64_t plane = id / a.nq, qi = id - plane * a.nq;
    const int64_t b = plane / a.H, h = plane - b * a.H;
    const int64_t kplane = b * a.G + h / (a.H / a.G);
    int len = (int)a.seq_k;                        // <= 2^18
    if (kv_len) {
        const int n = kv_len[b];
        len = n < 0 ? 0 : n > len ? len : n;
    }
    if (wave == 0)
        read_list(blocks ? blocks + id * a.keep : nullptr, a.keep, (len + kKB - 1) / kKB, lds.list,
                  lds.count(), made && piece == 0 ? made + id * a.keep : nullptr);
    __syncthreads();
    int first = 0, last = *lds.count();
    if (SPLIT) {
        const int n = last;
        first = (int)((int64_t)n * piece / splits);
        last = (int)((int64_t)n * (piece + 1) / splits);
    }

    const uint8_t *kb = reinterpret_cast<const uint8_t *>(k + kplane * a.seq_k * D);
    const uint8_t *vb = reinterpret_cast<const uint8_t *>(v + kplane * a.seq_k * D);
    // Rows at or past the sequence's length are not read: K is left as it is (its scores
    // are masked, whatever they are), V is zero (the weights are zero, and zero times
    // what is not finite would be NaN).
    const int cp_row = wave * COPIES * RPT + lane / SEGS, cp_slot = lane % SEGS;
    uint32_t k_at[COPIES], v_at[COPIES];           // byte offsets within a block
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
        const int row = cp_row + c * RPT;
        k_at[c] = row * (D * 2) + 16 * (cp_slot ^ swz_k<D>(row));
        v_at[c] = row * (D * 2) + 16 * (cp_slot ^ swz_v<D>(row));
    }
    auto issue = [&](int i, auto buffer) {
        constexpr int BUF = decltype(buffer)::value;
        const int n0 = __builtin_amdgcn_readfirstlane(lds.list[i]) * kKB, left = len - n0;
        const uint8_t *k0 = kb + (int64_t)n0 * (D * 2), *v0 = vb + (int64_t)n0 * (D * 2);
        uint8_t *kd = lds.k[BUF] + wave * COPIES * 1024, *vd = lds.v[BUF] + wave * COPIES * 1024;
        if (__builtin_expect(left >= kKB, 1)) {
#pragma unroll
            for (int c = 0; c < COPIES; ++c) {
                copy16_to_lds(k0 + k_at[c], kd + c * 1024);
                copy16_to_lds(v0 + v_at[c], vd + c * 1024);
            }
        } else {                                   // the block of the last key
#pragma unroll
            for (int c = 0; c < COPIES; ++c) {
                const int row = cp_row + c * RPT;
                if (row < left) {
                    copy16_to_lds(k0 + k_at[c], kd + c * 1024);
                    copy16_to_lds(v0 + v_at[c], vd + c * 1024);
                } else {
                    *reinterpret_cast<u32x4 *>(vd + c * 1024 + lane * 16) = u32x4{};
                }
            }
        }
    };
    if (first < last) issue(first, std::integral_constant<int, 0>());

    // This lane's query, rows past the last re-reading it (never stored).
    const int64_t row0 = qi * kQB + wave * 32;
    const bool active = row0 < a.seq_q;            // uniform over the wave
    const int64_t qrow = row0 + col < a.seq_q ? row0 + col : a.seq_q - 1;
    u32x4 qf[DK];
    {
        const uint16_t *p = q + (plane * a.seq_q + qrow) * D + 8 * h2;
#pragma unroll
        for (int s = 0; s < DK; ++s) qf[s] = *reinterpret_cast<const u32x4 *>(p + 16 * s);
    }

    // LDS offsets (of buffer 0): K row `col` (and 32 further), segment 2 t + h2 of
    // step t; V: lane i of a 16-lane group supplies row i / 4 of four keys, 4
    // columns from 4 (i % 4) of the group's 16, and gets column i of the four
    // rows; a step of 16 keys is 16 rows further (the same swizzle).
    const uint8_t *k_rd[DK], *v_rd[DB];
#pragma unroll
    for (int t = 0; t < DK; ++t)
        k_rd[t] = lds.k[0] + col * (D * 2) + 16 * ((2 * t + h2) ^ swz_k<D>(col));
    {
        const int i = lane & 15, row = 4 * h2 + (i >> 2);
        const int sub = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);     // segment of a 32-wide block
#pragma unroll
        for (int d = 0; d < DB; ++d)
            v_rd[d] = lds.v[0] + row * (D * 2) + 16 * ((4 * d + sub) ^ swz_v<D>(row)) + 8 * (lane & 1);
    }

    f32x16 o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] = f32x16{};
    float m = -__builtin_inff(), l = 0.0f;

    auto block = [&](int i, auto buffer) {
        constexpr int BUF = decltype(buffer)::value, AT = BUF * Lds<D>::TILE;
        const int n0 = __builtin_amdgcn_readfirstlane(lds.list[i]) * kKB;
        wait_loads<0>();
        wave_barrier_all();
        if (i + 1 < last) issue(i + 1, std::integral_constant<int, 1 - BUF>());
        if (!active) return;
        f32x16 s[2] = {f32x16{}, f32x16{}};
        {
            // fragments two steps ahead of the products that use them
            u32x4 kf[3][2];
            auto load = [&](int t) {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    kf[t % 3][kk] = *reinterpret_cast<const u32x4 *>(k_rd[t] + AT + 32 * kk * (D * 2));
                }
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
        auto load_v = [&](int st) {
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
        if (n0 + kKB > len) {                      // the sequence ends in this block
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int n = n0 + 32 * kk + 8 * (e / 4) + 4 * h2 + e % 4;
                    if (n >= len) s[kk][e] = -__builtin_inff();
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
            const float f = __builtin_amdgcn_exp2f((m - m1) * scale_log2);
            m = m1;
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[d][e] *= f;
        }
        // A weight's exponent is s c - fl(m c), c = scale log2 e, in one operation: off by
        // the rounding of m c, which all keys of a row share: at most 2^-15 up to |m c| =
        // 2^10, but from 2^32 on more than any exponent of fp32.  Past 2^10 the difference
        // s - m is taken first (exact where a weight counts).  That for every row takes 2 to
        // 3 % longer, this choice 0.1 to 0.8 % (12 heads of 32760 queries, 48 of 4608).
        float off = m * scale_log2;
        const bool far = fabsf(off) > 1024.0f;
        if (__any(far)) {
            const float by = far ? m : 0.0f;
            off = far ? 0.0f : off;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[kk][e] -= by;
        }
        // [kk][step of 16 keys]: weights, rounded to bf16, the type of the matrix instruction's
        // operand beside V.  Rounded once, and the same values go into their sum, so a row's
        // weights still add up to one; the output's error against 64 bits is 0.0023 of its
        // size instead of 0.0017, which its own rounding to bf16 makes.  (A second product of
        // what the rounding leaves would take half as much time again in the products.)
        u32x4 p[2][2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[kk][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kk][e], scale_log2, -off));
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    p[kk][t][w] = pack_bf16x2(s[kk][8 * t + 2 * w], s[kk][8 * t + 2 * w + 1]);
                    l = add_pair(p[kk][t][w], l);
                }
        }
#pragma unroll
        for (int st = 0; st < 4; ++st) {
            if (st < 3) load_v(st + 1);
#pragma unroll
            for (int d = 0; d < DB; ++d) o[d] = mfma_bf16_32x32x16(vf[st & 1][d], p[st >> 1][st & 1], o[d]);
        }
    };
    for (int i = first; i < last; i += 2) {
        block(i, std::integral_constant<int, 0>());
        if (i + 1 < last) block(i + 1, std::integral_constant<int, 1>());
    }
    if (!active) return;

    l = sum_both_halves(l);
    if (SPLIT) {
        // unnormalized sums fp32 [piece][B H Sq][D], maximum and sum [piece][B H Sq][2]
        if (row0 + col < a.seq_q) {
            const int64_t at = (int64_t)piece * a.planes_q * a.seq_q + plane * a.seq_q + row0 + col;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<f32x4 *>(part + at * D + 32 * d + 8 * e + 4 * h2) =
                        f32x4{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
            if (h2 == 0) {
                stat[2 * at] = m;
                stat[2 * at + 1] = l;
            }
        }
        return;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    // A lane holds d = 32 db + 8 e + 4 h2 + (0 .. 3) of its query; the swap of
    // the lane halves gives each eight consecutive ones: 16-byte stores.
    uint16_t *dst = out + ((b * a.seq_q + row0 + col) * a.H + h) * D;
    const bool in = row0 + col < a.seq_q;
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

// Joins the pieces of each row: the largest maximum, weights 2^(m_i - m) on sums
// and results.  D / 4 lanes per row, whose first lanes hold one piece's maximum
// and sum each (D / 4 >= 16 pieces at a time), so that the loads of all pieces
// are in flight together.  32 rows of 8 pieces: 4.6 us, 3 of them the launch.
template <int D>
__global__ void __launch_bounds__(256)
join_kernel(const float *__restrict__ part, const float *__restrict__ stat, AttnShape a, int splits,
            float scale_log2, uint16_t *__restrict__ out) {
    constexpr int LANES = D / 4;
    const int64_t rows = a.planes_q * a.seq_q;
    const int64_t row = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    const int c = threadIdx.x % LANES;
    if (row >= rows) return;                       // whole groups of LANES
    float m = -__builtin_inff(), l = 0.0f;
    f32x4 o = {};
    for (int i0 = 0; i0 < splits; i0 += LANES) {
        const int mine = i0 + c;
        f32x2 s = {-__builtin_inff(), 0.0f};
        if (mine < splits) s = *reinterpret_cast<const f32x2 *>(stat + 2 * (mine * rows + row));
        float top = s.x;
#pragma unroll
        for (int d = LANES / 2; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
        const float m1 = fmaxf(m, top);
        // No maximum yet: pieces without a key, whose sums are zero, or the NaN sums of a
        // query that is not finite, which have to stay.
        const bool none = m1 == -__builtin_inff();
        const float f = none ? 1.0f : __builtin_amdgcn_exp2f((m - m1) * scale_log2);
        const float w = none ? 1.0f : __builtin_amdgcn_exp2f((s.x - m1) * scale_log2);
        m = m1;
        l = l * f + w * s.y;                       // this lane's pieces; summed below
        o *= f;
        const int n = splits - i0 < LANES ? splits - i0 : LANES;
#pragma unroll 8
        for (int i = 0; i < n; ++i)
            o += __shfl(w, (threadIdx.x & 63) - c + i) *
                 *reinterpret_cast<const f32x4 *>(part + ((i0 + i) * rows + row) * D + 4 * c);
    }
#pragma unroll
    for (int d = LANES / 2; d >= 1; d >>= 1) l += __shfl_xor(l, d);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int64_t plane = row / a.seq_q, s = row - plane * a.seq_q;
    const int64_t b = plane / a.H, h = plane - b * a.H;
    *reinterpret_cast<u32x2 *>(out + ((b * a.seq_q + s) * a.H + h) * D + 4 * c) =
        u32x2{pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv)};
}

template <int D>
hipError_t launch(const uint16_t *q, const uint16_t *k, const uint16_t *v, const int32_t *kv_len,
                  const AttnShape &a, float scale, const int32_t *blocks, int32_t *made,
                  uint16_t *out, void *ws, hipStream_t stream) {
    const float c = scale * 1.4426950408889634f;
    const int splits = attention_splits(a);
    const unsigned grid = (unsigned)(a.planes_q * a.nq * splits);
    if (splits == 1) {
        block_attention_kernel<D, false><<<grid, 256, 0, stream>>>(q, k, v, kv_len, a, c, blocks, made,
                                                                   out, 1, nullptr, nullptr);
        return hipGetLastError();
    }
    const int64_t rows = a.planes_q * a.seq_q;
    float *part = static_cast<float *>(ws), *stat = part + rows * splits * D;
    block_attention_kernel<D, true><<<grid, 256, 0, stream>>>(q, k, v, kv_len, a, c, blocks, made, out,
                                                              splits, part, stat);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int per = 256 / (D / 4);
    join_kernel<D><<<(unsigned)((rows + per - 1) / per), 256, 0, stream>>>(part, stat, a, splits, c, out);
    return hipGetLastError();
}

}  // namespace attn

// Few query blocks: their lists are split into pieces, of two key blocks at least,
// for a workgroup each.  The number of pieces with the least time, in ns: a piece's
// key blocks one after another (a second workgroup on a compute unit gains nothing:
// both take twice as long), and the join's launch with its partial results, written
// and read again.  16 heads, D = 128, one piece | the choice: one row, 8 and 32
// blocks 11.9 | 9.3 and 37 | 12.5 us; 300 rows, 16 and 64 blocks 22.4 | 19.6 and 81
// | 30 us; 60 heads of 300 rows, 8 blocks 15.9 (one piece; two take 26.8).  256 is
// the whole card's compute units, not the current device's: the workspace's size
// follows from the result, and has to be the same wherever it is asked for.
int attention_splits(const AttnShape &a) {
    const int64_t wgs = a.planes_q * a.nq, rows = a.planes_q * a.seq_q;
    const int64_t taken = a.keep < a.nk ? a.keep : a.nk, each = a.D == 128 ? 1250 : 900;
    int best = 1;
    int64_t least = 0;
    for (int s = 1; s <= 32 && (s == 1 || (2 * s <= taken && wgs < 256)); ++s) {
        const int64_t full = wgs * s > 256 ? wgs * s : 256;
        const int64_t join = s > 1 ? 3200 + 300 * s + rows * s * a.D / 400 : 0;
        const int64_t ns = (taken + s - 1) / s * each * full / 256 + join;
        if (s == 1 || ns < least) best = s, least = ns;
    }
    return best;
}

size_t attention_workspace(const AttnShape &a) {
    const int s = attention_splits(a);
    return s == 1 ? 0 : align256((size_t)(a.planes_q * a.seq_q) * s * (a.D + 2) * 4);
}

hipError_t launch_block_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                                  const int32_t *kv_len, const AttnShape &a, float scale,
                                  const int32_t *blocks, int32_t *made, uint16_t *out, void *ws,
                                  hipStream_t stream) {
    return a.D == 64 ? attn::launch<64>(q, k, v, kv_len, a, scale, blocks, made, out, ws, stream)
                     : attn::launch<128>(q, k, v, kv_len, a, scale, blocks, made, out, ws, stream);
}

}  // namespace svdq
