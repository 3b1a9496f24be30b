// block_select.hip -- which key blocks each query block attends to: block means
// of Q and K, their products, and the `keep` highest of them.
//
// Means and scores are taken in 64 bits: a list is a discrete choice, and two
// scores that differ by less than the rounding of fp32 sums would choose
// another block there than by the definition.  The work in 64 bits is small
// (one product of D per pair of blocks, 1/8192 of the pairs of rows).
#include "attention_internal.h"
#include "svdq_wave.h"

namespace svdq {

constexpr int kQB = SVDQ_QUERY_BLOCK, kKB = SVDQ_KEY_BLOCK;

__device__ __forceinline__ int64_t valid_keys(const int32_t *kv_len, int64_t b, int64_t seq_k) {
    if (!kv_len) return seq_k;
    const int64_t n = kv_len[b];
    return n < 0 ? 0 : n > seq_k ? seq_k : n;
}

typedef double f64x2 __attribute__((ext_vector_type(2)));
typedef double f64x4 __attribute__((ext_vector_type(4)));

// Means of a head: tiles of 16 blocks; within one, column pair 2 p (p < D / 2)
// of block c is the 16-byte element (p / 4) 64 + (p % 4) 16 + c.
template <int D>
__device__ __forceinline__ int64_t mean_at(int64_t blk, int p) {
    return (blk >> 4) * (8 * D) + (p >> 2) * 64 + (p & 3) * 16 + (blk & 15);
}
__host__ __device__ inline int64_t mean_tiles(int64_t blocks) { return (blocks + 15) / 16; }

// A score as an unsigned key in the same order (-0 as +0), at least 1; a NaN
// counts as the lowest.  Key 0: a block that must not be taken.
__device__ __forceinline__ uint64_t order_key(double x) {
    x += 0.0;
    if (x != x) return 1;
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint64_t o = u >> 63 ? ~u : u | 0x8000000000000000ull;
    return o ? o : 1;
}

// One query block of few rows: the workgroup of a key block sums them itself, in
// its 16 groups of threads (one head each at a time), and stores the block's
// scores instead of its means.  Selection over 20000 keys for 2 x 16 heads (4 of
// keys), by scores | by means: 1 row 18.4 | 23.2 us, 16 rows 21.1 | 23.3 us; 64
// rows of 24 heads (24 of keys) 67 | 38 us.
__host__ __device__ inline bool few_queries(const AttnShape &a) {
    return a.nq == 1 && a.seq_q * ((a.H / a.G + 15) / 16) <= 16;
}

// Means over blocks of rows.  One workgroup per block of one head: 16-byte
// loads, 64 rows' at once, 64-bit sums of eight columns a thread, then sums over
// the threads of a wave and, through LDS, over the waves.  Bound by reading Q and
// K once.  Stored in the order in which the score kernel's matrix
// instruction takes them (mean_at), so that each of its loads is one run.
// 12 heads of 32760 x 128, Q and K: 46 us, 4.4 TB/s; 48 heads of 4608: 28 us.
//
// FEW: one query block of few rows (few_queries).  Workgroups for key blocks
// only; LANES threads a query head then sum its rows, and the block's scores go
// out instead of its means.
template <int D, bool FEW>
__global__ void __launch_bounds__(256)
block_means_kernel(const uint16_t *__restrict__ q, const uint16_t *__restrict__ k,
                   const int32_t *__restrict__ kv_len, AttnShape a, f64x2 *__restrict__ qm,
                   f64x2 *__restrict__ km, uint64_t *__restrict__ scores) {
    constexpr int LANES = D / 8, ROWS = 256 / LANES;   // rows at a time
    __shared__ double part[4][D];
    const int64_t query_wgs = FEW ? 0 : a.planes_q * a.nq;
    // neighbouring blocks' means share cache lines: one XCD writes them
    const int64_t wg = xcd_range(blockIdx.x, query_wgs + a.planes_k * a.nk);
    const bool query = wg < query_wgs;                       // uniform
    const int64_t id = query ? wg : wg - query_wgs;
    const int64_t nb = query ? a.nq : a.nk, size = query ? kQB : kKB;
    const int64_t plane = id / nb, blk = id - plane * nb;
    const int64_t seq = query ? a.seq_q : a.seq_k;
    const int64_t have = query ? a.seq_q : valid_keys(kv_len, plane / a.G, a.seq_k);
    const int64_t left = have - blk * size;
    const int rows = (int)(left < size ? left : size);
    if (rows <= 0) return;                                   // a key block without a valid key
    const int r0 = threadIdx.x / LANES, c = threadIdx.x % LANES;
    auto add = [](double *s, const u32x4 x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[2 * i] += (double)bf16_lo(x[i]);
            s[2 * i + 1] += (double)bf16_hi(x[i]);
        }
    };
    auto row_of = [&](const uint16_t *src, int r) {
        return *reinterpret_cast<const u32x4 *>(src + r * D + 8 * c);
    };
    const int group = a.H / a.G;
    const int64_t head0 = plane / a.G * a.H + plane % a.G * group;   // the first that reads these keys
    u32x4 first = {};                                        // row 0 of the group's first head
    if (FEW && r0 < group) first = row_of(q + (head0 + r0) * a.seq_q * D, 0);
    const uint16_t *src = (query ? q : k) + (plane * seq + blk * size) * D;
    double s[8] = {};
    for (int r = r0; r < rows; r += kKB) {                   // 64 rows' loads at once
        u32x4 x[kKB / ROWS];
#pragma unroll
        for (int i = 0; i < kKB / ROWS; ++i)
            x[i] = row_of(src, r + i * ROWS < rows ? r + i * ROWS : rows - 1);
#pragma unroll
        for (int i = 0; i < kKB / ROWS; ++i) add(s, r + i * ROWS < rows ? x[i] : u32x4{});
    }
    // over the rows of a wave (lanes LANES, 2 LANES .. apart), then over the waves
#pragma unroll
    for (int m = LANES; m < 64; m <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += __shfl_xor(s[i], m);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) < LANES)
#pragma unroll
        for (int i = 0; i < 8; ++i) part[wave][8 * c + i] = s[i];
    __syncthreads();
    double mean[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        mean[i] = (part[0][8 * c + i] + part[1][8 * c + i] + part[2][8 * c + i] +
                   part[3][8 * c + i]) / rows;
    if (!FEW) {
        if (r0 == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                (query ? qm : km)[plane * mean_tiles(nb) * (8 * D) + mean_at<D>(blk, 4 * c + i)] =
                    f64x2{mean[2 * i], mean[2 * i + 1]};
        return;
    }
    for (int h = r0; h < group; h += ROWS) {
        const uint16_t *qh = q + (head0 + h) * a.seq_q * D;
        double t[8] = {}, dot = 0;
        add(t, h == r0 ? first : row_of(qh, 0));
        for (int r = 1; r < a.seq_q; ++r) add(t, row_of(qh, r));
#pragma unroll
        for (int i = 0; i < 8; ++i) dot += t[i] / (double)a.seq_q * mean[i];
#pragma unroll
        for (int m = LANES / 2; m >= 1; m >>= 1) dot += __shfl_xor(dot, m);
        if (c == 0) scores[(head0 + h) * a.nk + blk] = order_key(dot);
    }
}

constexpr int kChooseWaves = 8;

// x OR-ed over the wave, every lane getting it: lane exchanges within 16 lanes,
// then the swaps with the lanes 16 and 32 away.
__device__ __forceinline__ uint32_t wave_or(uint32_t x) {
    x |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true);    // lane ^ 1
    x |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true);    // lane ^ 2
    x |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, true);   // 7 - lane
    x |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, true);   // 15 - lane
    const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = a[0] | a[1];
    const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return b[0] | b[1];
}
__device__ __forceinline__ uint64_t wave_or64(uint64_t x) {
    return (uint64_t)wave_or((uint32_t)(x >> 32)) << 32 | wave_or((uint32_t)x);
}

// The `keep` highest of a query block's keys, by one wave: the largest
// threshold that at least `keep` keys reach, bit by bit below the first bit in
// which the highest and the lowest key differ (one ballot per 64 keys and bit,
// on the keys' upper words while the bit is one of theirs: a 64-bit compare
// takes four times as long; it ends early when exactly `keep` reach it), then
// the numbers of the keys above it in ascending order, equal ones from the
// lowest number up to the count.  NL: a lane's keys in registers (nk <= 64 NL),
// or 0: in LDS.
template <int NL>
__device__ __forceinline__ void choose(const uint64_t *kr, int nk, int valid, int keep, int lane,
                                       int32_t *out) {
    uint64_t x[NL ? NL : 1];
    if (NL)
#pragma unroll
        for (int i = 0; i < NL; ++i) x[i] = 64 * i + lane < nk ? kr[64 * i + lane] : 0;
    // f(the lane's key i, its chunk of 64) over all chunks, by all lanes; past nk: key 0
    auto each = [&](auto f) {
        if (NL) {
#pragma unroll
            for (int i = 0; i < NL; ++i) f(x[i], i);
        } else {
            for (int i = 0; 64 * i < nk; ++i) f(64 * i + lane < nk ? kr[64 * i + lane] : 0ull, i);
        }
    };
    uint64_t at = 1;                                         // keys >= at are taken,
    int ties = 0x7FFFFFFF;                                   // `ties` of those equal to it at most
    if (valid > keep) {
        uint64_t any = 0, none = 0;                          // bits set / clear in some valid key
        each([&](uint64_t y, int) {
            any |= y;
            none |= y ? ~y : 0;
        });
        any = wave_or64(any);
        const uint64_t all = ~wave_or64(none);
        const uint64_t differ = any & ~all;
        int bit = differ ? 63 - __builtin_clzll(differ) : -1;
        at = bit < 0 ? all : bit == 63 ? 0 : all & ~((2ull << bit) - 1);
        bool exact = false;
        for (; bit >= 32 && !exact; --bit) {
            const uint32_t t = (uint32_t)(at >> 32) | 1u << (bit - 32);
            int n = 0;
            each([&](uint64_t y, int) { n += __popcll(__ballot((uint32_t)(y >> 32) >= t)); });
            if (n >= keep) at = (uint64_t)t << 32;
            exact = n == keep;
        }
        for (; bit >= 0 && !exact; --bit) {
            const uint64_t t = at | 1ull << bit;
            int n = 0;
            each([&](uint64_t y, int) { n += __popcll(__ballot(y >= t)); });
            if (n >= keep) at = t;
            exact = n == keep;
        }
        if (!exact) {
            int above = 0;
            each([&](uint64_t y, int) { above += __popcll(__ballot(y > at)); });
            ties = keep - above;
        }
    }
    int n = 0;
    const uint64_t below = (1ull << lane) - 1;
    each([&](uint64_t y, int i) {
        const uint64_t equal = __ballot(y == at);
        const bool take = y > at || (y == at && __popcll(equal & below) < ties);
        const uint64_t taken = __ballot(take);
        const int pos = n + __popcll(taken & below);
        if (take && pos < keep) out[pos] = 64 * i + lane;
        n += __popcll(taken);
        ties -= __popcll(equal) < ties ? __popcll(equal) : ties;
    });
    for (int p = n + lane; p < keep; p += 64) out[p] = -1;
}

// One workgroup of eight waves per R <= 16 query blocks of a head.  Scores: 16
// query blocks x 16 key blocks a tile on the 64-bit matrix instruction
// (v_mfma_f64_16x16x4_f64: lane l supplies row / column l % 16, k = l / 16;
// result element i is row 4 i + l / 16, column l % 16), the query means in
// registers throughout, tiles of key blocks shared among the waves; the order
// of k is free, so a lane takes two neighbouring columns in one 16-byte load.
// The keys go to LDS, where a wave then chooses for each of its query blocks.
// 12 heads of 256 x 512 blocks: 26 us, of which the choice takes 10 (about 18
// bits, eight ballots each), the products 5 and their loads 5; 48 heads of 36 x
// 72 blocks: 9.8 us.
template <int D>
__global__ void __launch_bounds__(64 * kChooseWaves)
block_choose_kernel(const f64x2 *__restrict__ qm, const f64x2 *__restrict__ km,
                    const int32_t *__restrict__ kv_len, AttnShape a, int R,
                    int32_t *__restrict__ blocks) {
    extern __shared__ uint64_t keys[];                       // [R][nk]
    constexpr int STEPS = D / 8;                             // pairs of 16x16x4 products
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t per = (a.nq + R - 1) / R;
    const int64_t id = xcd_range(blockIdx.x, a.planes_q * per);   // a head's means in few L2s
    const int64_t plane = id / per;
    const int64_t i0 = (id - plane * per) * R;
    const int64_t b = plane / a.H, h = plane - b * a.H;
    const int64_t kplane = b * a.G + h / (a.H / a.G);
    const int nk = (int)a.nk;
    const int valid = (int)((valid_keys(kv_len, b, a.seq_k) + kKB - 1) / kKB);
    const int c = lane & 15, g = lane >> 4;
    // Blocks past the end, or without a valid key, have no mean: what is read in
    // their place is what the workspace held, and is used for no key.  (The loads
    // do not wait for the length.)
    const f64x2 *kp = km + kplane * mean_tiles(a.nk) * (8 * D) + lane;
    f64x2 qf[STEPS], kf[STEPS];
    auto load_k = [&](int j0) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) kf[s] = kp[(int64_t)(j0 >> 4) * (8 * D) + 64 * s];
    };
    if (16 * wave < nk) load_k(16 * wave);
    {
        const int64_t i = i0 + (c < R ? c : R - 1);
        const f64x2 *p = qm + plane * mean_tiles(a.nq) * (8 * D) +
                         mean_at<D>(i < a.nq ? i : a.nq - 1, g);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) qf[s] = p[64 * s];
    }
    for (int j0 = 16 * wave; j0 < nk; j0 += 16 * kChooseWaves) {
        const int j = j0 + c;
        f64x4 acc = {}, odd = {};                            // two chains of products
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64(qf[s].x, kf[s].x, acc, 0, 0, 0);
            odd = __builtin_amdgcn_mfma_f64_16x16x4f64(qf[s].y, kf[s].y, odd, 0, 0, 0);
        }
        acc += odd;
        if (j0 + 16 * kChooseWaves < nk) load_k(j0 + 16 * kChooseWaves);
        if (j < nk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * i + g < R)
                    keys[(4 * i + g) * nk + j] =
                        j >= valid ? 0ull : j < a.first ? ~0ull : order_key(acc[i]);
    }
    __syncthreads();
    for (int r = wave; r < R; r += kChooseWaves) {
        if (i0 + r >= a.nq) break;
        const uint64_t *kr = keys + r * nk;
        int32_t *out = blocks + (plane * a.nq + i0 + r) * a.keep;
        if (nk <= 128) choose<2>(kr, nk, valid, a.keep, lane, out);
        else if (nk <= 512) choose<8>(kr, nk, valid, a.keep, lane, out);
        else choose<0>(kr, nk, valid, a.keep, lane, out);
    }
}

// The same choice from stored scores: one workgroup per head (few_queries).  32
// heads of 313 blocks: 5.8 us, about 3 of them the launch and the loads.
__global__ void __launch_bounds__(256)
block_choose_few_kernel(const uint64_t *__restrict__ scores, const int32_t *__restrict__ kv_len,
                        AttnShape a, int32_t *__restrict__ blocks) {
    extern __shared__ uint64_t keys[];                       // [nk]
    const int64_t plane = blockIdx.x;
    const int nk = (int)a.nk;
    const int valid = (int)((valid_keys(kv_len, plane / a.H, a.seq_k) + kKB - 1) / kKB);
    for (int j = threadIdx.x; j < nk; j += 256) {
        const uint64_t x = scores[plane * nk + j];
        keys[j] = j >= valid ? 0ull : j < a.first ? ~0ull : x;
    }
    __syncthreads();
    if (threadIdx.x >= 64) return;
    int32_t *out = blocks + plane * a.keep;
    if (nk <= 128) choose<2>(keys, nk, valid, a.keep, threadIdx.x, out);
    else if (nk <= 512) choose<8>(keys, nk, valid, a.keep, threadIdx.x, out);
    else choose<0>(keys, nk, valid, a.keep, threadIdx.x, out);
}

// Lists of every block with a valid key (AttnShape::every): nothing to score.
__global__ void __launch_bounds__(256)
every_block_kernel(const int32_t *__restrict__ kv_len, AttnShape a, int64_t entries,
                   int32_t *__restrict__ blocks) {
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < entries; at += (int64_t)gridDim.x * 256) {
        const int64_t list = at / a.keep;
        const int p = (int)(at - list * a.keep);
        const int64_t valid = (valid_keys(kv_len, list / (a.H * a.nq), a.seq_k) + kKB - 1) / kKB;
        blocks[at] = p < valid ? p : -1;
    }
}

namespace {

// 64-bit means of a side, its blocks in tiles of 16.
size_t means_bytes(int64_t planes, int64_t blocks, int D) {
    return align256((size_t)planes * (size_t)mean_tiles(blocks) * 16 * D * 8);
}

// Query blocks per workgroup: their keys fit 64 KB of LDS (two workgroups per
// compute unit; 128 KB for the longest sequences).  The matrix instruction
// takes 16 rows whatever R is, so 8 of them cost twice the products: 34 us instead
// of 24 for 12 heads of 256 x 512 blocks.  But a wave then chooses for one query
// block instead of two, and where there is a compute unit for every workgroup that
// counts: means and choice of 8 heads of 235 x 469 blocks 43 us instead of 48, of 48
// heads of 36 x 72 30.7 instead of 32.7.  (256: the whole card's; a partition with
// fewer would choose 16 rows earlier, with the same lists.)
int choose_rows(const AttnShape &a) {
    int R = a.nk <= 512 ? 16 : a.nk <= 1024 ? 8 : 4;
    if (R == 16 && a.planes_q * ((a.nq + 7) / 8) <= 256) R = 8;
    return (int)(R < a.nq ? R : a.nq);
}

template <int D>
hipError_t launch(const uint16_t *q, const uint16_t *k, const int32_t *kv_len, const AttnShape &a,
                  int32_t *blocks, void *ws, hipStream_t stream) {
    if (a.every()) {
        const int64_t entries = a.planes_q * a.nq * a.keep;
        const int64_t wgs = (entries + 255) / 256;
        every_block_kernel<<<(unsigned)(wgs < 2048 ? wgs : 2048), 256, 0, stream>>>(kv_len, a, entries,
                                                                                    blocks);
        return hipGetLastError();
    }
    if (few_queries(a)) {
        uint64_t *scores = static_cast<uint64_t *>(ws);
        block_means_kernel<D, true><<<(unsigned)(a.planes_k * a.nk), 256, 0, stream>>>(
            q, k, kv_len, a, nullptr, nullptr, scores);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        block_choose_few_kernel<<<(unsigned)a.planes_q, 256, (size_t)a.nk * 8, stream>>>(
            scores, kv_len, a, blocks);
        return hipGetLastError();
    }
    f64x2 *qm = static_cast<f64x2 *>(ws);
    f64x2 *km = reinterpret_cast<f64x2 *>(static_cast<char *>(ws) + means_bytes(a.planes_q, a.nq, D));
    block_means_kernel<D, false><<<(unsigned)(a.planes_q * a.nq + a.planes_k * a.nk), 256, 0, stream>>>(
        q, k, kv_len, a, qm, km, nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int R = choose_rows(a);
    const unsigned grid = (unsigned)(a.planes_q * ((a.nq + R - 1) / R));
    block_choose_kernel<D><<<grid, 64 * kChooseWaves, (size_t)R * a.nk * 8, stream>>>(
        qm, km, kv_len, a, R, blocks);
    return hipGetLastError();
}

}  // namespace

size_t select_workspace(const AttnShape &a) {
    if (a.every()) return 0;
    if (few_queries(a)) return align256((size_t)a.planes_q * (size_t)a.nk * 8);
    return means_bytes(a.planes_q, a.nq, a.D) + means_bytes(a.planes_k, a.nk, a.D);
}

hipError_t launch_select_blocks(const uint16_t *q, const uint16_t *k, const int32_t *kv_len,
                                const AttnShape &a, int32_t *blocks, void *ws, hipStream_t stream) {
    return a.D == 64 ? launch<64>(q, k, kv_len, a, blocks, ws, stream)
                     : launch<128>(q, k, kv_len, a, blocks, ws, stream);
}

}  // namespace svdq
