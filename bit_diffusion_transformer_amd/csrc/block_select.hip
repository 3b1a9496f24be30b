// block_select.hip -- which key blocks each query block attends to: block means
// of Q and K, their products, and the `keep` highest of them.
//
// Means and scores are taken in 64 bits: a list is a discrete choice, and two
// scores that differ by less than the rounding of fp32 sums would choose
// another block there than by the definition.  The work in 64 bits is small
// (one product of D per pair of blocks, 1/8192 of the pairs of rows).
#include "attention_internal.h"
#include "svdq_device.h"

namespace svdq {

constexpr int kQB = SVDQ_QUERY_BLOCK, kKB = SVDQ_KEY_BLOCK;

__device__ __forceinline__ int64_t valid_keys(const int32_t *kv_len, int64_t b, int64_t seq_k) {
    if (!kv_len) return seq_k;
    const int64_t n = kv_len[b];
    return n < 0 ? 0 : n > seq_k ? seq_k : n;
}

// Means over blocks of rows.  One workgroup per block of one head: 16-byte
// loads, 16 (D = 128) or 32 (D = 64) rows at a time, 64-bit sums of eight
// columns a thread, then a sum over the rows through LDS.  Bound by reading Q
// and K once.
template <int D>
__global__ void __launch_bounds__(256)
block_means_kernel(const uint16_t *__restrict__ q, const uint16_t *__restrict__ k,
                   const int32_t *__restrict__ kv_len, AttnShape a, double *__restrict__ qm,
                   double *__restrict__ km) {
    constexpr int LANES = D / 8, ROWS = 256 / LANES;
    __shared__ double part[ROWS / 2][D];
    const bool query = blockIdx.x < a.planes_q * a.nq;       // uniform
    const int64_t id = query ? blockIdx.x : blockIdx.x - a.planes_q * a.nq;
    const int64_t nb = query ? a.nq : a.nk, size = query ? kQB : kKB;
    const int64_t plane = id / nb, blk = id - plane * nb;
    const int64_t seq = query ? a.seq_q : a.seq_k;
    const int64_t have = query ? a.seq_q : valid_keys(kv_len, plane / a.G, a.seq_k);
    const int64_t left = have - blk * size;
    const int rows = (int)(left < size ? left : size);
    if (rows <= 0) return;                                   // a key block without a valid key
    const uint16_t *src = (query ? q : k) + (plane * seq + blk * size) * D;
    const int r0 = threadIdx.x / LANES, c = threadIdx.x % LANES;
    double s[8] = {};
    for (int r = r0; r < rows; r += ROWS) {
        const u32x4 x = *reinterpret_cast<const u32x4 *>(src + r * D + 8 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[2 * i] += (double)bf16_lo(x[i]);
            s[2 * i + 1] += (double)bf16_hi(x[i]);
        }
    }
    for (int half = ROWS / 2; half >= 1; half >>= 1) {
        if (r0 >= half && r0 < 2 * half)
#pragma unroll
            for (int i = 0; i < 8; ++i) part[r0 - half][8 * c + i] = s[i];
        __syncthreads();
        if (r0 < half)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += part[r0][8 * c + i];
        __syncthreads();
    }
    if (r0 == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) (query ? qm : km)[id * D + 8 * c + i] = s[i] / rows;
    }
}

// A score as an unsigned key in the same order (-0 as +0), at least 1; a NaN
// counts as the lowest.  Key 0: a block that must not be taken.
__device__ __forceinline__ uint64_t order_key(double x) {
    x += 0.0;
    if (x != x) return 1;
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint64_t o = u >> 63 ? ~u : u | 0x8000000000000000ull;
    return o ? o : 1;
}

typedef double f64x2 __attribute__((ext_vector_type(2)));
typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kChooseWaves = 8;

// How many of a lane's NL keys (in registers; NL == 0: n keys in LDS) reach t,
// summed over the wave.
template <int NL>
__device__ __forceinline__ int count_from(const uint64_t (&x)[NL ? NL : 1], const uint64_t *kr,
                                          int nk, int lane, uint64_t t) {
    int n = 0;
    if (NL) {
#pragma unroll
        for (int i = 0; i < NL; ++i) n += __popcll(__ballot(x[i] >= t));
    } else {
        for (int j = lane; j < nk + lane; j += 64)          // all lanes take part
            n += __popcll(__ballot(j < nk && kr[j < nk ? j : 0] >= t));
    }
    return n;
}

// The `keep` highest of a query block's keys, by one wave: the largest
// threshold that at least `keep` keys reach, bit by bit below the first bit in
// which the highest and the lowest key differ (one ballot per 64 keys and bit;
// it ends early when exactly `keep` reach it), then the numbers of the keys
// above it in ascending order, equal ones from the lowest number up to the
// count.
template <int NL>
__device__ __forceinline__ void choose(const uint64_t *kr, int nk, int valid, int keep, int lane,
                                       int32_t *out) {
    uint64_t x[NL ? NL : 1];
    if (NL)
#pragma unroll
        for (int i = 0; i < NL; ++i) x[i] = 64 * i + lane < nk ? kr[64 * i + lane] : 0;
    uint64_t at = 1;                                         // keys >= at are taken,
    int ties = 0x7FFFFFFF;                                   // `ties` of those equal to it at most
    if (valid > keep) {
        uint64_t any = 0, all = ~0ull;                       // bits set in some / in every valid key
        for (int j = lane; j < valid; j += 64) {
            any |= kr[j];
            all &= kr[j];
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            any |= __shfl_xor(any, d);
            all &= __shfl_xor(all, d);
        }
        const uint64_t differ = any & ~all;
        const int top = differ ? 63 - __builtin_clzll(differ) : -1;
        at = top == 63 ? 0 : all & ~((2ull << (top < 0 ? 0 : top)) - 1);
        if (top < 0) at = all;                               // all equal
        bool exact = false;
        for (int bit = top; bit >= 0 && !exact; --bit) {
            const uint64_t t = at | 1ull << bit;
            const int n = count_from<NL>(x, kr, nk, lane, t);
            if (n >= keep) at = t;
            exact = n == keep;
        }
        if (!exact) ties = at == ~0ull ? keep : keep - count_from<NL>(x, kr, nk, lane, at + 1);
    }
    int n = 0;
    const uint64_t below = (1ull << lane) - 1;
    for (int j = lane; j < nk + lane; j += 64) {
        const uint64_t y = j < nk ? kr[j] : 0;
        const uint64_t equal = __ballot(y == at);
        const bool take = y > at || (y == at && __popcll(equal & below) < ties);
        const uint64_t taken = __ballot(take);
        const int pos = n + __popcll(taken & below);
        if (take && pos < keep) out[pos] = j;
        n += __popcll(taken);
        ties -= __popcll(equal) < ties ? __popcll(equal) : ties;
    }
    for (int p = n + lane; p < keep; p += 64) out[p] = -1;
}

// One workgroup of eight waves per R <= 16 query blocks of a head.  Scores: 16
// query blocks x 16 key blocks a tile on the 64-bit matrix instruction
// (v_mfma_f64_16x16x4_f64: lane l supplies row / column l % 16, k = l / 16;
// result element i is row 4 i + l / 16, column l % 16), the query means in
// registers throughout, tiles of key blocks shared among the waves; the order
// of k is free, so a lane takes two neighbouring columns in one 16-byte load.
// The keys go to LDS, where a wave then chooses for each of its query blocks.
template <int D>
__global__ void __launch_bounds__(64 * kChooseWaves)
block_choose_kernel(const double *__restrict__ qm, const double *__restrict__ km,
                    const int32_t *__restrict__ kv_len, AttnShape a, int R,
                    int32_t *__restrict__ blocks) {
    extern __shared__ uint64_t keys[];                       // [R][nk]
    constexpr int STEPS = D / 8;                             // pairs of 16x16x4 products
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t per = (a.nq + R - 1) / R;
    const int64_t plane = blockIdx.x / per;
    const int64_t i0 = (blockIdx.x - plane * per) * R;
    const int64_t b = plane / a.H, h = plane - b * a.H;
    const int64_t kplane = b * a.G + h / (a.H / a.G);
    const int nk = (int)a.nk;
    const int valid = (int)((valid_keys(kv_len, b, a.seq_k) + kKB - 1) / kKB);
    const int c = lane & 15, g = lane >> 4;
    f64x2 qf[STEPS];
    {
        int64_t i = i0 + (c < R ? c : R - 1);
        if (i >= a.nq) i = a.nq - 1;
        const double *p = qm + (plane * a.nq + i) * D + 2 * g;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) qf[s] = *reinterpret_cast<const f64x2 *>(p + 8 * s);
    }
    for (int j0 = 16 * wave; j0 < nk; j0 += 16 * kChooseWaves) {
        const int j = j0 + c;
        f64x4 acc = {};
        if (j0 < valid) {                                    // uniform
            // blocks without a valid key have no mean: read another, never used
            const double *p = km + (kplane * nk + (j < valid ? j : valid - 1)) * D + 2 * g;
            f64x2 kf[STEPS];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) kf[s] = *reinterpret_cast<const f64x2 *>(p + 8 * s);
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(qf[s].x, kf[s].x, acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(qf[s].y, kf[s].y, acc, 0, 0, 0);
            }
        }
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

namespace {

// Query blocks per workgroup: their keys fit 64 KB of LDS (two workgroups per
// compute unit), or 128 KB for the longest sequences.
int choose_rows(int64_t nk) { return nk <= 512 ? 16 : nk <= 1024 ? 8 : 4; }

template <int D>
hipError_t launch(const uint16_t *q, const uint16_t *k, const int32_t *kv_len, const AttnShape &a,
                  int32_t *blocks, void *ws, hipStream_t stream) {
    double *qm = static_cast<double *>(ws);
    double *km = reinterpret_cast<double *>(static_cast<char *>(ws) +
                                            align256((size_t)a.planes_q * a.nq * D * 8));
    block_means_kernel<D><<<(unsigned)(a.planes_q * a.nq + a.planes_k * a.nk), 256, 0, stream>>>(
        q, k, kv_len, a, qm, km);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int R = (int)(choose_rows(a.nk) < a.nq ? choose_rows(a.nk) : a.nq);
    const unsigned grid = (unsigned)(a.planes_q * ((a.nq + R - 1) / R));
    block_choose_kernel<D><<<grid, 64 * kChooseWaves, (size_t)R * a.nk * 8, stream>>>(
        qm, km, kv_len, a, R, blocks);
    return hipGetLastError();
}

}  // namespace

size_t select_workspace(const AttnShape &a) {
    return align256((size_t)a.planes_q * a.nq * a.D * 8) +
           align256((size_t)a.planes_k * a.nk * a.D * 8);
}

hipError_t launch_select_blocks(const uint16_t *q, const uint16_t *k, const int32_t *kv_len,
                                const AttnShape &a, int32_t *blocks, void *ws, hipStream_t stream) {
    return a.D == 64 ? launch<64>(q, k, kv_len, a, blocks, ws, stream)
                     : launch<128>(q, k, kv_len, a, blocks, ws, stream);
}

}  // namespace svdq
