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
// and K once.  Query means are stored [block][D]; key means transposed,
// [D][block], so that the score kernel's lanes (one key block each) read them
// in runs.
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
        for (int i = 0; i < 8; ++i) {
            const double m = s[i] / rows;
            if (query) qm[id * D + 8 * c + i] = m;
            else km[(plane * D + 8 * c + i) * nb + blk] = m;
        }
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

// One workgroup per `R` query blocks of a head.  Scores: a thread takes key
// block j for R query blocks (or, with `spread`, each wave R / 4 of them: few
// key blocks leave threads idle otherwise), the query means uniform operands.
// The keys go to LDS.  Choice: one wave per query block finds the largest
// threshold that at least `keep` keys reach, bit by bit from the top (64
// ballots at most; it ends early when exactly `keep` keys reach it), and
// writes the numbers of the keys above it in ascending order, equal ones from
// the lowest number up to the count.
template <int D, int R, bool SPREAD>
__global__ void __launch_bounds__(256)
block_choose_kernel(const double *__restrict__ qm, const double *__restrict__ km,
                    const int32_t *__restrict__ kv_len, AttnShape a, int32_t *__restrict__ blocks) {
    extern __shared__ uint64_t keys[];                       // [R][nk]
    constexpr int RT = SPREAD ? R / 4 : R;                   // query blocks per thread
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t per = (a.nq + R - 1) / R;
    const int64_t plane = blockIdx.x / per;
    const int64_t i0 = (blockIdx.x - plane * per) * R;
    const int64_t b = plane / a.H, h = plane - b * a.H;
    const int64_t kplane = b * a.G + h / (a.H / a.G);
    const int64_t len = valid_keys(kv_len, b, a.seq_k);
    const int nk = (int)a.nk, valid = (int)((len + kKB - 1) / kKB);
    const int rt0 = SPREAD ? wave * RT : 0;
    const double *kp = km + kplane * D * nk;
    const double *qp[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t i = i0 + rt0 + r;
        qp[r] = qm + (plane * a.nq + (i < a.nq ? i : a.nq - 1)) * D;
    }
    for (int j = SPREAD ? lane : (int)threadIdx.x; j < nk; j += SPREAD ? 64 : 256) {
        double s[RT] = {};
        if (j < valid && j >= a.first) {
#pragma unroll 8
            for (int d = 0; d < D; ++d) {
                const double x = kp[(int64_t)d * nk + j];
#pragma unroll
                for (int r = 0; r < RT; ++r) s[r] = fma(qp[r][d], x, s[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
            keys[(rt0 + r) * nk + j] = j >= valid ? 0ull : j < a.first ? ~0ull : order_key(s[r]);
    }
    __syncthreads();
    for (int r = wave; r < R; r += 4) {
        const int64_t i = i0 + r;
        if (i >= a.nq) break;
        const uint64_t *kr = keys + r * nk;
        int32_t *out = blocks + (plane * a.nq + i) * a.keep;
        uint64_t at = 1;                                     // threshold: keys >= at are taken,
        int ties = 0x7FFFFFFF;                               // of those equal to it `ties` at most
        if (valid > a.keep) {
            at = 0;
            bool exact = false;
            for (int bit = 63; bit >= 0 && !exact; --bit) {
                const uint64_t t = at | 1ull << bit;
                int n = 0;
                for (int j = lane; j < nk + lane; j += 64)   // all lanes take part
                    n += __popcll(__ballot(j < nk && kr[j < nk ? j : 0] >= t));
                if (n >= a.keep) at = t;
                exact = n == a.keep;
            }
            if (!exact) {
                int above = 0;
                for (int j = lane; j < nk + lane; j += 64)
                    above += __popcll(__ballot(j < nk && kr[j < nk ? j : 0] > at));
                ties = a.keep - above;
            }
        }
        int n = 0;
        for (int j = lane; j < nk + lane; j += 64) {
            const uint64_t x = j < nk ? kr[j] : 0;
            const uint64_t below = (1ull << lane) - 1;
            const uint64_t equal = __ballot(x == at);
            const bool take = x > at || (x == at && __popcll(equal & below) < ties);
            const uint64_t taken = __ballot(take);
            const int pos = n + __popcll(taken & below);
            if (take && pos < a.keep) out[pos] = j;
            n += __popcll(taken);
            ties -= __popcll(equal) < ties ? __popcll(equal) : ties;
        }
        for (int p = n + lane; p < a.keep; p += 64) out[p] = -1;
    }
}

namespace {

// Query blocks per workgroup: their keys fit 32 KB of LDS.
int choose_rows(int64_t nk) { return nk <= 512 ? 8 : nk <= 1024 ? 4 : nk <= 2048 ? 2 : 1; }

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
    const int R = choose_rows(a.nk);
    const unsigned grid = (unsigned)(a.planes_q * ((a.nq + R - 1) / R));
    const size_t lds = (size_t)R * a.nk * 8;
    if (R == 8 && a.nk <= 128)
        block_choose_kernel<D, 8, true><<<grid, 256, lds, stream>>>(qm, km, kv_len, a, blocks);
    else if (R == 8)
        block_choose_kernel<D, 8, false><<<grid, 256, lds, stream>>>(qm, km, kv_len, a, blocks);
    else if (R == 4)
        block_choose_kernel<D, 4, false><<<grid, 256, lds, stream>>>(qm, km, kv_len, a, blocks);
    else if (R == 2)
        block_choose_kernel<D, 2, false><<<grid, 256, lds, stream>>>(qm, km, kv_len, a, blocks);
    else
        block_choose_kernel<D, 1, false><<<grid, 256, lds, stream>>>(qm, km, kv_len, a, blocks);
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
