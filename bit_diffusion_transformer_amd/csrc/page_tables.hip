// page_tables.hip -- page tables, token starts, slots and positions of a step,
// from the requests' lengths.
//
// A launch and two chains of dependent loads: 64 requests with a token each 3.5 us, 512 requests
// with 66000 tokens and 1200 new pages 7.0 us (0.55 MB).  One workgroup that also counted what
// has no slot took 13.4 there, so the count has a workgroup of its own.
#include "paged_internal.h"
#include "svdq_device.h"

namespace svdq {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = SVDQ_MAX_REQUESTS / kThreads;   // requests, at most
constexpr int kItems = 512;                                // tokens, or pages, of a workgroup

__device__ __forceinline__ int clamp_count(int x, int most) { return x < 0 ? 0 : x < most ? x : most; }

// Inclusive sums over the workgroup's threads of two counts.
__device__ __forceinline__ void scan2(int64_t &x, int64_t &y, int64_t (*waves)[2]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t ox = __shfl_up(x, d), oy = __shfl_up(y, d);
        if (lane >= d) x += ox, y += oy;
    }
    if (lane == 63) waves[wave][0] = x, waves[wave][1] = y;
    __syncthreads();
    for (int i = 0; i < wave; ++i) x += waves[i][0], y += waves[i][1];
}

// The last request of 0 .. B - 1 that starts at or before i (start[0] = 0).
__device__ __forceinline__ int request_of(const int *start, int B, int i) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Every workgroup sums the requests' tokens and new pages itself (B values, from
// the caches), so that none waits for another.  All but the last do kItems tokens
// and kItems new pages, whose request they find by bisection in LDS; the last one
// writes what there is one of per request, and counts.  A token's page is taken
// from the table only if the page was there before this call, from free_pages
// otherwise: the entries that other workgroups write are not read.
template <int PER>
__global__ void __launch_bounds__(kThreads)
page_tables_kernel(TableArgs a) {
    __shared__ int have[PER * kThreads];            // cached tokens of each request
    __shared__ int start[PER * kThreads];           // its first token, at most T
    __shared__ int fresh[PER * kThreads];           // its first new page, at most 2^31 - 1
    __shared__ int64_t waves[kThreads / 64][2];
    __shared__ int64_t missing[kThreads / 64];
    const int page = 1 << a.page_shift, first = threadIdx.x * PER;
    const int T = (int)a.T;
    const bool last = blockIdx.x == gridDim.x - 1;
    int cached[PER], added[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        cached[i] = first + i < a.B ? a.cached[first + i] : 0;
        added[i] = first + i < a.B ? a.added[first + i] : 0;
    }
    int64_t pag[PER];                               // new pages of the thread's requests
    int64_t x = 0, y = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        cached[i] = clamp_count(cached[i], SVDQ_MAX_SLOTS);
        added[i] = clamp_count(added[i], 0x7FFFFFFF);
        // a token past the table's width has no page
        const int64_t held = ((int64_t)cached[i] + page - 1) >> a.page_shift;
        int64_t want = ((int64_t)cached[i] + added[i] + page - 1) >> a.page_shift;
        want = want < a.width ? want : a.width;
        pag[i] = want > held ? want - held : 0;
        x += added[i];
        y += pag[i];
    }
    const int64_t sum_x = x, sum_y = y;
    scan2(x, y, waves);
    const int64_t total_x = waves[0][0] + waves[1][0] + waves[2][0] + waves[3][0];
    const int64_t total_y = waves[0][1] + waves[1][1] + waves[2][1] + waves[3][1];
    int64_t at_x = x - sum_x, at_y = y - sum_y;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = first + i;
        have[b] = cached[i];
        start[b] = at_x < T ? (int)at_x : T;
        fresh[b] = at_y < 0x7FFFFFFF ? (int)at_y : 0x7FFFFFFF;
        if (last && b < a.B) {
            const int64_t kv = (int64_t)cached[i] + added[i];
            a.q_starts[b] = start[b];
            a.kv_len[b] = (int)(kv < SVDQ_MAX_SLOTS ? kv : SVDQ_MAX_SLOTS);
        }
        at_x += added[i];
        at_y += pag[i];
    }
    __syncthreads();
    const int64_t pages = total_y < 0x7FFFFFFF ? total_y : 0x7FFFFFFF;
    auto held_of = [&](int b) { return ((int64_t)have[b] + page - 1) >> a.page_shift; };

    if (!last) {
        const int64_t step = (int64_t)(gridDim.x - 1) * kItems;
        const int64_t tokens = total_x < T ? total_x : T;
        for (int64_t i0 = (int64_t)blockIdx.x * kItems; i0 < T; i0 += step)   // slots and positions
#pragma unroll
            for (int u = 0; u < kItems / kThreads; ++u) {
                const int64_t i = i0 + u * kThreads + threadIdx.x;
                if (i >= T) break;
                int slot = -1, position = -1;
                if (i < tokens) {
                    const int b = request_of(start, a.B, (int)i);
                    const int64_t p = (int64_t)have[b] + (i - start[b]);
                    const int64_t at = p >> a.page_shift, held = held_of(b);
                    position = (int)p;
                    int from = -1;
                    if (at < a.width) {
                        const int64_t j = fresh[b] + (at - held);
                        if (at < held)
                            from = a.tables[(int64_t)b * a.width + at];
                        else if (j < a.free_count)
                            from = a.free_pages[j];
                    }
                    if (from >= 0 && from < a.pages) slot = (int)(((int64_t)from << a.page_shift) + (p & (page - 1)));
                }
                a.slots[i] = slot;
                a.positions[i] = position;
            }
        for (int64_t j0 = (int64_t)blockIdx.x * kItems; j0 < pages; j0 += step)   // the new pages
#pragma unroll
            for (int u = 0; u < kItems / kThreads; ++u) {
                const int64_t j = j0 + u * kThreads + threadIdx.x;
                if (j >= pages) break;
                const int b = request_of(fresh, a.B, (int)j);
                const int64_t at = held_of(b) + (j - fresh[b]);
                if (at < a.width) a.tables[(int64_t)b * a.width + at] = j < a.free_count ? a.free_pages[j] : -1;
            }
        return;
    }

    // Tokens without a slot: of each request those past T, past the table's width and in a page
    // that was there, then those of the new pages (each has a token at least, so T pages hold
    // all that count).
    int64_t lost = 0;
    auto inside = [&](int b, int64_t n) { return start[b] + n < T ? n : T - (int64_t)start[b]; };
    auto within = [&](int64_t at, int64_t c, int64_t n) {   // of tokens c .. c + n - 1, those of page `at`
        const int64_t lo = at << a.page_shift, hi = lo + page;
        const int64_t k = (hi < c + n ? hi : c + n) - (lo > c ? lo : c);
        return k > 0 ? k : 0;
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = first + i;
        if (b >= a.B || added[i] == 0) continue;
        const int64_t c = cached[i], n = inside(b, added[i]);
        const int64_t room = (int64_t)a.width << a.page_shift, at = c >> a.page_shift;
        lost += added[i] - n;
        if (c + n > room) lost += c + n - (c > room ? c : room);
        if ((c & (page - 1)) && at < a.width) {
            const int from = a.tables[(int64_t)b * a.width + at];
            if (from < 0 || from >= a.pages) lost += within(at, c, n);
        }
    }
    const int64_t look = pages < T ? pages : T;
#pragma unroll 4
    for (int64_t j = threadIdx.x; j < look; j += kThreads) {
        const int from = j < a.free_count ? a.free_pages[j] : -1;
        if (from >= 0 && from < a.pages) continue;
        const int b = request_of(fresh, a.B, (int)j);
        lost += within(held_of(b) + (j - fresh[b]), have[b], inside(b, clamp_count(a.added[b], 0x7FFFFFFF)));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) lost += __shfl_xor(lost, d);
    if ((threadIdx.x & 63) == 0) missing[threadIdx.x >> 6] = lost;
    __syncthreads();
    if (threadIdx.x == 0) {
        const int64_t n = missing[0] + missing[1] + missing[2] + missing[3];
        a.q_starts[a.B] = total_x < T ? (int)total_x : T;
        a.counts[0] = (int)pages;
        a.counts[1] = (int)(n < 0x7FFFFFFF ? n : 0x7FFFFFFF);
    }
}

}  // namespace

hipError_t launch_page_tables(const TableArgs &a, hipStream_t stream) {
    const int64_t want = (a.T + kItems - 1) / kItems;
    const unsigned grid = 1 + (unsigned)(want < 1 ? 1 : want < 1024 ? want : 1024);
    if (a.B <= kThreads)
        page_tables_kernel<1><<<grid, kThreads, 0, stream>>>(a);
    else if (a.B <= 4 * kThreads)
        page_tables_kernel<4><<<grid, kThreads, 0, stream>>>(a);
    else
        page_tables_kernel<kPerThread><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace svdq
