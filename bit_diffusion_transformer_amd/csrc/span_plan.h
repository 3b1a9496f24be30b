// span_plan.h -- how the attention of sequences whose lengths only the device
// knows is divided among workgroups (internal; not part of the ABI).
//
// The work is a line.  Per key head, sequence after sequence: tiles of R rows
// (row r of a sequence: token r / group, head r % group of the key head's
// group), each as long as its keys are many plus a constant for its start and
// end; the key heads follow one another.  The line is cut into equal pieces, one
// a worker.  A cut inside a tile falls between two blocks of 64 keys; the tile's
// parts go to the workspace then and are joined afterwards.  So a long request
// among short ones, a single row over a long cache, and a prompt whose late
// tiles see all keys give every worker the same time, without the host knowing
// a length.
//
// Lengths along the line are in keys times group, closed form: tile t of a
// sequence is A + S t long (S = R with `causal`: R rows are R / group tokens, so
// many more keys; S = 0 without).  Every worker computes the same cuts.
#pragma once

#include "paged_internal.h"
#include "svdq_device.h"

namespace svdq {

constexpr int kKeys = 64;          // keys of a block
constexpr int kTileCost = 128;     // keys' time that a tile takes beside its keys
constexpr int kLeast = 2;          // blocks on each side of a cut, at least

struct Seq {
    int q0, nq, k0, nk;            // first row and rows of q, of k
};

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

__device__ __forceinline__ Seq load_seq(const SpanArgs &a, int b) {
    Seq s;
    s.q0 = clamp_int(a.q_starts[b], 0, (int)a.T);
    s.nq = clamp_int(a.q_starts[b + 1], s.q0, (int)a.T) - s.q0;
    if (a.kv_len) {
        s.k0 = 0;
        s.nk = clamp_int(a.kv_len[b], 0, (int)a.Tk);
    } else {
        s.k0 = clamp_int(a.k_starts[b], 0, (int)a.Tk);
        s.nk = clamp_int(a.k_starts[b + 1], s.k0, (int)a.Tk) - s.k0;
    }
    return s;
}

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)x) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32);
}

template <int R>
struct Line {
    // of one sequence
    __device__ static __forceinline__ int64_t tiles(const SpanArgs &a, const Seq &s) {
        return ((int64_t)s.nq * a.group + R - 1) / R;
    }
    __device__ static __forceinline__ int64_t cost0(const SpanArgs &a, const Seq &s) {
        const int keys = a.causal ? (s.nk > s.nq ? s.nk - s.nq : 0) : s.nk;
        return ((int64_t)keys + kTileCost) * a.group + (a.causal ? R : 0);
    }
    __device__ static __forceinline__ int64_t cost(const SpanArgs &a, int64_t c0, int64_t t) {
        return a.causal ? c0 + R * t : c0;
    }
    __device__ static __forceinline__ int64_t before(const SpanArgs &a, int64_t c0, int64_t t) {
        return c0 * t + (a.causal ? R * (t * (t - 1) / 2) : 0);
    }
    __device__ static __forceinline__ int64_t length(const SpanArgs &a, const Seq &s) {
        return before(a, cost0(a, s), tiles(a, s));
    }
    // Blocks of keys that tile t needs.
    __device__ static __forceinline__ int blocks(const SpanArgs &a, const Seq &s, int64_t t) {
        int keys = s.nk;
        if (a.causal) {
            const int64_t row = (t + 1) * R < (int64_t)s.nq * a.group ? (t + 1) * R
                                                                      : (int64_t)s.nq * a.group;
            const int64_t n = (int64_t)s.nk - s.nq + (row - 1) / a.group + 1;
            keys = n < 0 ? 0 : n < keys ? (int)n : keys;
        }
        return (int)(((int64_t)keys + kKeys - 1) / kKeys);
    }

    // The line of one key head: lane l's part of a wave sums sequences l, l + 64, ..
    __device__ static int64_t per_head(const SpanArgs &a) {
        int64_t sum = 0;
        for (int b = threadIdx.x & 63; b < a.B; b += 64) sum += length(a, load_seq(a, b));
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        return uniform(sum);
    }
};

// A tile on the line (all values uniform over the wave).
template <int R>
struct Place {
    Seq s;
    int64_t t, begin, end;         // tile of the sequence; its part of the line
    int64_t c0, count;             // of the sequence: first tile's length, tiles
    int b, g, nb;

    // The tile that holds position x (0 <= x < G per_head).
    __device__ void find(const SpanArgs &a, int64_t head, int64_t x) {
        g = (int)(x / head);
        int64_t at = (int64_t)g * head;
        const int lane = threadIdx.x & 63;
        b = a.B - 1;
        int64_t base = at;
        for (int b0 = 0; b0 < a.B; b0 += 64) {
            int64_t sum = b0 + lane < a.B ? Line<R>::length(a, load_seq(a, b0 + lane)) : 0;
            const int64_t mine = sum;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t o = __shfl_up(sum, d);
                if (lane >= d) sum += o;
            }
            const uint64_t past = __ballot(at + sum > x);
            if (past) {
                const int l = __builtin_ctzll(past);
                b = b0 + l;
                base = at + uniform(__shfl(sum - mine, l));
                break;
            }
            at += uniform(__shfl(sum, 63));
        }
        b = __builtin_amdgcn_readfirstlane(b);
        load(a);
        int64_t lo = 0, hi = count > 0 ? count - 1 : 0;   // the last tile that begins at or before x
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (base + Line<R>::before(a, c0, mid) <= x)
                lo = mid;
            else
                hi = mid - 1;
        }
        t = lo;
        begin = base + Line<R>::before(a, c0, t);
        end = begin + Line<R>::cost(a, c0, t);
        nb = Line<R>::blocks(a, s, t);
    }
    __device__ void load(const SpanArgs &a) {
        Seq v = load_seq(a, b);
        s.q0 = __builtin_amdgcn_readfirstlane(v.q0);
        s.nq = __builtin_amdgcn_readfirstlane(v.nq);
        s.k0 = __builtin_amdgcn_readfirstlane(v.k0);
        s.nk = __builtin_amdgcn_readfirstlane(v.nk);
        count = Line<R>::tiles(a, s);
        c0 = Line<R>::cost0(a, s);
    }
    // The next tile of the line; false behind the last.
    __device__ bool next(const SpanArgs &a) {
        ++t;
        while (t >= count) {
            if (++b >= a.B) {
                b = 0;
                if (++g >= a.G) return false;
            }
            load(a);
            t = 0;
        }
        begin = end;
        end = begin + Line<R>::cost(a, c0, t);
        nb = Line<R>::blocks(a, s, t);
        return true;
    }
    // The block in front of which position x cuts this tile.
    __device__ int block_at(int64_t x) const {
        return x <= begin ? 0 : x >= end ? nb : (int)((x - begin) * nb / (end - begin));
    }
    // x, moved to an end of the tile that has fewer than kLeast blocks on one side of it.
    __device__ int64_t snap(int64_t x) const {
        const int i = block_at(x);
        return i < kLeast ? begin : nb - i < kLeast ? end : x;
    }
};

// The cuts: worker w has the line from cut(w) to cut(w + 1).
struct Cuts {
    int64_t each, more;            // the first `more` workers have one more
    int workers;
    __device__ Cuts(int64_t total, int64_t least, int most) {
        const int64_t n = total / least;
        workers = n < 1 ? 1 : n < most ? (int)n : most;
        each = total / workers;
        more = total - each * workers;
    }
    __device__ int64_t at(int64_t w) const { return w * each + (w < more ? w : more); }
    // The worker that has position x.
    __device__ int64_t of(int64_t x) const {
        const int64_t y = more * (each + 1);
        return x < y ? x / (each + 1) : more + (x - y) / each;
    }
};

// A tile whose keys are shared: by the worker that has the tile's begin.
struct Shared {
    int32_t parts;                 // workers; 0: no such tile
    int32_t q0, g, rows;           // first row of the sequence, key head, rows of the tile
    int64_t row0;                  // first row of the tile in its sequence
    int64_t pad;
};

}  // namespace svdq
