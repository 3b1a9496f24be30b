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
    const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1];
    if (a.kv_len) {
        s.k0 = 0;
        s.nk = clamp_int(a.kv_len[b], 0, (int)a.Tk);
    } else {
        const int k0 = a.k_starts[b], k1 = a.k_starts[b + 1];
        s.k0 = clamp_int(k0, 0, (int)a.Tk);
        s.nk = clamp_int(k1, s.k0, (int)a.Tk) - s.k0;
    }
    s.q0 = clamp_int(q0, 0, (int)a.T);
    s.nq = clamp_int(q1, s.q0, (int)a.T) - s.q0;
    return s;
}

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)((uint64_t)(uint32_t)uniform((int)x) | (uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32);
}

// floor(x / y), 0 <= x < 2^52, 0 < y < 2^52: a 64-bit division takes several times as
// long.  (Both are exact in 64-bit floating point; the quotient may round up to the next
// whole number.)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    const int64_t q = (int64_t)((double)x / (double)y);
    return uniform(q * y > x ? q - 1 : q);
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
    // The tile that holds position x of the sequence's part of the line: the root of
    // before(t) = x, to the whole number below, and mended.
    __device__ static __forceinline__ int64_t tile_at(const SpanArgs &a, int64_t c0, int64_t count, int64_t x) {
        int64_t t;
        if (a.causal) {
            const double h = (double)c0 - 0.5 * R;
            t = uniform((int64_t)((sqrt(h * h + 2.0 * R * (double)x) - h) * (1.0 / R)));
        } else {
            t = quotient(x, c0);
        }
        t = t < 0 ? 0 : t < count ? t : count - 1;
        while (t > 0 && before(a, c0, t) > x) --t;
        while (t + 1 < count && before(a, c0, t + 1) <= x) ++t;
        return t;
    }
    // Blocks of keys that tile t needs.
    __device__ static __forceinline__ int blocks(const SpanArgs &a, const Seq &s, int64_t t) {
        int keys = s.nk;
        if (a.causal) {
            const int64_t all = (int64_t)s.nq * a.group, row = (t + 1) * R < all ? (t + 1) * R : all;
            const int64_t n = (int64_t)s.nk - s.nq + quotient(row - 1, a.group) + 1;
            keys = n < 0 ? 0 : n < keys ? (int)n : keys;
        }
        return (keys + kKeys - 1) / kKeys;
    }
};

// A place on the line: a tile (all values uniform over the wave).  `seqs` (LDS) holds the
// 64 sequences from `chunk` on; every wave writes and reads the same there.
template <int R>
struct Place {
    Seq *seqs;
    Seq s;
    int64_t head;                  // length of the line of one key head
    int64_t t, begin, end;         // tile of the sequence; its part of the line
    int64_t c0, count;             // of the sequence: first tile's length, tiles
    int b, g, nb, chunk;

    // The 64 sequences from b0 on: to LDS; -> this lane's part of the line.
    __device__ int64_t load_chunk(const SpanArgs &a, int b0) {
        const int lane = threadIdx.x & 63;
        chunk = b0;
        Seq v = {0, 0, 0, 0};
        if (b0 + lane < a.B) v = load_seq(a, b0 + lane);
        seqs[lane] = v;
        return Line<R>::length(a, v);
    }
    __device__ static int64_t scan(int64_t x) {    // inclusive sums over the lanes
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t o = __shfl_up(x, d);
            if (lane >= d) x += o;
        }
        return x;
    }

    // The whole line's length, and where x0 and x1 of it are: this tile becomes x0's, both are
    // moved by snap.  cut(total, x0, x1) gives them (false: nothing to do).
    template <class Cut>
    __device__ bool open(const SpanArgs &a, Seq *lds, int64_t &x0, int64_t &x1, Cut cut) {
        seqs = lds;
        int64_t sum = scan(load_chunk(a, 0));
        head = uniform(__shfl(sum, 63));
        for (int b0 = 64; b0 < a.B; b0 += 64) {
            sum = scan(load_chunk(a, b0));
            head += uniform(__shfl(sum, 63));
        }
        if (head <= 0 || !cut(head * a.G, x0, x1)) return false;
        const bool last = x1 >= head * a.G;
        // x1 first: this object ends as x0's
        if (!last) {
            find(a, sum, x1);
            x1 = snap(x1);
        }
        find(a, sum, x0);
        if (x0 > 0) x0 = snap(x0);
        return x0 < x1 && (x0 < end || next(a));
    }
    // The tile that holds position x; sum: the first chunk's, where there is only one.
    __device__ void find(const SpanArgs &a, int64_t sum, int64_t x) {
        g = (int)quotient(x, head);
        int64_t base = g * head;
        b = a.B - 1;
        for (int b0 = 0;; b0 += 64) {
            if (a.B > 64) sum = scan(load_chunk(a, b0));
            const uint64_t past = __ballot(base + sum > x);
            if (past) {
                const int l = __builtin_ctzll(past);
                b = b0 + l;
                if (l > 0) base += uniform(__shfl(sum, l - 1));
                break;
            }
            if (b0 + 64 >= a.B) break;
            base += uniform(__shfl(sum, 63));
        }
        load(a);
        t = count > 0 ? Line<R>::tile_at(a, c0, count, x - base) : 0;
        begin = base + Line<R>::before(a, c0, t);
        end = begin + Line<R>::cost(a, c0, t);
        nb = Line<R>::blocks(a, s, t);
    }
    __device__ void load(const SpanArgs &a) {
        const Seq v = seqs[b - chunk];
        s.q0 = uniform(v.q0);
        s.nq = uniform(v.nq);
        s.k0 = uniform(v.k0);
        s.nk = uniform(v.nk);
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
            if (b < chunk || b >= chunk + 64) load_chunk(a, b & ~63);
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
        if (x <= begin || x >= end) return x <= begin ? 0 : nb;
        const int i = uniform((int)((double)(x - begin) * nb / (double)(end - begin)));
        return i < nb ? i : nb;
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
        const int64_t n = quotient(total, least);
        workers = n < 1 ? 1 : n < most ? (int)n : most;
        each = quotient(total, workers);
        more = total - each * workers;
    }
    __device__ int64_t at(int64_t w) const { return w * each + (w < more ? w : more); }
};

// A worker's piece of the line: its first tile, and where the piece ends.
template <int R>
struct Piece {
    Place<R> at;
    int64_t x0, x1;
    int64_t each, more;            // of the cuts
    int w;
    __device__ bool open(const SpanArgs &a, Seq *lds, int worker, int most) {
        w = worker;
        return at.open(a, lds, x0, x1, [&](int64_t total, int64_t &from, int64_t &to) {
            const Cuts c(total, (int64_t)kLeast * kKeys * a.group, most);
            each = c.each;
            more = c.more;
            if (w >= c.workers) return false;
            from = c.at(w);
            to = c.at(w + 1);
            return true;
        });
    }
    __device__ bool begins() const { return x0 <= at.begin; }    // the tile begins in this piece
    __device__ bool whole() const { return begins() && x1 >= at.end; }
    // The workers that share the tile that begins here and ends outside: to the last whose cut
    // stays inside it.
    __device__ int parts() const {
        const int64_t y = more * (each + 1), x = at.end - 1;
        int64_t z = x < y ? quotient(x, each + 1) : more + quotient(x - y, each);
        while (z > w + 1 && at.snap(z * each + (z < more ? z : more)) >= at.end) --z;
        return (int)(z - w) + 1;
    }
    __device__ bool next(const SpanArgs &a) { return x1 > at.end && at.next(a); }
};

// A tile whose keys are shared: by the worker that has the tile's begin.
struct Shared {
    int32_t parts;                 // workers; 0: no such tile
    int32_t q0, g, rows;           // first row of the sequence, key head, rows of the tile
    int64_t row0;                  // first row of the tile in its sequence
    int64_t pad;
};

// The workspace: shared tiles' headers (one a worker), then partial results of R
// rows, unnormalized sums and (maximum, sum) of the weights: two slots a worker,
// 2 w + 1 for the tile that begins in its piece and ends outside, 2 w for the one
// that began before.
template <int D, int R>
struct Workspace {
    Shared *shared;
    float *part, *stat;
    static size_t head(int workers) { return align256((size_t)workers * sizeof(Shared)); }
    static size_t bytes(int workers) { return head(workers) + (size_t)workers * 2 * R * (D + 2) * 4; }
    Workspace(void *ws, int workers)
        : shared(static_cast<Shared *>(ws)), part(reinterpret_cast<float *>(static_cast<char *>(ws) + head(workers))),
          stat(part + (size_t)workers * 2 * R * D) {}
};

// Can any tile be shared, with the most keys that the shape allows?
inline bool may_share(const SpanArgs &a) { return a.Tk > (2 * kLeast - 1) * kKeys; }

// `most` workers, or fewer where the most keys that the shape allows make fewer pieces.
// (`most` follows from the whole card's 256 compute units, not the current device's: the
// workspace's size has to be the same wherever it is asked for.)
template <int R>
int span_workers(const SpanArgs &a, int most) {
    const double tiles = (double)(a.T * a.group / R + (a.B < a.T ? a.B : a.T));
    const double blocks = (double)((a.Tk + kKeys - 1) / kKeys + kTileCost / kKeys);
    const double pieces = tiles * a.G * blocks / kLeast + 1;
    return pieces < most ? (int)pieces : most;
}

// The parts of one row and four columns: the largest maximum, weights 2^(m_i - m) on
// sums and results.
struct Joined {
    float m, l;
    f32x4 o;
    __device__ static Joined none() { return Joined{-__builtin_inff(), 0.0f, f32x4{}}; }
    __device__ __forceinline__ void add(float m2, float l2, f32x4 o2, float scale_log2) {
        const float m1 = fmaxf(m, m2);
        // No maximum yet: parts without a key, whose sums are zero, or the NaN sums of a
        // query that is not finite, which have to stay.
        const bool none = m1 == -__builtin_inff();
        const float f = none ? 1.0f : __builtin_amdgcn_exp2f((m - m1) * scale_log2);
        const float e = none ? 1.0f : __builtin_amdgcn_exp2f((m2 - m1) * scale_log2);
        m = m1;
        l = l * f + l2 * e;
        o = o * f + o2 * e;
    }
};

template <int D>
__device__ __forceinline__ void store_joined(const SpanArgs &a, const Shared &sh, int r, int c, const Joined &j) {
    const float inv = j.l > 0.0f ? 1.0f / j.l : 0.0f;
    const int64_t row = sh.row0 + r, tok = row / a.group;
    *reinterpret_cast<u32x2 *>(a.out + ((sh.q0 + tok) * a.H + sh.g * a.group + (row - tok * a.group)) * D + 4 * c) =
        u32x2{pack_bf16x2(j.o.x * inv, j.o.y * inv), pack_bf16x2(j.o.z * inv, j.o.w * inv)};
}

}  // namespace svdq
