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
// Positions are in keys times group, whole numbers up to 2^52 or (with narrow tiles) quarters up
// to 2^51, in 64-bit floating point (exact; a 64-bit integer product or quotient takes many times
// as long, and a short call is mostly this).  A shape that could make the line longer is
// refused, and a line longer than any ascending starts make it is not worked on, so every
// worker finds the same tiles.  Tile t of a sequence is c0 + S t long (S = R with `causal`: R
// rows are R / group tokens, so many more keys; S = 0 without).  Cuts are anywhere, but every
// worker computes them in the same way.  More than 64 sequences are measured in 64 ranges, a
// lane each, and searched in two levels: 2048 requests over 100 keys, 8 heads on 2 of 128, 47 us
// (59 in chunks of 64), 8192 213 (286).
#pragma once

#include "paged_internal.h"
#include "svdq_device.h"

namespace svdq {

constexpr int kKeys = 64;          // keys of a block
// Of tiles of R rows.  kTileCost: keys' time that a tile takes beside its keys (its queries, its
// first copies, its result).  kLeast: blocks on each side of a cut, at least.  Tiles of 128, cost
// and least 128 and 2 | 256 and 4 | 384 and 4 | 128 and 8, us: 77 tokens, 12 heads of 64 9.4 | 9.3
// | 9.4 | 19.4; 500 tokens, 24 heads 26.0 | 18.3 | 18.5 | 21.9; twelve prompts of 1 to 2000, 32
// heads 105 | 103 | 112 | 104; 40 tokens over 4000 44 | 32 | 33 | 33.
template <int R>
constexpr int kTileCost = R < 128 ? 128 : 256;
template <int R>
constexpr int kLeast = R < 128 ? 2 : 4;

// Of a narrow tile (a paged request of at most 32 rows beside wide tiles): a key's length, and
// the tile's own.  0.25 and 512 | 0.25 and 256 | 0.5 and 256 | 0.125 and 256, us: 31 requests of up
// to 6000 keys, D = 64 19.6 | 20.8 | 20.9 | 20.3, D = 128 26.9 | 31.1 | 30.7 | 29.3.
constexpr double kNarrow = 0.25;
constexpr int kNarrowCost = 512;

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
__device__ __forceinline__ double uniform(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)uniform((int)u) |
                                          (uint64_t)(uint32_t)uniform((int)(u >> 32)) << 32);
}
__device__ __forceinline__ double lane_of(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)u, lane) |
                                          (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane) << 32);
}

// Inclusive sums over the lanes: within rows of 16, then rows 1 and 3 get their
// neighbour's, then the upper half the lower's.
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, false);
    return x + __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32);
}
__device__ __forceinline__ double scan(double x) {
    x = scan_step<0x111, 0xF>(x);                  // one lane up
    x = scan_step<0x112, 0xF>(x);                  // two
    x = scan_step<0x114, 0xF>(x);
    x = scan_step<0x118, 0xF>(x);
    x = scan_step<0x142, 0xA>(x);                  // lane 15 of the row below
    return scan_step<0x143, 0xC>(x);               // lane 31
}

// The token of row x of a sequence: floor(x / group), x < 2^34.
__device__ __forceinline__ int token_of(const SpanArgs &a, double x) {
    const int q = (int)((x + 0.5) * a.inv_group);
    return uniform(q);
}
// The same for x < 2^16.
__device__ __forceinline__ int token_of(const SpanArgs &a, int x) {
    return (int)(((float)x + 0.5f) * a.inv_group_f);
}

// A place on the line: a tile (all values uniform over the wave).  `seqs` (LDS) holds the
// 64 sequences from `chunk` on, for this wave alone.
template <int R>
struct Place {
    Seq *seqs;
    Seq s;
    double head;                   // length of the line of one key head
    double begin, end;             // the tile's part of the line
    double c0;                     // length of the sequence's first tile
    int t, count;                  // tile of the sequence, its tiles
    int b, g, nb, chunk;           // sequence, key head, blocks of keys; first sequence in LDS

    __device__ static __forceinline__ double step(const SpanArgs &a) { return a.causal ? R : 0.0; }
    __device__ static __forceinline__ double tiles(const SpanArgs &a, const Seq &v) {
        return floor(((double)v.nq * a.group + (R - 1)) * (1.0 / R));
    }
    // A paged sequence of one wave's rows in a wide tile: the waves divide its keys.
    __device__ static __forceinline__ bool narrow(const SpanArgs &a, const Seq &v) {
        return R > 32 && a.kv_len && (int64_t)v.nq * a.group <= 32;
    }
    __device__ static __forceinline__ double cost0(const SpanArgs &a, const Seq &v) {
        if (narrow(a, v)) return (v.nk * kNarrow + kNarrowCost) * a.group;
        const int less = a.causal ? v.nq : 0;
        return ((double)(v.nk > less ? v.nk - less : 0) + kTileCost<R>) * a.group + step(a);
    }
    __device__ static __forceinline__ double before(const SpanArgs &a, double c, double n) {
        return c * n + step(a) * 0.5 * (n * (n - 1.0));
    }

    // The 64 sequences from b0 on: to LDS; -> the sums of their lengths up to this lane's.
    __device__ __forceinline__ double load_chunk(const SpanArgs &a, int b0) {
        const int lane = threadIdx.x & 63;
        chunk = b0;
        Seq v = {0, 0, 0, 0};
        if (b0 + lane < a.B) v = load_seq(a, b0 + lane);
        seqs[lane] = v;
        return scan(before(a, cost0(a, v), tiles(a, v)));
    }
    // The sequence b and the key head g, whose part of the line begins at `base`; the tile that
    // holds x.
    __device__ __forceinline__ void load(const SpanArgs &a) {
        const Seq v = seqs[b - chunk];
        s.q0 = uniform(v.q0);
        s.nq = uniform(v.nq);
        s.k0 = uniform(v.k0);
        s.nk = uniform(v.nk);
        count = uniform((int)tiles(a, s));
        c0 = uniform(cost0(a, s));
    }
    __device__ __forceinline__ void set_tile(const SpanArgs &a, double at) {
        begin = at;
        end = uniform(at + c0 + step(a) * t);
        int keys = s.nk;
        if (a.causal) {
            const double all = (double)s.nq * a.group, row = (double)(t + 1) * R;
            const int n = s.nk - s.nq + token_of(a, (row < all ? row : all) - 1.0) + 1;
            keys = n < 0 ? 0 : n < keys ? n : keys;
        }
        nb = (keys + kKeys - 1) / kKeys;
    }
    // The line of one key head -> its length; -> the sums up to this lane's sequence or, where
    // there are more than 64, up to the end of its range of them.
    __device__ static __forceinline__ int range_of(const SpanArgs &a) { return (a.B + 63) >> 6; }
    __device__ __forceinline__ double measure(const SpanArgs &a) {
        double sum;
        if (a.B <= 64) {
            sum = load_chunk(a, 0);
        } else {
            const int range = range_of(a), b0 = (threadIdx.x & 63) * range;
            sum = 0.0;
#pragma unroll 4
            for (int i = 0; i < range; ++i) {
                if (b0 + i >= a.B) break;
                const Seq v = load_seq(a, b0 + i);
                sum += before(a, cost0(a, v), tiles(a, v));
            }
            sum = scan(sum);
        }
        head = lane_of(sum, 63);
        return sum;
    }
    // The tile that holds position x (0 <= x < G head); sum: measure's.
    __device__ __forceinline__ void find(const SpanArgs &a, double sum, double x) {
        g = uniform((int)(x * __builtin_amdgcn_rcp(head)));
        while (g > 0 && g * head > x) --g;
        while (g + 1 < a.G && (g + 1) * head <= x) ++g;
        double base = g * head;
        b = a.B - 1;
        int b0 = 0;
        if (a.B > 64) {
            const uint64_t past = __ballot(base + sum > x);
            const int l = past ? __builtin_ctzll(past) : 63;
            if (l > 0) base += lane_of(sum, l - 1);
            b0 = l * range_of(a);
        }
        for (;; b0 += 64) {
            if (a.B > 64) sum = load_chunk(a, b0);
            const uint64_t past = __ballot(base + sum > x);
            if (past) {
                const int l = __builtin_ctzll(past);
                b = b0 + l;
                if (l > 0) base += lane_of(sum, l - 1);
                break;
            }
            if (b0 + 64 >= a.B) break;
            base += lane_of(sum, 63);
        }
        load(a);
        // the root of before(t) = x - base, from 32 bits and mended
        const float h = (float)(c0 - 0.5 * step(a)), y = (float)(x - base);
        t = uniform((int)(2.0f * y / (h + sqrtf(h * h + 2.0f * (float)step(a) * y))));
        t = t < 0 ? 0 : t < count ? t : count > 0 ? count - 1 : 0;
        while (t > 0 && base + before(a, c0, t) > x) --t;
        while (t + 1 < count && base + before(a, c0, t + 1) <= x) ++t;
        set_tile(a, uniform(base + before(a, c0, t)));
    }
    // The next tile of the line; false behind the last.
    __device__ __forceinline__ bool next(const SpanArgs &a) {
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
        set_tile(a, end);
        return true;
    }
    // The block in front of which position x cuts this tile.
    __device__ __forceinline__ int block_at(double x) const {
        if (x <= begin) return 0;
        if (x >= end) return nb;
        const int i = uniform((int)((x - begin) * nb * __builtin_amdgcn_rcp(end - begin)));
        return i < nb ? i : nb;
    }
    // x, moved to an end of the tile that has fewer than kLeast blocks on one side of it.
    __device__ __forceinline__ double snap(double x) const {
        const int i = block_at(x);
        return i < kLeast<R> ? begin : nb - i < kLeast<R> ? end : x;
    }
};

// A worker's piece of the line, tile by tile: the tile `at`, of which the piece has the
// blocks first .. last - 1.
template <int R>
struct Piece {
    Place<R> at;
    double x0, x1, total;
    int w, workers;
    int first, last;
    bool begins, whole;            // the piece has the tile's begin; all of it

    __device__ __forceinline__ double cut(int i) const { return i < workers ? total * i * __builtin_amdgcn_rcp((double)workers) : total; }

    __device__ __forceinline__ bool open(const SpanArgs &a, Seq *lds, int worker, int most) {
        w = worker;
        at.seqs = lds;
        const double sum = at.measure(a);
        total = uniform(at.head * a.G);
        if (!(total > 0.0 && total <= a.line)) return false;
        const double n = total * a.inv_group * (1.0 / (kLeast<R> * kKeys));
        workers = uniform(n < 1.0 ? 1 : n < (double)most ? (int)n : most);
        if (w >= workers) return false;
        x0 = uniform(cut(w));
        x1 = uniform(cut(w + 1));
        at.find(a, sum, x0);
        if (w > 0) x0 = at.snap(x0);
        if (x0 >= at.end && !at.next(a)) return false;
        return enter();
    }
    // This tile's part of the piece; false where the piece ends before it.
    __device__ __forceinline__ bool enter() {
        if (x1 < at.end) x1 = at.snap(x1);
        begins = x0 <= at.begin;
        whole = begins && x1 >= at.end;
        first = at.block_at(x0);
        last = at.block_at(x1);
        return x1 > at.begin;
    }
    __device__ __forceinline__ bool next(const SpanArgs &a) { return x1 > at.end && at.next(a) && enter(); }
    // The pieces that share this tile: the last that begins at or before the tile's begin, and
    // the last that begins before its end.  (A cut in another tile snaps to no further than
    // this tile's ends.)
    __device__ __forceinline__ int near(double x) const {
        const int z = uniform((int)(x * workers * __builtin_amdgcn_rcp(total)));
        return z < workers ? z : workers - 1;
    }
    __device__ __forceinline__ int first_piece() const {
        if (begins) return w;
        int z = near(at.begin);
        while (z + 1 < w && (cut(z + 1) <= at.begin || at.snap(cut(z + 1)) <= at.begin)) ++z;
        while (z > 0 && cut(z) > at.begin && at.snap(cut(z)) > at.begin) --z;
        return z;
    }
    __device__ __forceinline__ int last_piece() const {
        int z = near(at.end);
        while (z + 1 < workers && cut(z + 1) < at.end && at.snap(cut(z + 1)) < at.end) ++z;
        while (z > w && (cut(z) >= at.end || at.snap(cut(z)) >= at.end)) --z;
        return z;
    }
};

// A tile whose keys several pieces share, as one of them sees it.
struct Shared {
    int32_t parts, index;          // pieces (0: no such tile), and which this one is
    int32_t rows, q0, g, pad;      // rows of the tile, first row of its sequence, key head
    int64_t row0;                  // first row of the tile in its sequence
};

// For the tile that the piece is at, with `rows` rows from row0 on: the slot of its partial
// result (-1: the tile is this piece's alone), and the slot's header.
template <int R>
__device__ __forceinline__ int share(const Piece<R> &p, int64_t row0, int rows, Shared *__restrict__ shared) {
    if (p.whole) return -1;
    const int slot = 2 * p.w + (p.begins ? 1 : 0);
    const int first = p.first_piece(), last = p.last_piece();
    if (threadIdx.x == 0) shared[slot] = Shared{last - first + 1, p.w - first, rows, p.at.s.q0, p.at.g, 0, row0};
    return slot;
}

// The workspace: headers, then partial results of R rows, unnormalized sums and
// (maximum, sum) of the weights: two slots a piece, 2 w + 1 for the tile that
// begins in it and ends outside, 2 w for the one that began before.
template <int D, int R>
struct Workspace {
    Shared *shared;
    float *part, *stat;
    static size_t head(int pieces) { return align256((size_t)pieces * 2 * sizeof(Shared)); }
    static size_t bytes(int pieces) { return head(pieces) + (size_t)pieces * 2 * R * (D + 2) * 4; }
    Workspace(void *ws, int pieces)
        : shared(static_cast<Shared *>(ws)), part(reinterpret_cast<float *>(static_cast<char *>(ws) + head(pieces))),
          stat(part + (size_t)pieces * 2 * R * D) {}
};

// Can any tile be shared, with the most keys that the shape allows?
template <int R>
bool may_share(const SpanArgs &a) { return a.Tk > (2 * kLeast<R> - 1) * kKeys; }

// `most` workers, or fewer where the most keys that the shape allows make fewer pieces.
// (`most` follows from the whole card's 256 compute units, not the current device's: the
// workspace's size has to be the same wherever it is asked for.)
template <int R>
int span_workers(const SpanArgs &a, int most) {
    const double tiles = (double)(a.T * a.group / R + (a.B < a.T ? a.B : a.T));
    const double blocks = (double)((a.Tk + kKeys - 1) / kKeys + kTileCost<R> / kKeys);
    const double pieces = tiles * a.G * blocks / kLeast<R> + 1;
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

// Where row r of a shared tile goes.
template <int D>
__device__ __forceinline__ uint16_t *joined_row(const SpanArgs &a, const Shared &sh, int r) {
    const int64_t row = sh.row0 + r, tok = row / a.group;
    return a.out + ((sh.q0 + tok) * a.H + sh.g * a.group + (row - tok * a.group)) * D;
}

}  // namespace svdq
