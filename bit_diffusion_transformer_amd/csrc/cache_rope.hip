// cache_rope.hip -- the per-head RMS norm and rotary turn of a written projection
// [T, (H + 2 G) D], Q to rows, K and V to the slots of a paged cache.
#include "paged_internal.h"
#include "svdq_wave.h"

namespace svdq {

namespace {

constexpr int kPer = 4;                // 16-byte pieces per thread
constexpr int kStep = 256 * kPer;      // pieces per workgroup

// Bound by memory: each element is read and written once, 2 bytes each way, plus
// the token's table rows, position and slot.  A lane holds 16 bytes (8 elements)
// of one head, so a head is 8 or 16 neighbouring lanes and its sum of squares
// three or four lane exchanges.  Pairs of neighbours are in one lane; in the
// half layout the partner of a lane's piece is the piece rotary / 16 lanes
// further (or back), one lane exchange for each of its 8 values.  8000 tokens of 32 heads on 4 of
// 128, a quarter turned: 39 us, 4.2 TB/s (all turned, tables of 8000 rows: 37, in halves 40); 64
// tokens of 32 on 8 6.4 us, the launch and three dependent loads.  Four pieces a thread, all
// loaded first, keep enough in flight for that.
template <int D, bool HALF>
__global__ void __launch_bounds__(256)
cache_rope_kernel(CacheArgs a) {
    constexpr int LPH = D / 8;                              // lanes per head
    const uint32_t row = (uint32_t)(a.H + 2 * a.G) * LPH;   // pieces per token
    const int64_t id0 = (int64_t)blockIdx.x * kStep;
    const int64_t tok0 = id0 / row;                         // uniform
    const uint32_t rem0 = (uint32_t)(id0 - tok0 * row);
    const int64_t total = a.T * row;
    const int64_t room = a.pages << a.page_shift;
    const int half = a.R / 2;
    u32x4 x[kPer];
    int pos[kPer], slot[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int64_t id = id0 + j * 256 + threadIdx.x;
        x[j] = u32x4{};
        pos[j] = slot[j] = -1;
        if (id < total) {
            const int64_t tok = tok0 + (rem0 + j * 256 + threadIdx.x) / row;
            x[j] = reinterpret_cast<const u32x4 *>(a.qkv)[id];
            pos[j] = a.positions[tok];
            slot[j] = a.slots[tok];
        }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int64_t id = id0 + j * 256 + threadIdx.x;
        if (id >= total) break;                             // whole heads: `total` is a multiple of LPH
        const uint32_t r = rem0 + j * 256 + threadIdx.x;
        const uint32_t dt = r / row;
        const uint32_t piece = r - dt * row;
        const int64_t tok = tok0 + dt;
        const int head = (int)(piece / LPH), l = (int)(piece % LPH);   // head over the three sections
        const bool is_q = head < a.H, is_v = head >= a.H + a.G;
        if (pos[j] < 0 || pos[j] >= a.P) continue;          // whole heads
        if (!is_q && (slot[j] < 0 || slot[j] >= room)) continue;
        u32x4 y = x[j];
        if (!is_v) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(x[j][i]);
                v[2 * i + 1] = bf16_hi(x[j][i]);
            }
            const uint16_t *gamma = is_q ? a.gq : a.gk;
            if (gamma) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
                ss = head_sum<LPH>(ss);
                const float inv = 1.0f / sqrtf(__builtin_fmaf(ss, 1.0f / D, a.eps));
                const u32x4 g = *reinterpret_cast<const u32x4 *>(gamma + 8 * l);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] *= inv * bf16_lo(g[i]);
                    v[2 * i + 1] *= inv * bf16_hi(g[i]);
                }
            }
            const float *ct = a.cos_t + (int64_t)pos[j] * half, *st = a.sin_t + (int64_t)pos[j] * half;
            if (HALF) {
                const int hl = half / 8;                    // lanes of half the turned part
                const bool turned = l < 2 * hl, second = l >= hl;
                const int from = turned ? (second ? l - hl : l + hl) - l : 0;
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __shfl(v[i], (int)(threadIdx.x & 63) + from);
                if (turned) {
                    const int at = 8 * (second ? l - hl : l);
                    const f32x4 c0 = *reinterpret_cast<const f32x4 *>(ct + at);
                    const f32x4 c1 = *reinterpret_cast<const f32x4 *>(ct + at + 4);
                    const f32x4 n0 = *reinterpret_cast<const f32x4 *>(st + at);
                    const f32x4 n1 = *reinterpret_cast<const f32x4 *>(st + at + 4);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float c = i < 4 ? c0[i & 3] : c1[i & 3], n = i < 4 ? n0[i & 3] : n1[i & 3];
                        const float t = w[i] * n;
                        v[i] = __builtin_fmaf(v[i], c, second ? t : -t);
                    }
                }
            } else if (l < a.R / 8) {
                const f32x4 c = *reinterpret_cast<const f32x4 *>(ct + 4 * l);
                const f32x4 n = *reinterpret_cast<const f32x4 *>(st + 4 * l);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = v[2 * i], q = v[2 * i + 1];
                    v[2 * i] = __builtin_fmaf(p, c[i], -(q * n[i]));
                    v[2 * i + 1] = __builtin_fmaf(p, n[i], q * c[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        }
        uint16_t *dst;
        int64_t at;
        if (is_q) {
            dst = a.q;
            at = (tok * a.H + head) * LPH + l;
        } else {
            const int g = head - a.H - (is_v ? a.G : 0), page = 1 << a.page_shift;
            dst = is_v ? a.v_cache : a.k_cache;
            at = ((((int64_t)(slot[j] >> a.page_shift) * a.G + g) << a.page_shift) +
                  (slot[j] & (page - 1))) * LPH + l;
        }
        reinterpret_cast<u32x4 *>(dst)[at] = y;
    }
}

}  // namespace

int64_t cache_rope_groups(const CacheArgs &a) {
    return (a.T * (a.H + 2 * (int64_t)a.G) * (a.D / 8) + kStep - 1) / kStep;
}

hipError_t launch_cache_rope(const CacheArgs &a, hipStream_t stream) {
    const unsigned grid = (unsigned)cache_rope_groups(a);
    auto *kernel = a.D == 64 ? (a.half ? cache_rope_kernel<64, true> : cache_rope_kernel<64, false>)
                             : (a.half ? cache_rope_kernel<128, true> : cache_rope_kernel<128, false>);
    kernel<<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace svdq
