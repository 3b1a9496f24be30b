// qkv_rope.hip -- rotary tables of tokens with several position axes, and the
// Q / K norm and rotary turn of a projection written as [M, 3 H D] (the work
// that the fused QKV epilogue of w4a4_tile.h does on its own tile, for the
// GEMMs without one).
#include "attention_internal.h"
#include "svdq_wave.h"

namespace svdq {

namespace {

constexpr int kPairs = SVDQ_ROPE_MAX_DIM / 2;

// cos_t[s][p], sin_t[s][p] of angle pos[s][axis(p)] theta^(-2 i / dims): bound
// by the stores of both tables, 8 bytes a pair (118800 tokens of 64 pairs: 14.3
// us, 4.3 TB/s; 4608 tokens: 3.5 us, the launch and one pass of the sines).  The angle is taken in turns
// in 64 bits, t = pos (f / 2 pi), and loses its whole turns there (an exact
// step), so a position of 2^26 keeps 2^-27 of a turn; what is left,
// at most half a turn, fits fp32 and goes through the fp32 sine and cosine of
// a multiple of pi.  The pairs' frequencies are formed once per workgroup (a
// 64-bit exponential each), then 16 lanes (D = 128) write a token's row in
// 16-byte stores.
__global__ void __launch_bounds__(256)
rope_tables_kernel(const float *__restrict__ pos, int64_t S, RopeAxes ax, int pairs,
                   float *__restrict__ cos_t, float *__restrict__ sin_t) {
    __shared__ double freq[kPairs];   // turns per unit of position
    __shared__ int axis[kPairs];
    for (int p = threadIdx.x; p < pairs; p += 256) {
        int a = 0, i = p;
        while (i >= ax.dims[a] / 2) i -= ax.dims[a++] / 2;
        axis[p] = a;
        freq[p] = exp(-2.0 * i / ax.dims[a] * ax.log_theta[a]) * 0.15915494309189535;
    }
    __syncthreads();
    const int quads = pairs / 4;                  // 16-byte stores per row
    const int64_t total = S * quads;              // checked on the host: fits the grid
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += step) {
        const int64_t s = id / quads;
        const int p = 4 * (int)(id - s * quads);
        f32x4 c, d;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            double t = (double)pos[s * ax.axes + axis[p + j]] * freq[p + j];
            t -= rint(t);
            const float h = (float)(t + t);       // half turns, |h| <= 1
            c[j] = cospif(h);
            d[j] = sinpif(h);
        }
        *reinterpret_cast<f32x4 *>(cos_t + s * pairs + p) = c;
        *reinterpret_cast<f32x4 *>(sin_t + s * pairs + p) = d;
    }
}

constexpr int kPer = 4;                // 16-byte pieces per thread
constexpr int kStep = 256 * kPer;      // pieces per workgroup

// [M, 3 H D] -> Q, K (normed and turned), V [B, H, S, D].  Bound by memory: each
// element is read and written once, 2 bytes each way, plus the two table rows
// of a token (1/(6 H) of that).  A lane holds 16 bytes (8 elements, 4 pairs) of
// one head, so a head is 8 or 16 neighbouring lanes, its sum of squares is
// three or four lane exchanges, and loads and stores are 16 bytes wide and
// contiguous over a head's row.  A thread's four pieces are loaded before the
// first is used.  4608 tokens of 24 heads of 128: 37.5 us, 4.6 TB/s; 9003 tokens
// of 18 heads of 64: 26.1 us, 4.8 TB/s; one token: 3.2 us, the launch.
template <int D>
__global__ void __launch_bounds__(256)
qkv_norm_rope_kernel(const uint16_t *__restrict__ qkv, int64_t M, QkvArgs a) {
    constexpr int LPH = D / 8;                              // lanes per head
    const uint32_t row = 3u * (uint32_t)a.H * LPH;          // pieces per token
    const int64_t id0 = (int64_t)blockIdx.x * kStep;
    const int64_t tok0 = id0 / row;                         // uniform
    const uint32_t rem0 = (uint32_t)(id0 - tok0 * row);
    const int64_t total = M * row;
    const uint32_t S = (uint32_t)a.S;
    u32x4 x[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int64_t id = id0 + j * 256 + threadIdx.x;
        x[j] = id < total ? reinterpret_cast<const u32x4 *>(qkv)[id] : u32x4{};
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int64_t id = id0 + j * 256 + threadIdx.x;
        if (id >= total) break;                             // whole heads: `total` is a multiple of LPH
        const uint32_t r = rem0 + j * 256 + threadIdx.x;
        const uint32_t dt = r / row;
        const uint32_t piece = r - dt * row;
        const uint32_t tok = (uint32_t)tok0 + dt;           // < 2^28
        const uint32_t head = piece / LPH, l = piece % LPH; // head over the three sections
        const uint32_t sec = head / (uint32_t)a.H, h = head - sec * (uint32_t)a.H;
        const uint32_t b = tok / S, s = tok - b * S;
        uint16_t *dst = sec == 0 ? a.Q : sec == 1 ? a.K : a.V;
        u32x4 y = x[j];
        if (sec < 2) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(x[j][i]);
                v[2 * i + 1] = bf16_hi(x[j][i]);
            }
            const uint16_t *gamma = sec == 0 ? a.gq : a.gk;
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
            const f32x4 c = *reinterpret_cast<const f32x4 *>(a.cos_t + (int64_t)s * (D / 2) + 4 * l);
            const f32x4 n = *reinterpret_cast<const f32x4 *>(a.sin_t + (int64_t)s * (D / 2) + 4 * l);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = v[2 * i], q = v[2 * i + 1];
                y[i] = pack_bf16x2(__builtin_fmaf(p, c[i], -(q * n[i])),
                                   __builtin_fmaf(p, n[i], q * c[i]));
            }
        }
        const int64_t at = (((int64_t)b * a.H + h) * a.S + s) * LPH + l;
        reinterpret_cast<u32x4 *>(dst)[at] = y;
    }
}

}  // namespace

hipError_t launch_rope_tables(const float *pos, int64_t S, const RopeAxes &ax, int pairs,
                              float *cos_t, float *sin_t, hipStream_t stream) {
    const int64_t want = (S * (pairs / 4) + 255) / 256;
    const unsigned grid = (unsigned)(want < 2048 ? want : 2048);   // grid-stride
    rope_tables_kernel<<<grid, 256, 0, stream>>>(pos, S, ax, pairs, cos_t, sin_t);
    return hipGetLastError();
}

int64_t qkv_norm_rope_groups(int64_t M, int heads, int head_dim) {
    return (M * 3 * heads * (head_dim / 8) + kStep - 1) / kStep;
}

hipError_t launch_qkv_norm_rope(const uint16_t *qkv, int64_t M, const QkvArgs &a,
                                hipStream_t stream) {
    const unsigned grid = (unsigned)qkv_norm_rope_groups(M, a.H, a.D);
    if (a.D == 64)
        qkv_norm_rope_kernel<64><<<grid, 256, 0, stream>>>(qkv, M, a);
    else
        qkv_norm_rope_kernel<128><<<grid, 256, 0, stream>>>(qkv, M, a);
    return hipGetLastError();
}

}  // namespace svdq
