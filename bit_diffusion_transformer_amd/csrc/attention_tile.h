// attention_tile.h -- device helpers of the attention kernels' tiles (internal;
// not part of the ABI).
#pragma once

#include "svdq_wave.h"

namespace svdq {

namespace attn {

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

}  // namespace attn

}  // namespace svdq
