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
// 0x8000 in each half of x whose bf16 value is not finite.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
    return ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
// bf16 ones in the halves of a pair of keys n, n + 1 that a row sees, the first `limit` keys.
__device__ __forceinline__ uint32_t seen_pair(int n, int limit) {
    return (n < limit ? 0x3F80u : 0u) | (n + 1 < limit ? 0x3F800000u : 0u);
}
__device__ __forceinline__ float max_both_halves(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float sum_both_halves(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// The LDS address of a __shared__ object.
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}
// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ const uint8_t *uniform_pointer(const uint8_t *p) {
    const uint64_t x = reinterpret_cast<uint64_t>(p);
    return reinterpret_cast<const uint8_t *>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)x) |
                                             (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32);
}

// 16 bytes per lane from base + off[i] (base uniform) straight into LDS, lane l's to address
// `to` + 1024 i + 16 l (to uniform).  As assembly, because the compiler waits for all copies
// that it knows of before a transposing read, those into other buffers too; the callers count
// their copies and wait for them (wait_loads).  There is no output register, and the waits
// that the compiler puts for its own loads can only get longer by it.  The first wait states
// are what a load needs behind a vector instruction that wrote its base (five), the others
// what it needs behind a write of m0 (one).
__device__ __forceinline__ void copy_in_flight(const uint8_t *base, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(off), "s"(uniform_pointer(base)), "s"(__builtin_amdgcn_readfirstlane(to)) : "memory");
}
__device__ __forceinline__ void copies_in_flight(const uint8_t *base, const uint32_t (&off)[1], uint32_t to) {
    copy_in_flight(base, off[0], to);
}
__device__ __forceinline__ void copies_in_flight(const uint8_t *base, const uint32_t (&off)[2], uint32_t to) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %2\n\t"
                 "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "v"(off[0]), "v"(off[1]), "s"(uniform_pointer(base)), "s"(__builtin_amdgcn_readfirstlane(to)) : "memory", "scc");
}
__device__ __forceinline__ void copies_in_flight(const uint8_t *base, const uint32_t (&off)[4], uint32_t to) {
    asm volatile("s_mov_b32 m0, %5\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %4\n\t"
                 "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %4\n\t"
                 "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %4\n\t"
                 "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %4"
                 :: "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(uniform_pointer(base)), "s"(__builtin_amdgcn_readfirstlane(to))
                 : "memory", "scc");
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
