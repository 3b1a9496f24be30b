// i8_internal.h -- launchers of the 8-bit integer linear (internal; not part
// of the ABI).
#pragma once

#include "svdq_i8.h"
#include "svdq_internal.h"

namespace svdq {

// X bf16 [M, K] (smoothed by 1 / lambda unless lambda is null) or, with
// `fp32`, fp32 rows without smoothing -> codes [M, K] and scales [M]
hipError_t launch_i8_quantize(const void *X, bool fp32, const float *lambda, int64_t M, int64_t K,
                              int8_t *q, float *s, hipStream_t stream);
int64_t i8_quantize_groups(int64_t M, int64_t K);   // workgroups, and their threads
int64_t i8_quantize_threads(int64_t K);

hipError_t launch_i8_gemm(const int8_t *qa, const float *sa, const int8_t *qw, const float *sw,
                          const uint16_t *bias, int act, int64_t M, int64_t N, int64_t K,
                          uint16_t *Y, hipStream_t stream);
int64_t i8_gemm_groups(int64_t M, int64_t N);       // workgroups at most, of 512

// Quantization and product in one launch, for a few tokens (i8_few_tokens):
// workgroups of 256 for 32 channels each (16 up to N = 8192, 8 up to 2048).
bool i8_few_tokens(int64_t M, int64_t N, int64_t K);
hipError_t launch_i8_few(const uint16_t *X, const float *lambda, const int8_t *qw, const float *sw,
                         const uint16_t *bias, int act, int64_t M, int64_t N, int64_t K,
                         uint16_t *Y, hipStream_t stream);

}  // namespace svdq
