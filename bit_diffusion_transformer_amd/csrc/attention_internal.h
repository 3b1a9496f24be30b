// attention_internal.h -- launchers of the rotary and attention kernels
// (internal; not part of the ABI).
#pragma once

#include "svdq_attention.h"
#include "svdq_internal.h"

namespace svdq {

struct RopeAxes {
    int axes;
    int dims[SVDQ_ROPE_MAX_AXES];
    double log_theta[SVDQ_ROPE_MAX_AXES];   // natural logarithms
};
// pairs = sum(dims) / 2, a multiple of 4
hipError_t launch_rope_tables(const float *pos, int64_t S, const RopeAxes &ax, int pairs,
                              float *cos_t, float *sin_t, hipStream_t stream);

int64_t qkv_norm_rope_groups(int64_t M, int heads, int head_dim);   // workgroups of 256
// gamma pointers of `a` may be null (no norm of that section)
hipError_t launch_qkv_norm_rope(const uint16_t *qkv, int64_t M, const QkvArgs &a,
                                hipStream_t stream);

}  // namespace svdq
