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

// A checked svdq_attention_shape and what follows from it.
struct AttnShape {
    int64_t B, seq_q, seq_k;
    int64_t nq, nk;               // query blocks of 128 rows, key blocks of 64
    int64_t planes_q, planes_k;   // B H, B G
    int H, G, D, keep, first;
    bool every() const { return keep >= nk; }   // lists hold every block with a valid key
};

size_t select_workspace(const AttnShape &a);
hipError_t launch_select_blocks(const uint16_t *q, const uint16_t *k, const int32_t *kv_len,
                                const AttnShape &a, int32_t *blocks, void *ws, hipStream_t stream);

int attention_splits(const AttnShape &a);   // workgroups that share a query block's keys
size_t attention_workspace(const AttnShape &a);
// blocks null: every block with a valid key, the lists written to `made` unless null
hipError_t launch_block_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v,
                                  const int32_t *kv_len, const AttnShape &a, float scale,
                                  const int32_t *blocks, int32_t *made, uint16_t *out, void *ws,
                                  hipStream_t stream);

}  // namespace svdq
