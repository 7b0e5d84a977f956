// Internal declarations of the operators on chunks of new tokens: norm and rotation, attention over the BF16 cache.
#pragma once

#include "paged_internal.h"

namespace oscar {

// ---- norm and rotation of queries and keys (norm_rope.cu)
struct RopeRows {
    const uint16_t* in; int64_t in_stride;   // token stride in elements
    uint16_t* out; int64_t out_stride;
    const float* weight;                     // [d] or null: no norm
    int heads;                               // 0: none of these rows
};
struct RopeArgs {
    RopeRows q, k;
    float eps;
    const uint64_t* turns; int rot;          // [rot / 2] turns a position, in units of 2^-64
    int interleaved;
    float scale;                             // of the rotated channels
    const int32_t* positions;                // [n] or null: from the two below
    const int32_t* row_start;                // [batch + 1]
    const int32_t* total_len;                // [batch]
    int batch, n;
};
cudaError_t launch_norm_rope(const RopeArgs& a, int d, int num_sms, cudaStream_t st);

}  // namespace oscar
