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

// ---- attention of new tokens over BF16 pages (chunk_attend.cu)
constexpr int kChunkRows = 256;              // query rows (token, head of the group) of a work item
constexpr int kChunkTile = 128;              // cached tokens of a step
constexpr uint32_t kChunkWait = 2000000000u; // cycles of a wait at most, about a second
constexpr uint32_t kLostWait = 2000000u;     // the same where loads are lost on purpose, about a millisecond

// Where the parts of a call's workspace lie, in bytes.
struct ChunkPlan {
    int unit_cap;                            // row blocks of all requests at most
    int item_cap;                            // work items at most
    int part_cap;                            // rows of split items at most
    int fold_rows;                           // rows of an item at most
    size_t tiles, units, items, odd, marked, part_ml, part_acc, fold_ml, fold_acc, total;
};
struct ChunkArgs {
    const uint16_t* q; int64_t q_stride;     // token stride in elements
    const uint16_t* pool; int64_t pages;
    const int32_t* tables; int stride;
    const int32_t* row_start;                // [batch + 1]
    const int32_t* total_len;                // [batch]
    uint16_t* out;                           // [n][H_q][d]
    int batch, n, h_kv, g, d;
    float scale_log2;                        // sm_scale * log2(e)
    int debug; DebugWord* dbg;
    uint32_t wait_ticks;                     // cycles that a role waits for another at most
    int lost_loads;                          // every other CTA's loader stops in its first item and tells nobody: waits run out
};
ChunkPlan plan_chunk(const Shape& s, int num_sms, int batch, int n);
cudaError_t launch_chunk(const ChunkArgs& a, const ChunkPlan& plan, void* workspace, int d, int num_sms, cudaStream_t st);

}  // namespace oscar
