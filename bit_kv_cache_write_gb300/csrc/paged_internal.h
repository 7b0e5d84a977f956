// Internal declarations of the BF16 paged-cache operators: planning, appending, dense and sparse decode.
#pragma once

#include "oscar_internal.h"

namespace oscar {

constexpr int kMaxTopPages = 1 << 16;       // selected pages per (sequence, KV head) of a sparse decode
constexpr int kMaxPagedLen = 1 << 30;       // tokens per sequence: page and token indices stay in 32 bits

// ---- planning (plan_kernels.cu)
struct PlanArgs {
    const int32_t* seq_len;      // [batch] tokens cached
    const int32_t* new_len;      // [batch] tokens to append
    const int32_t* free_pages;   // [n_free]
    int n_free;
    const int32_t* free_head;    // [1]; may be state[0]
    int32_t* tables; int stride; // [batch][stride]
    int64_t* slots; int slot_cap;
    int32_t* row_start;          // [batch + 1]
    int32_t* total_len;          // [batch]
    int32_t* state;              // [4]
    int batch;
};
cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st);

// ---- appending (append_kernels.cu)
struct AppendArgs {
    const uint16_t* k; int64_t k_stride;     // token stride in elements
    const uint16_t* v; int64_t v_stride;
    const int64_t* slots; int n;
    uint16_t* pool; int64_t pages;
    const int8_t* steps;                     // [H_kv][d] or null
    int8_t* bounds;                          // [pages][H_kv][2][d] or null
    int h_kv;
    int debug; DebugWord* dbg;
};
cudaError_t launch_append(const AppendArgs& a, int d, int num_sms, cudaStream_t st);

// ---- attention of one new token (paged_attend.cu)
struct AttendPlan {
    int pages_per_split;
    int splits;                  // CTAs of one (sequence, KV head)
    bool cluster;                // they are a cluster and join their parts without a second kernel
    size_t ws_acc;               // bytes of the splits' accumulators
    size_t ws_total;             // and of their references and sums
};
struct AttendArgs {
    const uint16_t* q; int64_t q_stride;     // sequence stride in elements
    const uint16_t* pool; int64_t pages;
    const int32_t* tables; int stride;
    const int32_t* seq_len; int max_len;
    const int32_t* chosen; const int32_t* n_chosen; int cap;   // sparse: logical pages per (sequence, KV head)
    void* out; int out_bf16;
    float* split_acc;                        // [batch][H_q][splits][d]
    float2* split_ml;                        // [batch][H_q][splits] reference and sum of weights
    int h_kv, g, splits, pages_per_split, cluster, batch;
    float scale_log2;                        // sm_scale * log2(e)
    int debug; DebugWord* dbg;
};
// max_pages: pages that one (sequence, KV head) reads at most.
AttendPlan plan_attend(const Shape& s, int num_sms, int batch, int max_pages, bool sparse);
// What plan_attend's workspaces need at most for this many sequences and pages, or fewer of either.
size_t attend_workspace_bytes(const Shape& s, int num_sms, int batch, int max_pages, bool sparse);
cudaError_t launch_attend(const AttendArgs& a, int d, cudaStream_t st);

// ---- page selection of the sparse decode (page_select.cu)
struct SelectArgs {
    const uint16_t* q; int64_t q_stride;
    const int8_t* steps;                     // [H_kv][d]
    const int8_t* bounds; int64_t pages;     // [pages][H_kv][2][d]
    const int32_t* tables; int stride;
    const int32_t* seq_len; int max_len;
    int32_t* chosen; int32_t* n_chosen; int cap;
    uint32_t* keys;                          // [batch][H_kv][max_pages], for sequences too long for shared memory
    int max_pages, top, sink, recent;
    int sorted;                              // clusters start with the longest sequences
    int h_kv, g, batch;
    int debug; DebugWord* dbg;
};
size_t select_workspace_bytes(const Shape& s, int batch, int max_pages);
cudaError_t launch_select(const SelectArgs& a, int d, int num_sms, cudaStream_t st);

// ---- both in one kernel, for few (sequence, KV head) pairs (sparse_small.cu)
// CTAs of a pair's cluster, or 0 where the separate kernels serve better.
int sparse_small_ranks(const Shape& s, int num_sms, int batch, int max_pages, int top);
cudaError_t launch_sparse_small(const SelectArgs& a, const AttendArgs& t, int d, int ranks, cudaStream_t st);

// Entries of one (sequence, KV head)'s list of chosen pages: the sink's pages, the pages that a recent
// window can touch (one more than it fills), the selected ones.
inline int sparse_capacity(const Shape& s, int top) {
    return (s.sink + kPage - 1) / kPage + (s.recent + kPage - 1) / kPage + 1 + top;
}

}  // namespace oscar
