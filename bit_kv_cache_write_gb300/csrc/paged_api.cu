// Host side of the BF16 paged-cache calls in include/oscar.h: argument checks, plans, launches.
#include "paged_internal.h"

namespace {

using oscar::record_failure;

oscar_status cuda_status(cudaError_t e, const char* where) {
    return e == cudaSuccess ? OSCAR_OK : record_failure(OSCAR_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Whether n ints at a and m ints at b share memory.
bool overlap(const int32_t* a, long long n, const int32_t* b, long long m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return n > 0 && m > 0 && x < y + 4 * (uintptr_t)m && y < x + 4 * (uintptr_t)n;
}

int pages_of(int tokens) { return (tokens + oscar::kPage - 1) / oscar::kPage; }

bool sizes_ok(const oscar_ctx_t* ctx, int batch, int max_len) {
    return ctx && batch >= 0 && batch <= oscar::kMaxBatch && max_len >= 0 && max_len <= oscar::kMaxPagedLen;
}

// Pages that one (sequence, KV head) of a sparse decode reads at most.
int sparse_pages(const oscar_ctx_t* ctx, int max_len, int top) {
    const int cap = oscar::sparse_capacity(ctx->shape, top), all = pages_of(max_len);
    return cap < all ? cap : all;
}

// What the dense and the sparse decode check alike.
oscar_status check_decode(const oscar_ctx_t* ctx, const void* q, int64_t q_stride, const void* pool, int64_t pages,
                          const int32_t* tables, int stride, const int32_t* seq_len, int max_len, const void* out,
                          int out_type, int batch) {
    if (batch < 0 || max_len < 0)
        return record_failure(OSCAR_ERR_INVALID_ARG, "batch %d / max_len %d negative", batch, max_len);
    if (batch > oscar::kMaxBatch || max_len > oscar::kMaxPagedLen)
        return record_failure(OSCAR_ERR_UNSUPPORTED, "batch %d above %d or max_len %d above %d", batch,
                              oscar::kMaxBatch, max_len, oscar::kMaxPagedLen);
    if (out_type != OSCAR_OUT_FP32 && out_type != OSCAR_OUT_BF16)
        return record_failure(OSCAR_ERR_UNSUPPORTED, "out_type %d not in {0 (fp32), 1 (bf16)}", out_type);
    if (batch == 0) return OSCAR_OK;
    if (!q || !seq_len || !out) return record_failure(OSCAR_ERR_INVALID_ARG, "device pointer is NULL");
    if (!pool || pages <= 0 || (max_len > 0 && (!tables || stride <= 0)))
        return record_failure(OSCAR_ERR_INVALID_ARG, "BF16 pool/tables missing");
    if (max_len > 0 && (long long)max_len > (long long)stride * oscar::kPage)
        return record_failure(OSCAR_ERR_INVALID_ARG, "max_len %d exceeds table stride %d pages", max_len, stride);
    if (q_stride < 0 || q_stride % 8 || !aligned(q, 16) || !aligned(pool, 32) || !aligned(out, 16))
        return record_failure(OSCAR_ERR_INVALID_ARG,
                              "q and out must be 16-byte aligned, the pool 32-byte, q_stride a multiple of 8 (is %lld)",
                              (long long)q_stride);
    return OSCAR_OK;
}

oscar_status check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (need > 0 && (!workspace || bytes < need))
        return record_failure(OSCAR_ERR_WORKSPACE, "workspace %zu bytes, need %zu", bytes, need);
    if (need > 0 && !aligned(workspace, 256))
        return record_failure(OSCAR_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    if (oscar::injected_fault("launch"))
        return record_failure(OSCAR_ERR_CUDA, "injected launch failure (OSCAR_FAULT=launch)");
    return OSCAR_OK;
}

oscar::AttendArgs attend_args(oscar_ctx_t* ctx, const oscar::AttendPlan& plan, const void* q, int64_t q_stride,
                              const void* pool, int64_t pages, const int32_t* tables, int stride,
                              const int32_t* seq_len, int max_len, void* out, int out_type, void* workspace,
                              int batch) {
    oscar::AttendArgs a{};
    a.q = static_cast<const uint16_t*>(q); a.q_stride = q_stride;
    a.pool = static_cast<const uint16_t*>(pool); a.pages = pages;
    a.tables = tables; a.stride = max_len > 0 ? stride : 0;      // page ids are looked up ahead of the lengths
    a.seq_len = seq_len; a.max_len = max_len;
    a.out = out; a.out_bf16 = out_type == OSCAR_OUT_BF16;
    a.split_acc = static_cast<float*>(workspace);
    a.split_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + plan.ws_acc);
    a.h_kv = ctx->shape.h_kv; a.g = ctx->shape.h_q / ctx->shape.h_kv;
    a.splits = plan.splits; a.pages_per_split = plan.pages_per_split; a.cluster = plan.cluster; a.batch = batch;
    a.scale_log2 = (float)(ctx->shape.sm_scale * 1.4426950408889634073599);
    a.debug = ctx->shape.debug; a.dbg = ctx->dbg;
    return a;
}

}  // namespace

extern "C" {

oscar_status oscar_plan_append(oscar_ctx_t* ctx, const int32_t* seq_len, const int32_t* new_len, int batch,
                               const int32_t* free_pages, int n_free, const int32_t* free_head, int32_t* tables,
                               int table_stride, int64_t* slots, int slot_cap, int32_t* row_start,
                               int32_t* total_len, int32_t* state, void* stream) {
    if (oscar_status st = oscar::check_context(ctx); st != OSCAR_OK) return st;
    if (batch < 0 || n_free < 0 || table_stride < 0 || slot_cap < 0)
        return record_failure(OSCAR_ERR_INVALID_ARG, "batch %d, n_free %d, table_stride %d or slot_cap %d negative",
                              batch, n_free, table_stride, slot_cap);
    if (batch > oscar::kMaxBatch || table_stride > oscar::kMaxPagedLen / oscar::kPage)
        return record_failure(OSCAR_ERR_UNSUPPORTED, "batch %d above %d or table_stride %d above %d", batch,
                              oscar::kMaxBatch, table_stride, oscar::kMaxPagedLen / oscar::kPage);
    if (!free_head || !row_start || !state || (batch > 0 && (!seq_len || !new_len || !total_len)) ||
        (n_free > 0 && !free_pages) || (slot_cap > 0 && !slots) || (batch > 0 && table_stride > 0 && !tables))
        return record_failure(OSCAR_ERR_INVALID_ARG, "device pointer is NULL");
    // every CTA reads the lengths while others write: what is written has to lie apart
    if (overlap(total_len, batch, seq_len, batch) || overlap(total_len, batch, new_len, batch) ||
        overlap(row_start, batch + 1LL, seq_len, batch) || overlap(row_start, batch + 1LL, new_len, batch) ||
        overlap(row_start, batch + 1LL, total_len, batch) || overlap(state, 4, seq_len, batch) ||
        overlap(state, 4, new_len, batch) || overlap(state, 4, total_len, batch) ||
        overlap(state, 4, row_start, batch + 1LL) || overlap(total_len, batch, free_head, 1) ||
        overlap(row_start, batch + 1LL, free_head, 1))
        return record_failure(OSCAR_ERR_INVALID_ARG,
                              "seq_len, new_len, row_start, total_len and state must not overlap (free_head may lie in state)");
    if (oscar::injected_fault("launch"))
        return record_failure(OSCAR_ERR_CUDA, "injected launch failure (OSCAR_FAULT=launch)");
    oscar::PlanArgs a{seq_len, new_len, free_pages, n_free, free_head, tables, table_stride, slots, slot_cap,
                      row_start, total_len, state, batch};
    oscar::ProfScope ps(&ctx->prof, OSCAR_KERNEL_PLAN, static_cast<cudaStream_t>(stream));
    return cuda_status(oscar::launch_plan(a, static_cast<cudaStream_t>(stream)), "plan launch");
}

oscar_status oscar_append_bf16(oscar_ctx_t* ctx, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               const int64_t* slots, int n, void* bf16_pool, int64_t bf16_pool_pages,
                               const int8_t* key_steps, int8_t* key_bounds, void* stream) {
    if (oscar_status st = oscar::check_context(ctx); st != OSCAR_OK) return st;
    if (n < 0) return record_failure(OSCAR_ERR_INVALID_ARG, "n = %d is negative", n);
    if (n == 0) return OSCAR_OK;
    if (!k || !v || !slots || !bf16_pool) return record_failure(OSCAR_ERR_INVALID_ARG, "device pointer is NULL");
    if (!key_steps != !key_bounds)
        return record_failure(OSCAR_ERR_INVALID_ARG, "key_steps and key_bounds go together");
    if (bf16_pool_pages <= 0) return record_failure(OSCAR_ERR_INVALID_ARG, "bf16_pool_pages must be positive");
    if (k_stride < 0 || v_stride < 0 || k_stride % 8 || v_stride % 8 || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(bf16_pool, 16) || !aligned(key_bounds, 16) || !aligned(key_steps, 8))
        return record_failure(OSCAR_ERR_INVALID_ARG,
                              "k, v, the pool and the bounds must be 16-byte aligned, the steps 8-byte, the strides "
                              "multiples of 8 (are %lld and %lld)", (long long)k_stride, (long long)v_stride);
    if (oscar::injected_fault("launch"))
        return record_failure(OSCAR_ERR_CUDA, "injected launch failure (OSCAR_FAULT=launch)");
    oscar::AppendArgs a{};
    a.k = static_cast<const uint16_t*>(k); a.k_stride = k_stride;
    a.v = static_cast<const uint16_t*>(v); a.v_stride = v_stride;
    a.slots = slots; a.n = n;
    a.pool = static_cast<uint16_t*>(bf16_pool); a.pages = bf16_pool_pages;
    a.steps = key_steps; a.bounds = key_bounds;
    a.h_kv = ctx->shape.h_kv; a.debug = ctx->shape.debug; a.dbg = ctx->dbg;
    oscar::ProfScope ps(&ctx->prof, OSCAR_KERNEL_APPEND, static_cast<cudaStream_t>(stream));
    return cuda_status(oscar::launch_append(a, ctx->shape.d, ctx->num_sms, static_cast<cudaStream_t>(stream)),
                       "append launch");
}

size_t oscar_decode_bf16_workspace_size(const oscar_ctx_t* ctx, int batch, int max_len) {
    if (!sizes_ok(ctx, batch, max_len)) return 0;
    return oscar::attend_workspace_bytes(ctx->shape, ctx->num_sms, batch, pages_of(max_len), false);
}

oscar_status oscar_decode_bf16(oscar_ctx_t* ctx, const void* q, int64_t q_stride, const void* bf16_pool,
                               int64_t bf16_pool_pages, const int32_t* tables, int table_stride,
                               const int32_t* seq_len, int max_len, void* out, int out_type, void* workspace,
                               size_t workspace_bytes, int batch, void* stream) {
    if (oscar_status st = oscar::check_context(ctx); st != OSCAR_OK) return st;
    oscar_status st = check_decode(ctx, q, q_stride, bf16_pool, bf16_pool_pages, tables, table_stride, seq_len, max_len,
                                   out, out_type, batch);
    if (st != OSCAR_OK || batch == 0) return st;
    const oscar::AttendPlan plan = oscar::plan_attend(ctx->shape, ctx->num_sms, batch, pages_of(max_len), false);
    st = check_workspace(workspace, workspace_bytes, plan.ws_total);
    if (st != OSCAR_OK) return st;
    const oscar::AttendArgs a = attend_args(ctx, plan, q, q_stride, bf16_pool, bf16_pool_pages, tables, table_stride,
                                            seq_len, max_len, out, out_type, workspace, batch);
    oscar::ProfScope ps(&ctx->prof, OSCAR_KERNEL_ATTEND, static_cast<cudaStream_t>(stream));
    return cuda_status(oscar::launch_attend(a, ctx->shape.d, static_cast<cudaStream_t>(stream)), "BF16 decode launch");
}

int oscar_sparse_capacity(const oscar_ctx_t* ctx, int top_pages) {
    if (!ctx || top_pages < 0 || top_pages > oscar::kMaxTopPages) return 0;
    return oscar::sparse_capacity(ctx->shape, top_pages);
}

size_t oscar_decode_bf16_sparse_workspace_size(const oscar_ctx_t* ctx, int batch, int max_len, int top_pages) {
    if (!sizes_ok(ctx, batch, max_len) || top_pages < 0 || top_pages > oscar::kMaxTopPages) return 0;
    return oscar::attend_workspace_bytes(ctx->shape, ctx->num_sms, batch, sparse_pages(ctx, max_len, top_pages), true) +
           oscar::select_workspace_bytes(ctx->shape, batch, pages_of(max_len));
}

oscar_status oscar_decode_bf16_sparse(oscar_ctx_t* ctx, const void* q, int64_t q_stride, const void* bf16_pool,
                                      int64_t bf16_pool_pages, const int8_t* key_steps, const int8_t* key_bounds,
                                      const int32_t* tables, int table_stride, const int32_t* seq_len, int max_len,
                                      int top_pages, int32_t* chosen, int32_t* n_chosen, void* out, int out_type,
                                      void* workspace, size_t workspace_bytes, int batch, void* stream) {
    if (oscar_status st = oscar::check_context(ctx); st != OSCAR_OK) return st;
    oscar_status st = check_decode(ctx, q, q_stride, bf16_pool, bf16_pool_pages, tables, table_stride, seq_len, max_len,
                                   out, out_type, batch);
    if (st != OSCAR_OK) return st;
    if (top_pages < 0) return record_failure(OSCAR_ERR_INVALID_ARG, "top_pages %d negative", top_pages);
    if (top_pages > oscar::kMaxTopPages)
        return record_failure(OSCAR_ERR_UNSUPPORTED, "top_pages %d above %d", top_pages, oscar::kMaxTopPages);
    if (batch == 0) return OSCAR_OK;
    if (!key_steps || !key_bounds || !chosen || !n_chosen)
        return record_failure(OSCAR_ERR_INVALID_ARG, "device pointer is NULL");
    if (!aligned(key_bounds, 32))
        return record_failure(OSCAR_ERR_INVALID_ARG, "key_bounds must be 32-byte aligned");
    const int max_pages = pages_of(max_len);
    const int ranks = oscar::sparse_small_ranks(ctx->shape, ctx->num_sms, batch, max_pages, top_pages);
    const oscar::AttendPlan plan =
        ranks ? oscar::AttendPlan{} : oscar::plan_attend(ctx->shape, ctx->num_sms, batch, sparse_pages(ctx, max_len, top_pages), true);
    const size_t scores = ranks ? 0 : oscar::select_workspace_bytes(ctx->shape, batch, max_pages);
    st = check_workspace(workspace, workspace_bytes, scores + plan.ws_total);
    if (st != OSCAR_OK) return st;

    oscar::AttendArgs a = attend_args(ctx, plan, q, q_stride, bf16_pool, bf16_pool_pages, tables, table_stride,
                                      seq_len, max_len, out, out_type, static_cast<char*>(workspace) + scores, batch);
    a.chosen = chosen; a.n_chosen = n_chosen; a.cap = oscar::sparse_capacity(ctx->shape, top_pages);
    oscar::SelectArgs s{};
    s.q = static_cast<const uint16_t*>(q); s.q_stride = q_stride;
    s.steps = key_steps; s.bounds = key_bounds; s.pages = bf16_pool_pages;
    s.tables = tables; s.stride = a.stride;
    s.seq_len = seq_len; s.max_len = max_len;
    s.chosen = chosen; s.n_chosen = n_chosen; s.cap = a.cap;
    s.keys = static_cast<uint32_t*>(workspace);
    s.max_pages = max_pages; s.top = top_pages; s.sink = ctx->shape.sink; s.recent = ctx->shape.recent;
    s.h_kv = ctx->shape.h_kv; s.g = ctx->shape.h_q / ctx->shape.h_kv; s.batch = batch;
    s.debug = ctx->shape.debug; s.dbg = ctx->dbg;
    if (ranks) {
        oscar::ProfScope ps(&ctx->prof, OSCAR_KERNEL_ATTEND, static_cast<cudaStream_t>(stream));
        return cuda_status(oscar::launch_sparse_small(s, a, ctx->shape.d, ranks, static_cast<cudaStream_t>(stream)),
                           "sparse BF16 decode launch");
    }
    {
        oscar::ProfScope ps(&ctx->prof, OSCAR_KERNEL_SELECT, static_cast<cudaStream_t>(stream));
        st = cuda_status(oscar::launch_select(s, ctx->shape.d, ctx->num_sms, static_cast<cudaStream_t>(stream)), "page selection launch");
        if (st != OSCAR_OK) return st;
    }
    oscar::ProfScope ps(&ctx->prof, OSCAR_KERNEL_ATTEND, static_cast<cudaStream_t>(stream));
    return cuda_status(oscar::launch_attend(a, ctx->shape.d, static_cast<cudaStream_t>(stream)),
                       "sparse BF16 decode launch");
}

}  // extern "C"
