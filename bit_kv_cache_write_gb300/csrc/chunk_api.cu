// Host side of the calls on chunks of new tokens in include/oscar.h: argument checks, launches.
#include <cmath>

#include "chunk_internal.h"

namespace {

using oscar::record_failure;

oscar_status cuda_status(cudaError_t e, const char* where) {
    return e == cudaSuccess ? OSCAR_OK : record_failure(OSCAR_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// n rows of `width` elements, `stride` apart.
struct Rows {
    const void* p;
    int64_t stride, width;
};

// Whether two sets of n bf16 rows share an element. Sets of one stride that lie in each other's gaps (slices of one
// row) do not; sets of different strides whose spans meet count as sharing.
bool share(const Rows& a, const Rows& b, int n) {
    if (n <= 0 || a.width == 0 || b.width == 0) return false;
    const intptr_t x = reinterpret_cast<intptr_t>(a.p) / 2, y = reinterpret_cast<intptr_t>(b.p) / 2;
    const int64_t sa = n > 1 ? a.stride : a.width, sb = n > 1 ? b.stride : b.width;
    const intptr_t x_end = x + (n - 1) * sa + a.width, y_end = y + (n - 1) * sb + b.width;
    if (x_end <= y || y_end <= x) return false;
    if (n == 1 || sa != sb || sa == 0) return true;
    const int64_t off = ((y - x) % sa + sa) % sa;
    return off < a.width || sa - off < b.width;
}

oscar_status check_rows(const char* name, const void* in, int64_t in_stride, const void* out, int64_t out_stride,
                        const float* weight, int width) {
    if (!in != !out) return record_failure(OSCAR_ERR_INVALID_ARG, "%s and %s_out go together", name, name);
    if (!in) return OSCAR_OK;
    constexpr int64_t kMaxStride = (int64_t)1 << 31;
    if (in_stride < 0 || in_stride % 8 || in_stride > kMaxStride || out_stride < 0 || out_stride % 8 ||
        out_stride > kMaxStride || !aligned(in, 16) || !aligned(out, 16) || !aligned(weight, 16))
        return record_failure(OSCAR_ERR_INVALID_ARG,
                              "%s, %s_out and the weights must be 16-byte aligned, the strides multiples of 8 up to 2^31 "
                              "(are %lld and %lld)", name, name, (long long)in_stride, (long long)out_stride);
    if (out_stride < width)
        return record_failure(OSCAR_ERR_INVALID_ARG, "%s_out's rows of %d elements overlap (stride %lld)", name, width,
                              (long long)out_stride);
    return OSCAR_OK;
}

// Largest batch and row count of an attention call: row and part indices stay in 32 bits.
constexpr int kMaxChunkTokens = 1 << 24;
bool sizes_ok(const oscar_ctx_t* ctx, int batch, int n) {
    return ctx && batch >= 0 && batch <= oscar::kMaxBatch && n >= 0 && n <= kMaxChunkTokens;
}

}  // namespace

extern "C" {

oscar_status oscar_norm_rope(oscar_ctx_t* ctx, const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                             const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, const float* q_weight,
                             const float* k_weight, float eps, const uint64_t* turns, int rot_dim, int layout,
                             float scale, const int32_t* positions, const int32_t* row_start, const int32_t* total_len,
                             int batch, int n, void* stream) {
    if (oscar_status st = oscar::check_context(ctx); st != OSCAR_OK) return st;
    const oscar::Shape& s = ctx->shape;
    if (n < 0 || batch < 0) return record_failure(OSCAR_ERR_INVALID_ARG, "n %d or batch %d negative", n, batch);
    if (batch > oscar::kMaxBatch)
        return record_failure(OSCAR_ERR_UNSUPPORTED, "batch %d above %d", batch, oscar::kMaxBatch);
    if (layout != OSCAR_ROPE_HALF && layout != OSCAR_ROPE_INTERLEAVED)
        return record_failure(OSCAR_ERR_UNSUPPORTED, "layout %d not in {0 (half), 1 (interleaved)}", layout);
    if (rot_dim < 0 || rot_dim > s.d || rot_dim % 8)
        return record_failure(OSCAR_ERR_UNSUPPORTED, "rot_dim %d is not a multiple of 8 in [0, %d]", rot_dim, s.d);
    if (!(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(scale))
        return record_failure(OSCAR_ERR_INVALID_ARG, "eps %g is not finite and >= 0, or scale %g not finite", eps, scale);
    if (n == 0 || (!q && !k && !q_out && !k_out)) return OSCAR_OK;
    if (rot_dim > 0 && !turns) return record_failure(OSCAR_ERR_INVALID_ARG, "turns is NULL");
    if (!positions && (!row_start || (batch > 0 && !total_len)))
        return record_failure(OSCAR_ERR_INVALID_ARG, "positions, or row_start and total_len, must be given");
    const int q_width = s.h_q * s.d, k_width = s.h_kv * s.d;
    oscar_status st = check_rows("q", q, q_stride, q_out, q_out_stride, q_weight, q_width);
    if (st == OSCAR_OK) st = check_rows("k", k, k_stride, k_out, k_out_stride, k_weight, k_width);
    if (st != OSCAR_OK) return st;
    if (!aligned(turns, 8)) return record_failure(OSCAR_ERR_INVALID_ARG, "turns is not 8-byte aligned");
    // in place means the very rows: another head's warp may still have to read any other element
    const Rows qi{q, q_stride, q ? q_width : 0}, qo{q_out, q_out_stride, q ? q_width : 0};
    const Rows ki{k, k_stride, k ? k_width : 0}, ko{k_out, k_out_stride, k ? k_width : 0};
    const bool q_same = q == q_out && (n == 1 || q_stride == q_out_stride);
    const bool k_same = k == k_out && (n == 1 || k_stride == k_out_stride);
    if ((!q_same && share(qo, qi, n)) || (!k_same && share(ko, ki, n)) || share(qo, ki, n) || share(ko, qi, n) ||
        share(qo, ko, n))
        return record_failure(OSCAR_ERR_INVALID_ARG, "outputs overlap each other or other rows than their own input's");
    if (oscar::injected_fault("launch"))
        return record_failure(OSCAR_ERR_CUDA, "injected launch failure (OSCAR_FAULT=launch)");
    oscar::RopeArgs a{};
    a.q = {static_cast<const uint16_t*>(q), q_stride, static_cast<uint16_t*>(q_out), q_out_stride, q_weight, q ? s.h_q : 0};
    a.k = {static_cast<const uint16_t*>(k), k_stride, static_cast<uint16_t*>(k_out), k_out_stride, k_weight, k ? s.h_kv : 0};
    a.eps = eps;
    a.turns = turns; a.rot = rot_dim; a.interleaved = layout == OSCAR_ROPE_INTERLEAVED; a.scale = scale;
    a.positions = positions; a.row_start = row_start; a.total_len = total_len;
    a.batch = batch; a.n = n;
    oscar::ProfScope ps(&ctx->prof, OSCAR_KERNEL_ROPE, static_cast<cudaStream_t>(stream));
    return cuda_status(oscar::launch_norm_rope(a, s.d, ctx->num_sms, static_cast<cudaStream_t>(stream)),
                       "norm and rotation launch");
}

size_t oscar_extend_bf16_workspace_size(const oscar_ctx_t* ctx, int batch, int n) {
    if (!sizes_ok(ctx, batch, n) || batch == 0 || n == 0) return 0;
    return oscar::plan_chunk(ctx->shape, ctx->num_sms, batch, n).total;
}

oscar_status oscar_extend_bf16(oscar_ctx_t* ctx, const void* q, int64_t q_stride, const void* bf16_pool,
                               int64_t bf16_pool_pages, const int32_t* tables, int table_stride,
                               const int32_t* row_start, const int32_t* total_len, int batch, int n, void* out,
                               void* workspace, size_t workspace_bytes, void* stream) {
    if (oscar_status st = oscar::check_context(ctx); st != OSCAR_OK) return st;
    const oscar::Shape& s = ctx->shape;
    if (n < 0 || batch < 0 || table_stride < 0)
        return record_failure(OSCAR_ERR_INVALID_ARG, "n %d, batch %d or table_stride %d negative", n, batch, table_stride);
    if (!sizes_ok(ctx, batch, n) || table_stride > oscar::kMaxPagedLen / oscar::kPage)
        return record_failure(OSCAR_ERR_UNSUPPORTED, "batch %d above %d, n %d above %d or table_stride %d above %d", batch,
                              oscar::kMaxBatch, n, kMaxChunkTokens, table_stride, oscar::kMaxPagedLen / oscar::kPage);
    if (n == 0 || batch == 0) return OSCAR_OK;
    if (!q || !out || !row_start || !total_len) return record_failure(OSCAR_ERR_INVALID_ARG, "device pointer is NULL");
    if (!bf16_pool || bf16_pool_pages <= 0 || (table_stride > 0 && !tables))
        return record_failure(OSCAR_ERR_INVALID_ARG, "BF16 pool/tables missing");
    if (bf16_pool_pages > 0x7ffffff0LL / (2 * s.h_kv))
        return record_failure(OSCAR_ERR_UNSUPPORTED, "bf16_pool_pages %lld above %lld", (long long)bf16_pool_pages,
                              0x7ffffff0LL / (2 * s.h_kv));
    const int width = s.h_q * s.d;
    if (q_stride < 0 || q_stride % 8 || q_stride > (int64_t)1 << 31 || !aligned(q, 16) || !aligned(bf16_pool, 32) ||
        !aligned(out, 32))
        return record_failure(OSCAR_ERR_INVALID_ARG,
                              "q must be 16-byte aligned, the pool and out 32-byte, q_stride a multiple of 8 up to 2^31 (is %lld)",
                              (long long)q_stride);
    if (share({q, q_stride, width}, {out, width, width}, n))
        return record_failure(OSCAR_ERR_INVALID_ARG, "out overlaps q");
    const oscar::ChunkPlan plan = oscar::plan_chunk(s, ctx->num_sms, batch, n);
    if (!workspace || workspace_bytes < plan.total)
        return record_failure(OSCAR_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, plan.total);
    if (!aligned(workspace, 256)) return record_failure(OSCAR_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    if (oscar::injected_fault("launch"))
        return record_failure(OSCAR_ERR_CUDA, "injected launch failure (OSCAR_FAULT=launch)");
    oscar::ChunkArgs a{};
    a.q = static_cast<const uint16_t*>(q); a.q_stride = q_stride;
    a.pool = static_cast<const uint16_t*>(bf16_pool); a.pages = bf16_pool_pages;
    a.tables = tables; a.stride = table_stride;
    a.row_start = row_start; a.total_len = total_len;
    a.out = static_cast<uint16_t*>(out);
    a.batch = batch; a.n = n; a.h_kv = s.h_kv; a.g = s.h_q / s.h_kv; a.d = s.d;
    a.scale_log2 = (float)(s.sm_scale * 1.4426950408889634073599);
    a.debug = s.debug; a.dbg = ctx->dbg;
    a.lost_loads = oscar::injected_fault("wait");
    a.wait_ticks = a.lost_loads ? oscar::kLostWait : oscar::kChunkWait;
    oscar::ProfScope ps(&ctx->prof, OSCAR_KERNEL_EXTEND, static_cast<cudaStream_t>(stream));
    return cuda_status(oscar::launch_chunk(a, plan, workspace, s.d, ctx->num_sms, static_cast<cudaStream_t>(stream)),
                       "chunk attention launch");
}

}  // extern "C"
