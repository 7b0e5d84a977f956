// The host side of the BF16 paged-cache calls (paged_api.cu) with its launches replaced by counters, so that what the
// calls refuse can be tested without a GPU. Built by test_paged_host.py together with paged_api.cu.
#include <cstdarg>
#include <cstdio>

#include "paged_internal.h"

namespace {
int g_launches;
char g_message[256];
}  // namespace

namespace oscar {

oscar_status record_failure(oscar_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_message, sizeof(g_message), fmt, ap);
    va_end(ap);
    return st;
}
oscar_status check_context(const oscar_ctx* ctx) { return ctx ? OSCAR_OK : OSCAR_ERR_INVALID_ARG; }
bool injected_fault(const char*) { return false; }

AttendPlan plan_attend(const Shape&, int, int, int, bool) {
    AttendPlan p{};
    p.splits = p.pages_per_split = 1;
    return p;
}
size_t attend_workspace_bytes(const Shape&, int, int, int, bool) { return 0; }
size_t select_workspace_bytes(const Shape&, int, int) { return 0; }
int sparse_small_ranks(const Shape&, int, int, int, int) { return 0; }

cudaError_t launch_plan(const PlanArgs&, cudaStream_t) { return ++g_launches, cudaSuccess; }
cudaError_t launch_append(const AppendArgs&, int, int, cudaStream_t) { return ++g_launches, cudaSuccess; }
cudaError_t launch_attend(const AttendArgs&, int, cudaStream_t) { return ++g_launches, cudaSuccess; }
cudaError_t launch_select(const SelectArgs&, int, int, cudaStream_t) { return ++g_launches, cudaSuccess; }
cudaError_t launch_sparse_small(const SelectArgs&, const AttendArgs&, int, int, cudaStream_t) {
    return ++g_launches, cudaSuccess;
}

}  // namespace oscar

extern "C" {

OSCAR_API oscar_ctx_t* paged_host_context(int h_q, int h_kv, int d) {
    oscar_ctx_t* ctx = new oscar_ctx_t();
    ctx->shape.h_q = h_q;
    ctx->shape.h_kv = h_kv;
    ctx->shape.d = d;
    ctx->shape.sink = 64;
    ctx->shape.recent = 256;
    ctx->num_sms = 152;
    return ctx;
}
OSCAR_API void paged_host_free(oscar_ctx_t* ctx) { delete ctx; }
OSCAR_API int paged_host_launches(void) { return g_launches; }
OSCAR_API const char* paged_host_message(void) { return g_message; }

}  // extern "C"
