// The host side of the calls on chunks of new tokens (chunk_api.cu) with its launches replaced by counters, so that what
// the calls refuse can be tested without a GPU. Built by test_chunk_host.py together with chunk_api.cu.
#include <cstdarg>
#include <cstdio>

#include "chunk_internal.h"

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

ChunkPlan plan_chunk(const Shape&, int, int batch, int n) {
    ChunkPlan p{};
    p.total = 1024 + (size_t)batch + (size_t)n;
    return p;
}
cudaError_t launch_norm_rope(const RopeArgs&, int, int, cudaStream_t) { return ++g_launches, cudaSuccess; }
cudaError_t launch_chunk(const ChunkArgs&, const ChunkPlan&, void*, int, int, cudaStream_t) { return ++g_launches, cudaSuccess; }

}  // namespace oscar

extern "C" {

OSCAR_API oscar_ctx_t* chunk_host_context(int h_q, int h_kv, int d) {
    oscar_ctx_t* ctx = new oscar_ctx_t();
    ctx->shape.h_q = h_q;
    ctx->shape.h_kv = h_kv;
    ctx->shape.d = d;
    ctx->shape.sm_scale = 1.0;
    ctx->num_sms = 152;
    return ctx;
}
OSCAR_API void chunk_host_free(oscar_ctx_t* ctx) { delete ctx; }
OSCAR_API int chunk_host_launches(void) { return g_launches; }
OSCAR_API const char* chunk_host_message(void) { return g_message; }

}  // extern "C"
