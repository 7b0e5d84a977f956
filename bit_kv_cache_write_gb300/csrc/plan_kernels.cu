// Block tables and slot maps from request lengths (oscar_plan_append).
//
// With s_b tokens cached and n_b to append, request b's rows are [r_b, r_b + n_b) with r the exclusive sum
// of n, and it needs ceil((s_b + n_b) / 16) - ceil(s_b / 16) new pages, taken from the free list behind the
// pages of the requests before it (an inclusive sum P_b decides whether they are there). Row r_b + i goes to
// slot page * 16 + (s_b + i) % 16 of logical page (s_b + i) / 16.
//
// One cluster. Every CTA scans all requests (two 64-bit sums), 1,024 at a time, and writes its share of the
// chunk's table entries and slots; a page id is read from the free list, so no CTA reads what another one
// writes. The free head may be the word that the new head goes to, so the last barrier stands between every
// CTA's read of it and the write.
#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Inclusive sums of two values over the CTA; returns the totals too.
__device__ void scan2(long long& a, long long& b, long long& total_a, long long& total_b, long long (*warp_sum)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(~0u, a, o), y = __shfl_up_sync(~0u, b, o);
        if (lane >= o) { a += x; b += y; }
    }
    __syncthreads();                             // the sums of the last chunk have been read
    if (lane == 31) { warp_sum[warp][0] = a; warp_sum[warp][1] = b; }
    __syncthreads();
    long long before_a = 0, before_b = 0;
    total_a = total_b = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) { before_a = total_a; before_b = total_b; }
        total_a += warp_sum[w][0];
        total_b += warp_sum[w][1];
    }
    a += before_a;
    b += before_b;
}

// First i in [0, n) with key < v[i], for ascending v; n if none.
__device__ __forceinline__ int upper(const long long* v, int n, long long key) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] > key) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
    __shared__ long long warp_sum[kPlanThreads / 32][2];
    __shared__ long long row_end[kPlanThreads];      // rows up to and with request i of the chunk
    __shared__ long long page_end[kPlanThreads];     // its pages likewise
    __shared__ int cached[kPlanThreads];             // tokens cached; -1: request rejected
    __shared__ int rejected, first_rejected;
    const int tid = threadIdx.x;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int share = rank * kPlanThreads + tid, shares = ranks * kPlanThreads;
    if (tid == 0) { rejected = 0; first_rejected = INT_MAX; }
    grid_wait();
    const long long head = *reinterpret_cast<const volatile int32_t*>(a.free_head);
    const long long avail = head >= 0 && head < a.n_free ? a.n_free - head : 0;
    long long rows = 0, pages = 0, taken = 0;        // sums over the chunks so far; pages that were handed out
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int b = b0 + tid, count = min(kPlanThreads, a.batch - b0);
        const int s = b < a.batch ? a.seq_len[b] : 0, n = b < a.batch ? a.new_len[b] : 0;
        long long r = n > 0 ? n : 0, p = 0, total_r, total_p;
        bool ok = s >= 0 && n >= 0 && (long long)s + n <= (long long)kPage * a.stride;
        const int old = ok ? (s + kPage - 1) / kPage : 0;
        const int need = ok ? (int)(((long long)s + n + kPage - 1) / kPage) - old : 0;
        // A request whose rows pass the slot map takes no pages, but that is known only after the sum of rows.
        long long unused = 0, total_unused;
        scan2(r, unused, total_r, total_unused, warp_sum);
        ok = ok && rows + r <= a.slot_cap;
        p = ok ? need : 0;
        long long mine = p;
        unused = 0;
        scan2(p, unused, total_p, total_unused, warp_sum);
        ok = ok && (mine == 0 || pages + p <= avail);
        const long long got = ok ? mine : 0;
        long long g = got, total_g;
        unused = 0;
        scan2(g, unused, total_g, total_unused, warp_sum);
        row_end[tid] = rows + r;
        page_end[tid] = taken + g;
        cached[tid] = ok ? s : -1;
        if (b < a.batch) {
            if (!ok) { atomicAdd(&rejected, 1); atomicMin(&first_rejected, b); }
            if (b % ranks == rank) {
                a.total_len[b] = ok ? s + n : s;
                a.row_start[b] = (int32_t)min(rows + r - (n > 0 ? n : 0), (long long)INT_MAX);
            }
        }
        __syncthreads();
        // new table entries
        for (long long j = taken + share; j < taken + total_g; j += shares) {
            const int i = upper(page_end, count, j);
            const long long before = i ? page_end[i - 1] : taken;
            a.tables[(long long)(b0 + i) * a.stride + (cached[i] + kPage - 1) / kPage + (j - before)] =
                a.free_pages[head + j];
        }
        // slots
        const long long end = min(rows + total_r, (long long)a.slot_cap);
        for (long long t = rows + share; t < end; t += shares) {
            const int i = upper(row_end, count, t);
            int64_t slot = -1;
            if (cached[i] >= 0) {
                const int pos = cached[i] + (int)(t - (i ? row_end[i - 1] : rows));
                const int page = pos / kPage, first_new = (cached[i] + kPage - 1) / kPage;
                const int id = page < first_new ? a.tables[(long long)(b0 + i) * a.stride + page]
                                                : a.free_pages[head + (i ? page_end[i - 1] : taken) + page - first_new];
                slot = (int64_t)id * kPage + pos % kPage;
            }
            a.slots[t] = slot;
        }
        rows += total_r;
        pages += total_p;
        taken += total_g;
        __syncthreads();                             // the chunk's arrays have been read
    }
    for (long long t = min(rows, (long long)a.slot_cap) + share; t < a.slot_cap; t += shares) a.slots[t] = -1;
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    if (rank == 0 && tid == 0) {
        a.row_start[a.batch] = (int32_t)min(rows, (long long)INT_MAX);
        a.state[0] = (int32_t)(head + taken);
        a.state[1] = (int32_t)min(rows, (long long)INT_MAX);
        a.state[2] = rejected;
        a.state[3] = rejected ? first_rejected : -1;
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st) {
    return launch_dependent(plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, 1, a);
}

}  // namespace oscar
