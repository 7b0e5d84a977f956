// Block tables and slot maps from request lengths (oscar_plan_append).
//
// With s_b tokens cached and n_b to append, request b's rows are [r_b, r_b + n_b) with r the exclusive sum
// of n, and it needs ceil((s_b + n_b) / 16) - ceil(s_b / 16) new pages, taken from the free list behind the
// pages of the requests before it (an inclusive sum P_b decides whether they are there). Row r_b + i goes to
// slot page * 16 + (s_b + i) % 16 of logical page (s_b + i) / 16.
//
// One cluster. Every CTA scans all requests, 512 or 2,048 at a time (one pass of two sums; two more only
// where a request does not fit), and writes its share of the chunk's table entries and slots; a page id is
// read from the free list, so no CTA reads what another one writes. The free head may be the word that the
// new head goes to, so the last barrier stands between every CTA's read of it and the write.
//
// Nothing here is large: the time is a chain of dependent loads (lengths, sums, page ids), 3.7 us for 64 single
// tokens; 94,000 tokens of 96 requests take 8.5 us, their searches and writes on 16 SMs. The kernel does not let
// its successor start early: page ids and slots may be read ahead by the one after that.
#include <climits>

#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanMaxCluster = 16;
constexpr int kPlanTokens = 4;                       // slots that a thread looks up at once

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

// Inclusive sums of two values over the CTA, and their totals. Consecutive calls alternate `sums`.
__device__ void scan2(long long& a, long long& b, long long& total_a, long long& total_b, long long (*sums)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(~0u, a, o), y = __shfl_up_sync(~0u, b, o);
        if (lane >= o) { a += x; b += y; }
    }
    if (lane == 31) { sums[warp][0] = a; sums[warp][1] = b; }
    __syncthreads();
    long long wa = lane < kPlanWarps ? sums[lane][0] : 0, wb = lane < kPlanWarps ? sums[lane][1] : 0;
#pragma unroll
    for (int o = 1; o < kPlanWarps; o <<= 1) {
        const long long x = __shfl_up_sync(~0u, wa, o), y = __shfl_up_sync(~0u, wb, o);
        if (lane >= o) { wa += x; wb += y; }
    }
    total_a = __shfl_sync(~0u, wa, kPlanWarps - 1);
    total_b = __shfl_sync(~0u, wb, kPlanWarps - 1);
    const long long before_a = __shfl_sync(~0u, wa, warp ? warp - 1 : 0), before_b = __shfl_sync(~0u, wb, warp ? warp - 1 : 0);
    if (warp) { a += before_a; b += before_b; }
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

// PER: requests that a thread adds up. BULK: a thread writes several slots in a row (one search), else one of each
// stride's (a shorter program).
template <int PER, bool BULK>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
    constexpr int kPlanPer = PER, kPlanChunk = kPlanThreads * PER;
    __shared__ long long sums[2][kPlanWarps][2];
    __shared__ long long row_end[kPlanChunk];        // rows up to and with request i of the chunk
    __shared__ long long page_end[kPlanChunk];       // its pages likewise
    __shared__ int cached[kPlanChunk];               // tokens cached; -1: request rejected
    __shared__ int rejected, first_rejected;
    const int tid = threadIdx.x;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int share = rank * kPlanThreads + tid, shares = ranks * kPlanThreads;
    if (tid == 0) { rejected = 0; first_rejected = INT_MAX; }
    grid_wait();
    const long long head = *reinterpret_cast<const volatile int32_t*>(a.free_head);
    const long long avail = head >= 0 && head < a.n_free ? a.n_free - head : 0;
    long long rows = 0, wanted = 0, taken = 0;       // over the chunks so far: rows, pages needed, handed out
    for (int b0 = 0; b0 < a.batch; b0 += kPlanChunk) {
        const int count = min(kPlanChunk, a.batch - b0), i0 = tid * kPlanPer;
        int s[kPlanPer], n[kPlanPer];
#pragma unroll
        for (int k = 0; k < kPlanPer; ++k) {
            const bool inside = i0 + k < count;
            s[k] = inside ? a.seq_len[b0 + i0 + k] : 0;
            n[k] = inside ? a.new_len[b0 + i0 + k] : 0;
        }
        bool ok[kPlanPer];
        long long need[kPlanPer], r = 0, p = 0, total_r, total_p;
#pragma unroll
        for (int k = 0; k < kPlanPer; ++k) {
            ok[k] = s[k] >= 0 && n[k] >= 0 && (long long)s[k] + n[k] <= (long long)kPage * a.stride;
            need[k] = ok[k] ? ((long long)s[k] + n[k] + kPage - 1) / kPage - (s[k] + kPage - 1) / kPage : 0;
            r += max(n[k], 0);
            p += need[k];
        }
        const long long own_r = r, own_p = p;
        scan2(r, p, total_r, total_p, sums[0]);
        long long before_r = rows + r - own_r, before_g = taken + p - own_p, total_g = total_p;
        if (rows + total_r > a.slot_cap || wanted + total_p > avail) {
            // Some request passes the slot map or the free list. One that passes the map needs no page.
            long long end = before_r, unused = 0, t, q = 0;
#pragma unroll
            for (int k = 0; k < kPlanPer; ++k) {
                end += max(n[k], 0);
                ok[k] = ok[k] && end <= a.slot_cap;
                if (!ok[k]) need[k] = 0;
                q += need[k];
            }
            const long long own_q = q;
            scan2(q, unused, total_p, t, sums[1]);
            long long upto = wanted + q - own_q, g = 0;
#pragma unroll
            for (int k = 0; k < kPlanPer; ++k) {
                upto += need[k];
                ok[k] = ok[k] && (need[k] == 0 || upto <= avail);
                if (!ok[k]) need[k] = 0;
                g += need[k];
            }
            const long long own_g = g;
            unused = 0;
            scan2(g, unused, total_g, t, sums[0]);
            before_g = taken + g - own_g;
        }
#pragma unroll
        for (int k = 0; k < kPlanPer; ++k) {
            const int b = b0 + i0 + k;
            if (b < a.batch) {
                if (!ok[k]) { atomicAdd(&rejected, 1); atomicMin(&first_rejected, b); }
                if (b % ranks == rank) {
                    a.total_len[b] = ok[k] ? s[k] + n[k] : s[k];
                    a.row_start[b] = (int32_t)min(before_r, (long long)INT_MAX);
                }
            }
            before_r += max(n[k], 0);
            before_g += need[k];
            row_end[i0 + k] = before_r;
            page_end[i0 + k] = before_g;
            cached[i0 + k] = ok[k] ? s[k] : -1;
        }
        __syncthreads();
        // new table entries
        for (long long j = taken + share; j < taken + total_g; j += shares) {
            const int i = upper(page_end, count, j);
            const long long before = i ? page_end[i - 1] : taken;
            a.tables[(long long)(b0 + i) * a.stride + (cached[i] + kPage - 1) / kPage + (j - before)] =
                a.free_pages[head + j];
        }
        // slots, kPlanTokens a thread at once, whose page ids are asked for together
        const long long end = min(rows + total_r, (long long)a.slot_cap);
        const long long next = BULK ? 1 : shares;    // from one of a thread's slots to the next
        for (long long t0 = rows + (BULK ? (long long)kPlanTokens * share : share); t0 < end;
             t0 += (long long)kPlanTokens * shares) {
            const int32_t* from[kPlanTokens];
            int in_page[kPlanTokens], i = 0;
#pragma unroll
            for (int k = 0; k < kPlanTokens; ++k) {
                const long long t = t0 + k * next;
                from[k] = nullptr;
                if (t >= end) continue;
                if (!BULK || k == 0) i = upper(row_end, count, t);
                else while (t >= row_end[i]) ++i;
                if (cached[i] < 0) continue;
                const int pos = cached[i] + (int)(t - (i ? row_end[i - 1] : rows));
                const int page = pos / kPage, first_new = (cached[i] + kPage - 1) / kPage;
                in_page[k] = pos % kPage;
                from[k] = page < first_new ? a.tables + (long long)(b0 + i) * a.stride + page
                                           : a.free_pages + head + (i ? page_end[i - 1] : taken) + page - first_new;
            }
            int id[kPlanTokens];
#pragma unroll
            for (int k = 0; k < kPlanTokens; ++k) id[k] = from[k] ? *from[k] : 0;
#pragma unroll
            for (int k = 0; k < kPlanTokens; ++k)
                if (t0 + k * next < end) a.slots[t0 + k * next] = from[k] ? (int64_t)id[k] * kPage + in_page[k] : -1;
        }
        rows += total_r;
        wanted += total_p;
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
    // as many CTAs as have kPlanTokens slots a thread to write
    int cluster = 1;
    while (cluster < kPlanMaxCluster && (long long)cluster * kPlanThreads * kPlanTokens < a.slot_cap) cluster *= 2;
    // 64 single tokens 3.7 us, in bulk 4.7; 64 x 512 slots 6.0 and 5.3; 64 x 2,000 12.1 and 9.7. Four requests a thread:
    // 512 single tokens 6.0 us against 4.3 with one, 1,024 6.2 and 7.2, 2,048 8.0 and 13.3.
    const auto kernel = a.batch > 2 * kPlanThreads ? plan_kernel<4, true>
                        : a.slot_cap > 65536       ? plan_kernel<1, true>
                                                   : plan_kernel<1, false>;
    if (cluster > 8) {
        cudaError_t e = allow_large_clusters<plan_kernel<4, true>>();
        if (e == cudaSuccess) e = allow_large_clusters<plan_kernel<1, true>>();
        if (e == cudaSuccess) e = allow_large_clusters<plan_kernel<1, false>>();
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kernel, dim3(cluster), dim3(kPlanThreads), 0, st, cluster, a);
}

}  // namespace oscar
