// The pages that a sparse decode reads (oscar_decode_bf16_sparse): a cheap score per page, and the largest.
//
// Score of page p for KV head h: max over the head's g query heads of 2^e S with
// S = sum_c max(u_c lo_c, u_c hi_c), u the query's integer codes in the steps of the key bounds [lo, hi]. It
// bounds the logits of the page's keys (up to the rounding of u and to clipped codes). S is an integer below
// 2^23 and the scale a power of two, so the score is exact in fp32 and the choice does not depend on the
// order of any sum. sum max(u lo, u hi) = sum min(u, 0) lo + max(u, 0) hi, one integer product over 2 d bytes:
// mma.sync m16n8k32 with 16 pages as rows and the heads as columns, operands straight from memory (the
// order of the contraction is free, so a lane's 16 bytes serve two steps).
//
// One cluster per (sequence, KV head). Its warps score the pages, 16 at a time, into the first CTA's shared
// memory; that CTA finds the top-th largest key by counting (2,048 bins a pass, narrowed to the keys'
// range first) and writes the list in ascending order.
#include <cooperative_groups.h>

#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;
constexpr int kSmemKeys = 16384;                 // candidates whose keys fit in shared memory (64 KB); else the workspace

struct Window { int pages, sink, first; };       // pages of the sequence; kept: p < sink or p >= first
__device__ __forceinline__ Window window_of(const SelectArgs& a, int len) {
    Window w;
    w.pages = (len + kPage - 1) / kPage;
    w.sink = min(w.pages, (a.sink + kPage - 1) / kPage);
    w.first = min(w.pages, max(len - a.recent, 0) / kPage);
    return w;
}

// Keys in the order of the scores (none is NaN).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);        // -0 to +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Integer codes of the g query heads of KV head h: min(u, 0) for the lower bounds in bytes [0, D), max(u, 0)
// for the upper ones behind them, zeros for the heads that are not there. One warp a head.
template <int D, int T>
__device__ void query_codes(const SelectArgs& a, int b, int h, int8_t (*codes)[2 * D + 16], int* exponent) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < 8; i += T / 32) {
        float x[D / 32] = {}, top = 0.0f;
        if (i < a.g) {
            const uint16_t* q = a.q + b * a.q_stride + (int64_t)(h * a.g + i) * D;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const int c = lane + 32 * j, step = max(-100, min(100, (int)a.steps[h * D + c]));
                x[j] = __uint_as_float((uint32_t)q[c] << 16) * __int_as_float((127 + step) << 23);
                if (!isfinite(x[j])) x[j] = 0.0f;
                top = fmaxf(top, fabsf(x[j]));
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        // top = f 2^x with f in [1/2, 1): codes in units of 2^(x - 7)
        const int e = min((int)(__float_as_uint(top) >> 23) - 126 - 7, 60);
        const bool none = top < 0x1p-60f;
        const float inv = none ? 0.0f : __int_as_float((127 - e) << 23);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const int u = __float2int_rn(fminf(fmaxf(x[j] * inv, -127.0f), 127.0f));
            codes[i][lane + 32 * j] = (int8_t)min(u, 0);
            codes[i][D + lane + 32 * j] = (int8_t)max(u, 0);
        }
        if (lane == 0) exponent[i] = none ? 0 : e;
    }
}

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scores of the candidates (logical pages w.sink + i) of one (sequence, KV head) as ordered keys.
template <int D, int T>
__device__ void score_pages(const SelectArgs& a, int b, int h, const Window& w, uint32_t* keys, int warp, int warps,
                            int8_t (*codes)[2 * D + 16], int* exponent) {
    constexpr int kBlocks = 2 * D / 64;                  // 64-byte column blocks of a page's bounds
    const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
    const int32_t* table = a.tables + (int64_t)b * a.stride + w.sink;
    const int cand = w.first - w.sink;
    uint4 x[2][kBlocks];                                 // pages gid and gid + 8 of the tile
    int id[2];                                           // their page ids, one tile ahead of the bounds
    bool real[2];
    auto load_ids = [&](int i0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = i0 + gid + 8 * r;
            id[r] = i < cand ? table[i] : 0;
        }
    };
    auto load = [&]() {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            real[r] = id[r] >= 0 && id[r] < a.pages;
            if (!real[r] && a.debug && t == 0) record_error(&a.dbg->kind, &a.dbg->index, 2, id[r]);
            const int8_t* src = a.bounds + ((int64_t)(real[r] ? id[r] : 0) * a.h_kv + h) * (2 * D) + 16 * t;
#pragma unroll
            for (int j = 0; j < kBlocks; ++j) x[r][j] = ldg_stream(src + 64 * j);
        }
    };
    const int step = 16 * warps;
    int i0 = 16 * warp;
    load_ids(i0);
    load();                                              // on their way while the codes are made
    load_ids(i0 + step);
    query_codes<D, T>(a, b, h, codes, exponent);
    __syncthreads();
    // the heads of this lane's two result columns; columns without a head repeat head 0
    const float s0 = __int_as_float((127 + exponent[2 * t]) << 23), s1 = __int_as_float((127 + exponent[2 * t + 1]) << 23);
    const bool h0 = 2 * t < a.g, h1 = 2 * t + 1 < a.g;
    for (; i0 < cand; i0 += step) {
        int c[4] = {};
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const uint4 u = *reinterpret_cast<const uint4*>(&codes[gid][64 * j + 16 * t]);
            mma_s8(c, x[0][j].x, x[1][j].x, x[0][j].y, x[1][j].y, u.x, u.y);
            mma_s8(c, x[0][j].z, x[1][j].z, x[0][j].w, x[1][j].w, u.z, u.w);
        }
        const bool was[2] = {real[0], real[1]};
        if (i0 + step < cand) {
            load();
            load_ids(i0 + 2 * step);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float best = h0 ? (float)c[2 * r] * s0 : -INFINITY;
            if (h1) best = fmaxf(best, (float)c[2 * r + 1] * s1);
            best = fmaxf(best, __shfl_xor_sync(~0u, best, 1));
            best = fmaxf(best, __shfl_xor_sync(~0u, best, 2));
            const int i = i0 + gid + 8 * r;
            if (t == 0 && i < cand) keys[i] = was[r] ? ordered(best) : 0u;
        }
    }
}

struct SelectShared {
    int hist[kBins];
    int warp_sum[32], warp_ties[32];
    uint32_t warp_lo[32], warp_hi[32];
    int bin, left, count;
};

// The take largest of n keys (0 < take < n), ties to the lowest index: keys above base + mask, and the first
// `left` of those within [base, base + mask].
template <int T>
__device__ void find_threshold(const uint32_t* keys, int n, int take, SelectShared& s, uint32_t& base, uint32_t& mask,
                               int& left) {
    constexpr int kWarps = T / 32, kBinsPerThread = kBins / T;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t lo = ~0u, hi = 0;
    for (int i = tid; i < n; i += T) {
        const uint32_t k = keys[i];
        lo = min(lo, k);
        hi = max(hi, k);
    }
    lo = __reduce_min_sync(~0u, lo);
    hi = __reduce_max_sync(~0u, hi);
    if (lane == 0) { s.warp_lo[warp] = lo; s.warp_hi[warp] = hi; }
    __syncthreads();
    lo = __reduce_min_sync(~0u, s.warp_lo[lane % kWarps]);
    hi = __reduce_max_sync(~0u, s.warp_hi[lane % kWarps]);
    base = lo;
    left = take;
    int bits = 32 - __clz(hi - lo);
    mask = bits == 32 ? ~0u : (1u << bits) - 1;
    while (bits > 0) {
        const int shift = max(bits - 11, 0);
        for (int i = tid; i < kBins; i += T) s.hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += T) {
            const uint32_t d = keys[i] - base;
            if (d <= mask) atomicAdd(&s.hist[d >> shift], 1);
        }
        __syncthreads();
        // thread tid owns bins kBins - 1 - kBinsPerThread tid and below, so that its prefix counts larger keys
        int own = 0;
#pragma unroll
        for (int j = 0; j < kBinsPerThread; ++j) own += s.hist[kBins - 1 - kBinsPerThread * tid - j];
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) s.warp_sum[warp] = sum;
        __syncthreads();
        const int above_warp = __reduce_add_sync(~0u, lane < warp ? s.warp_sum[lane] : 0);
        int above = sum - own + above_warp;
        if (above < left && left <= above + own) {       // one thread
            int bin = kBins - 1 - kBinsPerThread * tid;
            while (above + s.hist[bin] < left) above += s.hist[bin--];
            s.bin = bin;
            s.left = left - above;
            s.count = s.hist[bin];
        }
        __syncthreads();
        base += (uint32_t)s.bin << shift;
        mask = (1u << shift) - 1;
        left = s.left;
        bits = s.count == left ? 0 : shift;              // all keys of the bin are taken: no need to look closer
        __syncthreads();
    }
}

template <int D, int T>
__global__ void __launch_bounds__(T, 1024 / T) select_kernel(SelectArgs a, int smem_keys) {
    __shared__ __align__(16) int8_t codes[8][2 * D + 16];     // padded: eight heads' words in eight bank groups
    __shared__ int exponent[8];
    __shared__ SelectShared s;
    extern __shared__ uint32_t key_store[];
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int unit = blockIdx.x / ranks, b = unit / a.h_kv, h = unit % a.h_kv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cluster.sync();                                      // the first CTA runs: its shared memory may be written
    grid_wait();
    grid_release();
    const int len = checked_len(a.seq_len[b], a.max_len, a.debug && tid == 0 && rank == 0, a.dbg);
    const Window w = window_of(a, len);
    const int cand = max(w.first - w.sink, 0), take = min(a.top, cand);
    const bool choose = take > 0 && take < cand;
    uint32_t* keys = cand <= smem_keys ? cluster.map_shared_rank(key_store, 0)
                                       : a.keys + (int64_t)unit * a.max_pages;
    if (choose)
        score_pages<D, T>(a, b, h, w, keys, rank + ranks * warp, ranks * (T / 32), codes, exponent);
    cluster.sync();
    if (rank != 0) return;
    if (cand <= smem_keys) keys = key_store;

    int32_t* list = a.chosen + (int64_t)unit * a.cap;
    const int recent = w.pages - max(w.first, w.sink), total = w.sink + take + recent;
    for (int i = tid; i < w.sink; i += T) list[i] = i;
    for (int i = tid; i < recent; i += T) list[w.sink + take + i] = w.pages - recent + i;
    for (int i = total + tid; i < a.cap; i += T) list[i] = -1;
    if (tid == 0) a.n_chosen[unit] = total;
    list += w.sink;
    if (!choose) {
        for (int i = tid; i < take; i += T) list[i] = w.sink + i;
        return;
    }
    uint32_t base, mask;
    int left;
    find_threshold<T>(keys, cand, take, s, base, mask, left);
    // Each warp lists its share of the candidates behind those of the warps before it.
    const int share = (cand + T - 1) / T * 32;
    const int i0 = min(cand, warp * share), i1 = min(cand, i0 + share);
    int above = 0, ties = 0;
    for (int i = i0 + lane; i < i1; i += 32) {
        const uint32_t k = keys[i];
        above += k > base && k - base > mask;
        ties += k - base <= mask;
    }
    above = __reduce_add_sync(~0u, above);
    ties = __reduce_add_sync(~0u, ties);
    if (lane == 0) { s.warp_sum[warp] = above; s.warp_ties[warp] = ties; }
    __syncthreads();
    int at = __reduce_add_sync(~0u, lane < warp ? s.warp_sum[lane] : 0);
    int tied = __reduce_add_sync(~0u, lane < warp ? s.warp_ties[lane] : 0);
    at += min(tied, left);
    for (int i = i0; i < i1; i += 32) {
        const uint32_t k = i + lane < i1 ? keys[i + lane] : 0u;
        const bool in_range = i + lane < i1;
        const bool tie = in_range && k - base <= mask;
        const uint32_t before = (1u << lane) - 1, tie_mask = __ballot_sync(~0u, tie);
        const bool in = in_range && (tie ? tied + __popc(tie_mask & before) < left : k > base);
        const uint32_t in_mask = __ballot_sync(~0u, in);
        if (in) list[at + __popc(in_mask & before)] = w.sink + i + lane;
        at += __popc(in_mask);
        tied += __popc(tie_mask);
    }
}

template <int D, int T>
cudaError_t launch(const SelectArgs& a, int num_sms, cudaStream_t st) {
    const long long units = (long long)a.batch * a.h_kv;
    // CTAs of a cluster: while all clusters fit on the card at once (1,024 threads an SM), with a tile of 16
    // pages for every warp.
    int cluster = 1;
    while (cluster < kMaxCluster && 2 * cluster * units <= num_sms * (1024 / T) && 2 * cluster * (T / 2) <= a.max_pages)
        cluster *= 2;
    if (cluster * units > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int smem_keys = a.max_pages < kSmemKeys ? a.max_pages : kSmemKeys;
    cudaError_t e = smem_opt_in<select_kernel<D, T>>(kSmemKeys * sizeof(uint32_t));
    if (e == cudaSuccess) e = allow_large_clusters<select_kernel<D, T>>();
    if (e != cudaSuccess) return e;
    return launch_dependent(select_kernel<D, T>, dim3((unsigned)(units * cluster)), dim3(T),
                            smem_keys * sizeof(uint32_t), st, cluster, a, smem_keys);
}

template <int D>
cudaError_t launch_threads(const SelectArgs& a, int num_sms, cudaStream_t st) {
    const long long units = (long long)a.batch * a.h_kv;
    if (units <= num_sms && a.max_pages > 512) return launch<D, 1024>(a, num_sms, st);
    if (units <= 2 * num_sms && a.max_pages > 256) return launch<D, 512>(a, num_sms, st);
    return launch<D, 256>(a, num_sms, st);
}

}  // namespace

size_t select_workspace_bytes(const Shape& s, int batch, int max_pages) {
    if (max_pages <= kSmemKeys) return 0;
    return ((size_t)batch * s.h_kv * max_pages * sizeof(uint32_t) + 255) / 256 * 256;
}

cudaError_t launch_select(const SelectArgs& a, int d, int num_sms, cudaStream_t st) {
    return d == 128 ? launch_threads<128>(a, num_sms, st) : launch_threads<64>(a, num_sms, st);
}

}  // namespace oscar
