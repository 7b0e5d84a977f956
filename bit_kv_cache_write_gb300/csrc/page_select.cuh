// The pages that a sparse decode reads (oscar_decode_bf16_sparse): a cheap score per page, and the largest.
//
// Score of page p for KV head h: max over the head's g query heads of 2^e S with
// S = sum_c max(u_c lo_c, u_c hi_c), u the query's integer codes in the steps of the key bounds [lo, hi]. It
// bounds the logits of the page's keys (up to the rounding of u and to clipped codes). S is an integer below
// 2^22 and the scale a power of two, so the score is exact in fp32 and the choice does not depend on the
// order of any sum. sum max(u lo, u hi) = sum min(u, 0) lo + max(u, 0) hi is one product over 2 d bytes.
//
// That product runs on mma.sync m16n8k16 in fp16, 16 pages as rows, the heads as columns: a byte b + 128 with a
// zero above it is the fp16 subnormal (b + 128) 2^-24, so two byte permutations and one exclusive-or turn four
// bounds into operands; products and sums are multiples of 2^-24 below 2^-2, exact in the fp32 accumulator, and
// 128 sum u is taken off at the end. (The integer m16n8k32 takes 65 cycles a warp on sm_103a, this 8: the
// scores of 64 sequences at 32k took 57k cycles with it, its rate.) Operands come straight from memory; the
// contraction's order is free, so a lane's 32 bytes serve eight steps.
//
// One cluster per (sequence, KV head). Its warps score the pages, 16 at a time, into the first CTA's shared
// memory; that CTA finds the top-th largest key by counting (2,048 bins a pass, from the keys' own range)
// and writes the list in ascending order.
//
// 64 sequences at 32k (266 MB of bounds): 54 us, 35 of them streaming at HBM rate, the rest the first loads'
// latency and the search, in which memory idles because every CTA is at the same point.
#pragma once

#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int kBins = 2048;
constexpr int kSelectMaxCluster = 16;
constexpr int kSortedBatch = 64;                 // sequences whose clusters may start with the longest
constexpr int kLongShare = 1536;                 // candidates that make a CTA's share a long one
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

// The query heads of one KV head as the product takes them.
template <int D>
struct QueryCodes {
    // min(u, 0) in [0, D), max(u, 0) in [D, 2 D), zeros for absent heads. 8 of padding behind each 32, rows 16 banks
    // apart: two heads' lanes (four at a time, 32 codes apart) read 32 banks.
    static constexpr int kRow = 2 * D + 8 * (2 * D / 32) + (D == 128 ? 32 : 0);
    static __device__ int at(int c) { return c + 8 * (c >> 5); }
    __half code[8][kRow];
    float scale[8];                      // 2^e
    float offset[8];                     // -128 sum u
};

// One warp a head: its query channels lane, lane + 32, ... and their steps, then their codes.
template <int D>
struct QueryRow {
    uint16_t q[D / 32];
    int8_t step[D / 32];
};

template <int D>
__device__ __forceinline__ QueryRow<D> fetch_query(const SelectArgs& a, int b, int h, int i) {
    const int lane = threadIdx.x & 31;
    const uint16_t* q = a.q + b * a.q_stride + (int64_t)(h * a.g + i) * D;
    QueryRow<D> r;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        r.q[j] = i < a.g ? q[lane + 32 * j] : 0;
        r.step[j] = a.steps[h * D + lane + 32 * j];
    }
    return r;
}

template <int D>
__device__ __forceinline__ void query_codes(const QueryRow<D>& r, int i, QueryCodes<D>& qc) {
    const int lane = threadIdx.x & 31;
    float x[D / 32], top = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const int step = max(-100, min(100, (int)r.step[j]));
        x[j] = __uint_as_float((uint32_t)r.q[j] << 16) * __int_as_float((127 + step) << 23);
        if (!isfinite(x[j])) x[j] = 0.0f;
        top = fmaxf(top, fabsf(x[j]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    // top = f 2^x with f in [1/2, 1): codes in units of 2^(x - 7)
    const int e = min((int)(__float_as_uint(top) >> 23) - 126 - 7, 60);
    const bool none = top < 0x1p-60f;
    const float inv = none ? 0.0f : __int_as_float((127 - e) << 23);
    int sum = 0;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const int u = __float2int_rn(fminf(fmaxf(x[j] * inv, -127.0f), 127.0f));
        qc.code[i][qc.at(lane + 32 * j)] = __int2half_rn(min(u, 0));
        qc.code[i][qc.at(D + lane + 32 * j)] = __int2half_rn(max(u, 0));
        sum += u;
    }
    sum = __reduce_add_sync(~0u, sum);
    if (lane == 0) {
        qc.scale[i] = none ? 1.0f : __int_as_float((127 + e) << 23);
        qc.offset[i] = -128.0f * (float)sum;
    }
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// One step: four bounds of page gid (x) and of page gid + 8 (y) against four codes of the lane's head.
__device__ __forceinline__ void mma_bounds(float (&c)[4], uint32_t x, uint32_t y, uint32_t u0, uint32_t u1) {
    x ^= 0x80808080u;
    y ^= 0x80808080u;
    mma_f16(c, __byte_perm(x, 0, 0x4140), __byte_perm(y, 0, 0x4140), __byte_perm(x, 0, 0x4342), __byte_perm(y, 0, 0x4342),
            u0, u1);
}

// Scores of the candidates (logical pages w.sink + i) of one (sequence, KV head) as ordered keys, and their
// range. `id` holds the page ids of this warp's first tile; `meanwhile` runs while its bounds are on their way and
// ends with the query's codes in place.
template <int D, typename F>
__device__ void score_pages(const SelectArgs& a, int h, const int32_t* table, int cand, uint32_t* keys, uint32_t* range,
                            int warp, int warps, int (&id)[2], const QueryCodes<D>& qc, F meanwhile) {
    constexpr int kBlocks = 2 * D / 64;                  // a lane's 16-byte pieces of a page's bounds
    const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
    uint4 x[2][kBlocks];                                 // pages gid and gid + 8 of the tile
    bool real[2];
    auto load_ids = [&](int i0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = i0 + gid + 8 * r;
            id[r] = i < cand ? table[i] : 0;
        }
    };
    auto load = [&](int i0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int page = id[r];
            const bool inside = i0 + gid + 8 * r < cand;
            real[r] = page >= 0 && page < a.pages;
            if (inside && !real[r] && a.debug && t == 0) record_error(&a.dbg->kind, &a.dbg->index, 2, page);
            const int8_t* src = a.bounds + ((int64_t)(inside && real[r] ? page : 0) * a.h_kv + h) * (2 * D) + 32 * t;
#pragma unroll
            for (int j = 0; j < kBlocks; j += 2) ldg_stream32(x[r][j], x[r][j + 1], src + 64 * j);
        }
    };
    const int step = 16 * warps;
    int i0 = 16 * warp;
    load(i0);
    load_ids(i0 + step);
    meanwhile();
    // the heads of this lane's two result columns
    const float s0 = qc.scale[2 * t], s1 = qc.scale[2 * t + 1], o0 = qc.offset[2 * t], o1 = qc.offset[2 * t + 1];
    const bool h0 = 2 * t < a.g, h1 = 2 * t + 1 < a.g;
    uint32_t least = ~0u, most = 0;
    for (; i0 < cand; i0 += step) {
        float c[4] = {};
#pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            const uint4* u = reinterpret_cast<const uint4*>(&qc.code[gid][qc.at(128 * (j / 2) + 32 * t) + 16 * (j % 2)]);
            const uint4 u0 = u[0], u1 = u[1];
            mma_bounds(c, x[0][j].x, x[1][j].x, u0.x, u0.y);
            mma_bounds(c, x[0][j].y, x[1][j].y, u0.z, u0.w);
            mma_bounds(c, x[0][j].z, x[1][j].z, u1.x, u1.y);
            mma_bounds(c, x[0][j].w, x[1][j].w, u1.z, u1.w);
        }
        const bool was[2] = {real[0], real[1]};
        if (i0 + step < cand) {
            load(i0 + step);
            load_ids(i0 + 2 * step);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float best = h0 ? fmaf(c[2 * r], 0x1p24f, o0) * s0 : -INFINITY;
            if (h1) best = fmaxf(best, fmaf(c[2 * r + 1], 0x1p24f, o1) * s1);
            best = fmaxf(best, __shfl_xor_sync(~0u, best, 1));
            best = fmaxf(best, __shfl_xor_sync(~0u, best, 2));
            const int i = i0 + gid + 8 * r;
            if (i < cand) {
                const uint32_t key = was[r] ? ordered(best) : 0u;
                if (t == 0) keys[i] = key;
                least = min(least, key);
                most = max(most, key);
            }
        }
    }
    least = __reduce_min_sync(~0u, least);
    most = __reduce_max_sync(~0u, most);
    if (lane == 0) {
        atomicMin(&range[0], least);
        atomicMax(&range[1], most);
    }
}

struct SelectShared {
    int hist[kBins];                                     // zero before the first pass
    uint32_t range[2];                                   // least and largest key
    int warp_sum[32];
    int bin, left, count, few;
    uint32_t few_keys[32];
};

// The take largest of n keys (0 < take < n), ties to the lowest index: keys above base + mask, and the first
// `left` of those within [base, base + mask]. Counting passes narrow the range by 2^11 each, until all keys of
// a bin are taken, or so few are left in it that a warp ranks them.
template <int T>
__device__ void find_threshold(const uint32_t* keys, int n, int take, SelectShared& s, uint32_t& base, uint32_t& mask,
                               int& left) {
    constexpr int kBinsPerThread = kBins / T;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    base = s.range[0];
    left = take;
    int bits = 32 - __clz(s.range[1] - base);
    mask = bits == 32 ? ~0u : (1u << bits) - 1;
    for (bool again = false; bits > 0; again = true) {
        const int shift = max(bits - 11, 0);
        if (again) {
            for (int i = tid; i < kBins; i += T) s.hist[i] = 0;
            __syncthreads();
        }
        if (tid == 0) s.few = 0;
#pragma unroll 4
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
        int above = sum - own + __reduce_add_sync(~0u, lane < warp ? s.warp_sum[lane] : 0);
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
        const int count = s.count;
        if (count == left) return;
        bits = shift;
        if (bits > 0 && count <= 32) {
            for (int i = tid; i < n; i += T) {
                const uint32_t k = keys[i];
                if (k - base <= mask) s.few_keys[atomicAdd(&s.few, 1)] = k;
            }
            __syncthreads();
            // every warp alike: the key with fewer than `left` larger ones and at least that many not smaller
            const uint32_t k = s.few_keys[lane];
            int larger = 0, equal = 0;
            for (int j = 0; j < count; ++j) {
                const uint32_t other = s.few_keys[j];
                larger += other > k;
                equal += other == k;
            }
            const uint32_t hit = __ballot_sync(~0u, lane < count && larger < left && left <= larger + equal);
            base = __shfl_sync(~0u, k, __ffs(hit) - 1);
            left -= __shfl_sync(~0u, larger, __ffs(hit) - 1);
            mask = 0;
            return;
        }
        __syncthreads();
    }
}

// What a cluster knows of its (sequence, KV head) once the candidates' keys are there.
struct Scored {
    int unit, b, h;                                      // the pair, its sequence and KV head
    int len;                                             // tokens
    Window w;
    int cand, take;                                      // candidates, and how many of them are selected
    const uint32_t* keys;                                // for the first CTA, where 0 < take < cand
    __device__ int recent() const { return w.pages - max(w.first, w.sink); }
    __device__ int total() const { return w.sink + take + recent(); }
};

// The sequence at place `at` in the order of falling length (equal ones in their own order), for the whole CTA;
// batch <= kSortedBatch.
__device__ __forceinline__ int longest_first(const int32_t* seq_len, int batch, int at) {
    __shared__ int lens[kSortedBatch], found;
    const int i = threadIdx.x, mine = i < batch ? seq_len[i] : 0;
    if (i < batch) lens[i] = mine;
    __syncthreads();
    if (i < batch) {
        int before = 0;
        for (int j = 0; j < batch; ++j) before += lens[j] > mine || (lens[j] == mine && j < i);
        if (before == at) found = i;
    }
    __syncthreads();
    return found;
}

// The cluster's CTAs score the candidates of pair blockIdx.x / ranks, or of the one at that place among the longest
// sequences (SORTED, where a.sorted says so); `frame` is called once in each, on the way.
template <int D, int T, bool SORTED, typename F>
__device__ Scored score_unit(const SelectArgs& a, int smem_keys, QueryCodes<D>& codes, SelectShared& s, uint32_t* key_store,
                             F frame) {
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kBins; i += T) s.hist[i] = 0;
    if (tid == 0) { s.range[0] = ~0u; s.range[1] = 0; }
    cluster.sync();                                      // the first CTA runs: its shared memory may be written
    grid_wait();
    grid_release();
    Scored u;
    u.unit = blockIdx.x / ranks;
    u.b = u.unit / a.h_kv;
    u.h = u.unit % a.h_kv;
    if (SORTED && a.sorted) {
        u.b = longest_first(a.seq_len, a.batch, u.b);
        u.unit = u.b * a.h_kv + u.h;
    }
    const int b = u.b, h = u.h;
    // What does not depend on the length is asked for with it: the query, and the page ids of the first tile
    // (behind the sink, wherever the sequence ends).
    const int tile = rank + ranks * warp, first_page = (a.sink + kPage - 1) / kPage;
    const int32_t* table = a.tables + (int64_t)b * a.stride + first_page;
    int id[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int i = 16 * tile + (lane >> 2) + 8 * r;
        id[r] = first_page + i < a.stride ? table[i] : 0;
    }
    QueryRow<D> query = {};
    if (warp < 8) query = fetch_query<D>(a, b, h, warp);
    u.len = checked_len(a.seq_len[b], a.max_len, a.debug && tid == 0 && rank == 0, a.dbg);
    u.w = window_of(a, u.len);
    u.cand = max(u.w.first - u.w.sink, 0);
    u.take = min(a.top, u.cand);
    uint32_t* keys = u.cand <= smem_keys ? cluster.map_shared_rank(key_store, 0) : a.keys + (int64_t)u.unit * a.max_pages;
    u.keys = u.cand <= smem_keys ? key_store : keys;
    if (u.take > 0 && u.take < u.cand)
        score_pages<D>(a, h, table, u.cand, keys, cluster.map_shared_rank(s.range, 0), tile, ranks * (T / 32), id, codes,
                          [&]() {
                              if (warp < 8) query_codes<D>(query, warp, codes);
                              frame(u);
                              __syncthreads();
                          });
    else
        frame(u);
    return u;
}

// The first CTA, behind a barrier of the cluster: put(i, p) for the i-th selected candidate p, in ascending order.
template <int T, typename F>
__device__ void list_selected(const Scored& u, SelectShared& s, F put) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cand = u.cand, take = u.take;
    const uint32_t* keys = u.keys;
    if (take == cand) {
        for (int i = tid; i < take; i += T) put(i, i);
        return;
    }
    if (take == 0) return;
    uint32_t base, mask;
    int left;
    find_threshold<T>(keys, cand, take, s, base, mask, left);
    // The list, 1,024 candidates a warp and round: lane j keeps the masks of the warp's j-th 32 of them, so the
    // keys are read once; a lane lists its own bits behind those of the lanes and warps before it.
    constexpr int kWarps = T / 32;
    int at = 0, tied = 0;                                // listed, and ties seen, in the rounds so far
    for (int i0 = 0; i0 < cand; i0 += kWarps * 1024) {
        const int share = (min(cand - i0, kWarps * 1024) + T - 1) / T * 32;
        const int from = i0 + warp * share, to = min(cand, from + share);
        uint32_t above_mask = 0, tie_mask = 0;
#pragma unroll 4
        for (int i = from; i < to; i += 32) {
            const uint32_t k = keys[min(i + lane, cand - 1)];
            const bool inside = i + lane < to, tie = k - base <= mask;
            const uint32_t above = __ballot_sync(~0u, inside && !tie && k > base), ties = __ballot_sync(~0u, inside && tie);
            if (lane == (i - from) / 32) { above_mask = above; tie_mask = ties; }
        }
        // sums over the lanes: ties and keys above, packed (each at most 1,024)
        const int own = __popc(above_mask) | __popc(tie_mask) << 16;
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) s.warp_sum[warp] = sum;
        __syncthreads();
        const int w_above = lane < kWarps ? s.warp_sum[lane] & 0xffff : 0, w_ties = lane < kWarps ? s.warp_sum[lane] >> 16 : 0;
        const int above_before = __reduce_add_sync(~0u, lane < warp ? w_above : 0) + ((sum - own) & 0xffff);
        int ties_before = tied + __reduce_add_sync(~0u, lane < warp ? w_ties : 0) + ((sum - own) >> 16);
        int out = at + above_before + min(ties_before, left) - min(tied, left);
        for (uint32_t bits = above_mask | tie_mask; bits; bits &= bits - 1) {
            const int bit = __ffs(bits) - 1;
            const bool tie = tie_mask >> bit & 1;
            if (tie && ties_before++ >= left) continue;
            put(out++, from + 32 * lane + bit);
        }
        const int all_ties = tied + __reduce_add_sync(~0u, w_ties);
        at += __reduce_add_sync(~0u, w_above) + min(all_ties, left) - min(tied, left);
        tied = all_ties;
        __syncthreads();                                 // warp_sum has been read
    }
}

}  // namespace
}  // namespace oscar
