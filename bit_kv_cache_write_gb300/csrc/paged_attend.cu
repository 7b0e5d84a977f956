// Attention of one new token over BF16 pages as kernels: the splits, their join, and how many there are. The
// arithmetic is in paged_attend.cuh.
#include "paged_attend.cuh"

namespace oscar {
namespace {

// Warps that share a split: four for the long splits of a dense decode, two for the short ones of a sparse one
// (batch 64 at 32k, 148 pages a head: 151 us, 154 with four and 147 with one; 16 of 4k to 131k: 77, 79 and 79).
constexpr int attend_warps(bool sparse) { return sparse ? 2 : 4; }
constexpr int kClusterWarps = 8;         // of a split that a cluster joins
constexpr int kMaxSplitPages = 256;      // pages of a split at most
constexpr int kSplitCost = 6;            // pages' time that a split costs apart from its pages
constexpr int kJoinCost = 16;            // and the join of several
constexpr int kMaxWaves = 8;             // waves of CTAs, unless kMaxSplitPages asks for more
// Resident CTAs an SM, by registers (168 and 128 a thread).
constexpr int attend_ctas(int d, int warps) { return (d == 128 ? 12 : 16) / warps; }

size_t part_bytes(size_t parts, size_t each) { return (parts * each + 255) / 256 * 256; }

// Block and thread once more, as values that the compiler cannot trace to the first ones: what follows a NaN works out
// anew what it needs, and the main loop keeps nothing for it in registers (40 bytes of spills and 1 % otherwise).
struct Place { int block, thread; };
__device__ __forceinline__ Place place_anew() {
    Place p;
    asm volatile("mov.u32 %0, %%ctaid.x;\nmov.u32 %1, %%tid.x;" : "=r"(p.block), "=r"(p.thread));
    return p;
}

// A warp's second way over its pages. The queries are still there: `out` may lie over them.
template <int D, bool SPARSE, int W>
__device__ __forceinline__ void odd_pages(const AttendArgs& a, WarpParts<D, W>& parts, const uint4 (&q)[D / 32]) {
    const Place p = place_anew();
    const int lane = p.thread & 31, warp = p.thread >> 5, gid = lane >> 2, t = lane & 3;
    const int unit = p.block / a.splits, h = unit % a.h_kv, b = unit / a.h_kv;
    const int32_t* table = a.tables + (int64_t)b * a.stride;
    const int32_t* list = SPARSE ? a.chosen + (int64_t)unit * a.cap : nullptr;
    const int len = max(0, min(a.seq_len[b], a.max_len)), first = p.block % a.splits * a.pages_per_split;
    const int last = min(SPARSE ? a.n_chosen[unit] : (len + kPage - 1) / kPage, first + a.pages_per_split);
    float sum[D / 16][4] = {};
    for (int i = first + warp; i < last; i += W) {
        const int logical = SPARSE ? list[i] : i, id = table[logical];
        const int valid = id >= 0 && id < a.pages ? min(kPage, len - logical * kPage) : 0;
        if (valid > 0)
            odd_page<D>(sum, q, a.pool + ((int64_t)id * a.h_kv + h) * (2 * kPage * D), valid, a.scale_log2, gid, t);
    }
    put_sums<D, W>(parts, sum, warp, gid, t);
}

// The outputs that such a way decides; `odd` has a bit for each of this thread's NaN.
template <int D, int W>
__device__ __forceinline__ void rewrite_odd(const AttendArgs& a, const WarpParts<D, W>& parts, uint32_t odd) {
    const Place p = place_anew();
    const int unit = p.block / a.splits, split = p.block % a.splits;
    const int64_t row0 = (int64_t)unit * a.g;
    for (int x = p.thread; odd; x += W * 32, odd >>= 1) {
        const int head = x / D, c = x % D;
        const float o = odd & 1 ? odd_sum<D, W>(parts, head, c) : 0.0f;
        if (o == 0.0f) continue;
        float l = 0.0f;                                      // 0, NaN: a head without weight, without result
        for (int i = 0; i < W; ++i) l += parts.l[i][head];
        if (a.splits == 1) store_out(a, (row0 + head) * D + c, o, l);
        else a.split_acc[((row0 + head) * a.splits + split) * D + c] = o;
    }
}

// W warps share a split. CLUSTER: the splits of a (sequence, KV head) are a cluster that joins them itself.
template <int D, bool SPARSE, int W, bool CLUSTER>
__global__ void __launch_bounds__(W * 32, CLUSTER ? 1 : attend_ctas(D, W)) attend_kernel(AttendArgs a) {
    __shared__ WarpParts<D, W> parts;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % a.splits;
    const int unit = blockIdx.x / a.splits, h = unit % a.h_kv, b = unit / a.h_kv;
    grid_wait();
    grid_release();
    const int32_t* table = a.tables + (int64_t)b * a.stride;
    const int32_t* list = SPARSE ? a.chosen + (int64_t)unit * a.cap : nullptr;
    // This warp's pages are first + warp, + W, ...; lane l holds the id and the valid tokens of the l-th of every
    // 32 of them, so that a page's address waits for no load. The first 32 logical pages are asked for together
    // with the length.
    const int first = split * a.pages_per_split;
    int lane_logical = first + warp + W * lane;
    if (SPARSE) lane_logical = lane_logical < a.cap ? list[lane_logical] : -1;
    int lane_id = lane_logical >= 0 && lane_logical < a.stride ? table[lane_logical] : -1;
    const int len = checked_len(a.seq_len[b], a.max_len, a.debug && split == 0 && threadIdx.x == 0, a.dbg);
    const int listed = SPARSE ? a.n_chosen[unit] : (len + kPage - 1) / kPage;
    const int last = min(listed, first + a.pages_per_split);
    if (!CLUSTER && first >= last && a.splits > 1) return;      // the join skips empty splits by the same rule

    uint4 q[D / 32];
    load_query<D>(q, a, b, h, gid, t);
    Gathered<D> s;
    const int mine = (last - first - warp + W - 1) / W;
    int lane_valid = 0;
    for (int n = 0; n < mine; ++n) {
        if ((n & 31) == 0) {
            const int i = first + warp + W * (n + lane);
            if (n > 0 && i < last) {
                lane_logical = SPARSE ? list[i] : i;
                lane_id = table[lane_logical];
            }
            lane_valid = 0;
            if (i < last) {
                if (lane_id >= 0 && lane_id < a.pages) lane_valid = min(kPage, len - lane_logical * kPage);
                else if (a.debug) record_error(&a.dbg->kind, &a.dbg->index, 2, lane_id);
            }
            if (lane_valid <= 0) lane_id = lane_valid = 0;
        }
        const uint16_t* page = a.pool + ((int64_t)__shfl_sync(~0u, lane_id, n & 31) * a.h_kv + h) * (2 * kPage * D);
        attend_page<D>(s, q, page, __shfl_sync(~0u, lane_valid, n & 31), a.scale_log2, gid, t);
    }

    put_warp<D, W>(parts, s, warp, gid, t);
    const int64_t row0 = (int64_t)b * a.h_kv * a.g + h * a.g;
    if (CLUSTER) {
        join_cluster<D, W, kAttendMaxCluster>(a, parts, row0, split, a.splits,
                                              [&]() { odd_pages<D, SPARSE, W>(a, parts, q); });
        return;
    }
    __syncthreads();
    static_assert(8 * D <= 32 * W * 32, "a bit for each output of a thread");
    uint32_t odd = 0;
    for (int x = threadIdx.x, n = 0; x < a.g * D; x += W * 32, ++n) {
        const int head = x / D, c = x % D;
        float m, l, o;
        join_warps<D, W>(parts, head, c, m, l, o);
        odd |= (o != o) << n;
        if (a.splits == 1) {
            store_out(a, (row0 + head) * D + c, o, l);
        } else {
            a.split_acc[((row0 + head) * a.splits + split) * D + c] = o;
            if (c == 0) a.split_ml[(row0 + head) * a.splits + split] = make_float2(m, l);
        }
    }
    if (!__syncthreads_or(odd)) return;
    odd_pages<D, SPARSE, W>(a, parts, q);
    __syncthreads();
    rewrite_odd<D, W>(a, parts, odd);
}

// Joins the splits of query heads, W warps to a head: a warp takes every W-th split, 16 bytes a lane.
template <int D, bool SPARSE, int W, int THREADS>
__global__ void __launch_bounds__(THREADS) join_kernel(AttendArgs a) {
    constexpr int kLanes = D / 4;                        // lanes that hold one split's channels
    constexpr int kPer = 32 / kLanes;                    // splits that a warp reads at a time
    constexpr int kRows = THREADS / 32 / W;
    __shared__ float4 warp_o[THREADS / 32][kLanes];
    __shared__ float warp_l[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % W;
    const int64_t row = (int64_t)blockIdx.x * kRows + warp / W;
    const int hq = a.h_kv * a.g;
    grid_wait();
    grid_release();
    const bool inside = row < (int64_t)a.batch * hq;
    float4 o = make_float4(0, 0, 0, 0);
    float l = 0.0f;
    if (inside) {
        const int b = (int)(row / hq), unit = b * a.h_kv + (int)(row % hq) / a.g;
        const int listed = SPARSE ? a.n_chosen[unit] : (checked_len(a.seq_len[b], a.max_len, 0, a.dbg) + kPage - 1) / kPage;
        const int n = (listed + a.pages_per_split - 1) / a.pages_per_split;
        const float2* ml = a.split_ml + row * a.splits;
        const float4* acc = reinterpret_cast<const float4*>(a.split_acc + row * a.splits * D) + lane % kLanes;
        float m = kNoLogit;
        for (int i = lane; i < a.splits; i += 32) {      // a split that is not there holds anything
            const float x = ml[i].x;
            if (i < n) m = fmaxf(m, x);
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, s));
#pragma unroll 4
        for (int i = part * kPer + lane / kLanes; i < n; i += W * kPer) {
            const float2 x = ml[i];
            const float4 y = acc[(int64_t)i * kLanes];
            const float f = exp2f(x.x - m);
            l += f * x.y;
            o.x += f * y.x; o.y += f * y.y; o.z += f * y.z; o.w += f * y.w;
        }
        if (o.x != o.x || o.y != o.y || o.z != o.z || o.w != o.w) {      // a NaN: infinities may be among its parts
            float4 r = make_float4(0, 0, 0, 0);
            for (int i = part * kPer + lane / kLanes; i < n; i += W * kPer) {
                const float4 y = acc[(int64_t)i * kLanes];
                const float f = exp2f(ml[i].x - m);
                // f x, where an infinite x stays one however small f has become
                const auto add = [f](float& sum, float x) { sum += fabsf(x) == INFINITY ? x : f * x; };
                add(r.x, y.x); add(r.y, y.y); add(r.z, y.z); add(r.w, y.w);
            }
            if (o.x != o.x) o.x = r.x;
            if (o.y != o.y) o.y = r.y;
            if (o.z != o.z) o.z = r.z;
            if (o.w != o.w) o.w = r.w;
        }
        if (kPer == 2) {
            l += __shfl_xor_sync(~0u, l, 16);
            o.x += __shfl_xor_sync(~0u, o.x, 16); o.y += __shfl_xor_sync(~0u, o.y, 16);
            o.z += __shfl_xor_sync(~0u, o.z, 16); o.w += __shfl_xor_sync(~0u, o.w, 16);
        }
    }
    if (W > 1) {
        if (lane < kLanes) warp_o[warp][lane] = o;
        if (lane == 0) warp_l[warp] = l;
        __syncthreads();
        if (part != 0) return;
        o = make_float4(0, 0, 0, 0);
        l = 0.0f;
#pragma unroll 8
        for (int w = 0; w < W; ++w) {
            const float4 y = warp_o[warp + w][lane % kLanes];
            l += warp_l[warp + w];
            o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
        }
    }
    if (!inside || lane >= kLanes) return;
    // no token: zeros
    const float4 r = l == 0.0f ? make_float4(0, 0, 0, 0) : make_float4(o.x / l, o.y / l, o.z / l, o.w / l);
    if (a.out_bf16) {
        uint2 x = make_uint2(pack_bf16(r.x, r.y), pack_bf16(r.z, r.w));
        reinterpret_cast<uint2*>(a.out)[row * kLanes + lane] = x;
    } else {
        reinterpret_cast<float4*>(a.out)[row * kLanes + lane] = r;
    }
}

template <int D, bool SPARSE>
cudaError_t launch(const AttendArgs& a, cudaStream_t st) {
    const long long ctas = (long long)a.splits * a.h_kv * a.batch;
    if (ctas > 0x7fffffffLL || (long long)a.batch * a.h_kv * a.g > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (a.cluster) {
        return launch_dependent(attend_kernel<D, SPARSE, kClusterWarps, true>, dim3((unsigned)ctas),
                                dim3(kClusterWarps * 32), 0, st, a.splits, a);
    }
    constexpr int kWarps = attend_warps(SPARSE);
    cudaError_t e = launch_dependent(attend_kernel<D, SPARSE, kWarps, false>, dim3((unsigned)ctas), dim3(kWarps * 32), 0,
                                     st, 1, a);
    if (e != cudaSuccess || a.splits == 1) return e;
    // Few splits: a warp per head; more: a CTA of 8 warps; hundreds (one long sequence, few heads): of 32. 32 x 4,000
    // tokens (5 splits) take 86.0 us with a warp, 86.6 with 8; 16 x 4,000 (7) 48.8 and 46.7; 100,000 of eight heads (57)
    // 72.4 and 65.7, with 32 66.0; of four heads (114) 37.7 with 8 and 37.2 with 32; of one (447) 17.4 and 15.0.
    const long long rows = (long long)a.batch * a.h_kv * a.g;
    if (a.splits > 96)
        return launch_dependent(join_kernel<D, SPARSE, 32, 1024>, dim3((unsigned)rows), dim3(1024), 0, st, 1, a);
    if (a.splits > 8)
        return launch_dependent(join_kernel<D, SPARSE, 8, 256>, dim3((unsigned)rows), dim3(256), 0, st, 1, a);
    return launch_dependent(join_kernel<D, SPARSE, 1, 256>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, 1, a);
}

}  // namespace

AttendPlan plan_attend(const Shape& s, int num_sms, int batch, int max_pages, bool sparse) {
    AttendPlan p{};
    const long long units = (long long)batch * s.h_kv;
    // Small work, at most two pages a warp: one cluster for each (sequence, KV head) and one launch. 84 pages, two KV
    // heads: 4.4 us on the GPU against 4.7 with the join as a kernel, and 7.0 us of host time against 9.2; 125 pages,
    // eight heads: 6.2 us both. Clusters of 16 do not all find their place at once (13 us there).
    int ranks = 1;
    while (ranks < kAttendMaxCluster && ranks * kClusterWarps < max_pages) ranks *= 2;
    if (max_pages > attend_warps(sparse) && units * ranks <= num_sms && max_pages <= 2 * ranks * kClusterWarps) {
        p.cluster = true;
        p.splits = ranks;
        p.pages_per_split = (max_pages + ranks - 1) / ranks;
        return p;
    }
    const int warps = attend_warps(sparse);
    const long long slots = (long long)attend_ctas(s.d, warps) * num_sms;     // resident CTAs
    const long long most = (max_pages + warps - 1) / warps;
    // One split, or splits that fill w waves of CTAs, for the w whose waves take least: a CTA's pages, about
    // kSplitCost pages' time to start, and the join's kJoinCost. No split is longer than kMaxSplitPages, so that
    // sequences of several lengths share out. 32 sequences of 1,024 tokens, 8 heads: 26.6 us in one split, 29.1 in three.
    long long best = 0, splits = 1;
    for (int w = 0; w <= kMaxWaves && units > 0; ++w) {
        long long n = w * slots / units;
        n = n > most ? most : n;
        if (n < 1) n = 1;
        const long long pages = (max_pages + n - 1) / n, waves = (units * n + slots - 1) / slots;
        const long long cost = waves * (pages + kSplitCost) + (n > 1 ? kJoinCost : 0);
        if (best == 0 || cost < best) { best = cost; splits = n; }
        if (n == most) break;
    }
    const long long by_len = (max_pages + kMaxSplitPages - 1) / kMaxSplitPages;
    if (splits < by_len) splits = by_len;
    p.pages_per_split = max_pages > 0 ? (int)((max_pages + splits - 1) / splits) : 1;
    p.splits = max_pages > 0 ? (max_pages + p.pages_per_split - 1) / p.pages_per_split : 1;
    const size_t parts = p.splits == 1 ? 0 : (size_t)batch * s.h_q * p.splits;
    p.ws_acc = part_bytes(parts, s.d * sizeof(float));
    p.ws_total = p.ws_acc + part_bytes(parts, sizeof(float2));
    return p;
}

size_t attend_workspace_bytes(const Shape& s, int num_sms, int batch, int max_pages, bool sparse) {
    const int warps = attend_warps(sparse);
    const long long units = (long long)batch * s.h_kv, most = (max_pages + warps - 1) / warps;
    const long long waves = (long long)kMaxWaves * attend_ctas(s.d, warps) * num_sms;
    const long long by_len = units * ((max_pages + kMaxSplitPages - 1) / kMaxSplitPages);
    const long long bound = waves > by_len ? waves : by_len;
    const size_t parts = most < 2 ? 0 : (size_t)(units * most < bound ? units * most : bound) * (s.h_q / s.h_kv);
    return part_bytes(parts, s.d * sizeof(float)) + part_bytes(parts, sizeof(float2));
}

cudaError_t launch_attend(const AttendArgs& a, int d, cudaStream_t st) {
    if (d == 128) return a.chosen ? launch<128, true>(a, st) : launch<128, false>(a, st);
    return a.chosen ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

}  // namespace oscar
