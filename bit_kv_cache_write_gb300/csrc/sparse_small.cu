// The sparse decode of few (sequence, KV head) pairs in one kernel: selection (page_select.cuh) and attention
// (paged_attend.cuh) by one cluster each.
//
// With few pairs everything is latency: three kernels' starts, the loads of lengths, lists and tables in each, and
// a join. Here the cluster that has scored the pages stays. While its first CTA selects, the warps of the others
// attend to the sink and the recent window; the selected pages come as page ids through the first CTA's shared
// memory, a page or two a warp, and the cluster joins its warps' parts.
//
// 100,000 tokens, 8 KV heads, 256 + 21 pages: 20.1 us on the GPU against 20.7 with separate kernels, and one launch
// instead of three (9.6 us of host time a call against 14.0). About 7 us go to the scores, 4.5 to the selection, 9 to
// the pages and the join: 64 of the 152 SMs fetch them.
#include "page_select.cuh"
#include "paged_attend.cuh"

namespace oscar {
namespace {

constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallCluster = 8;                     // larger ones do not all find their place at once
constexpr int kSmallPages = 3;                       // selected pages a warp at most
constexpr int kSmallTop = kSmallCluster * kSmallWarps * kSmallPages;

template <int D>
__global__ void __launch_bounds__(kSmallThreads, 1) sparse_small_kernel(SelectArgs a, AttendArgs t, int smem_keys) {
    __shared__ __align__(16) QueryCodes<D> codes;
    __shared__ SelectShared s;
    __shared__ int2 selected[kSmallTop];             // page id and logical page, in the first CTA
    extern __shared__ __align__(16) unsigned char dynamic[];     // keys (first CTA), then the warps' parts
    uint32_t* key_store = reinterpret_cast<uint32_t*>(dynamic);
    auto& parts = *reinterpret_cast<WarpParts<D, kSmallWarps>*>(dynamic);
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, quad = lane & 3;
    const Scored u = score_unit<D, kSmallThreads, false>(a, smem_keys, codes, s, key_store, [&](const Scored& u) {
        if (rank != 0) return;                       // everything but the selected pages
        int32_t* list = a.chosen + (int64_t)u.unit * a.cap;
        const int recent = u.recent(), total = u.total();
        for (int i = threadIdx.x; i < u.w.sink; i += kSmallThreads) list[i] = i;
        for (int i = threadIdx.x; i < recent; i += kSmallThreads) list[u.w.sink + u.take + i] = u.w.pages - recent + i;
        for (int i = total + threadIdx.x; i < a.cap; i += kSmallThreads) list[i] = -1;
        if (threadIdx.x == 0) a.n_chosen[u.unit] = total;
    });
    const int b = u.b, h = u.h;
    const int32_t* table = a.tables + (int64_t)b * a.stride;
    int32_t* list = a.chosen + (int64_t)u.unit * a.cap;
    uint4 q[D / 32];
    load_query<D>(q, t, b, h, gid, quad);
    Gathered<D> g;
    auto attend = [&](int id, int logical) {
        int valid = 0;
        if (id >= 0 && id < t.pages) valid = min(kPage, u.len - logical * kPage);
        else if (t.debug && lane == 0) record_error(&t.dbg->kind, &t.dbg->index, 2, id);
        const uint16_t* page = t.pool + ((int64_t)(valid > 0 ? id : 0) * t.h_kv + h) * (2 * kPage * D);
        attend_page<D>(g, q, page, max(valid, 0), t.scale_log2, gid, quad);
    };
    cluster.sync();                                  // the keys are there
    if (rank == 0)
        list_selected<kSmallThreads>(u, s, [&](int i, int p) {
            const int logical = u.w.sink + p;
            list[logical - p + i] = logical;
            selected[i] = make_int2(table[logical], logical);
        });
    if (rank != 0 || ranks == 1) {                   // the windows, whose pages need no selection
        const int kept = u.w.sink + u.recent(), warps = (ranks > 1 ? ranks - 1 : 1) * kSmallWarps;
        for (int i = (ranks > 1 ? rank - 1 : 0) + warp * (ranks > 1 ? ranks - 1 : 1); i < kept; i += warps) {
            const int logical = i < u.w.sink ? i : u.w.pages - u.recent() + i - u.w.sink;
            attend(table[logical], logical);
        }
    }
    cluster.sync();                                  // the selected pages are listed
    const int2* from = cluster.map_shared_rank(selected, 0);
    for (int i = rank + ranks * warp; i < u.take; i += ranks * kSmallWarps) {
        const int2 e = from[i];
        attend(e.x, e.y);
    }
    put_warp<D, kSmallWarps>(parts, g, warp, gid, quad);     // the keys have been read
    const auto again = [&]() {                       // the selected pages, then the windows'
        const bool windows = rank != 0 || ranks == 1;
        const int others = ranks > 1 ? ranks - 1 : 1, kept = windows ? u.w.sink + u.recent() : 0;
        int i = rank + ranks * warp, j = windows ? (ranks > 1 ? rank - 1 : 0) + warp * others : kept;
        float sum[D / 16][4] = {};
        while (i < u.take || j < kept) {
            int id, logical;
            if (i < u.take) {
                const int2 e = from[i];
                id = e.x;
                logical = e.y;
                i += ranks * kSmallWarps;
            } else {
                logical = j < u.w.sink ? j : u.w.pages - u.recent() + j - u.w.sink;
                id = table[logical];
                j += others * kSmallWarps;
            }
            const int valid = id >= 0 && id < t.pages ? min(kPage, u.len - logical * kPage) : 0;
            if (valid > 0)
                odd_page<D>(sum, q, t.pool + ((int64_t)id * t.h_kv + h) * (2 * kPage * D), valid, t.scale_log2, gid, quad);
        }
        put_sums<D, kSmallWarps>(parts, sum, warp, gid, quad);
    };
    join_cluster<D, kSmallWarps, kSmallCluster>(t, parts, (int64_t)b * t.h_kv * t.g + h * t.g, rank, ranks, again);
}

template <int D>
constexpr size_t kSmallSmem = kSmemKeys * sizeof(uint32_t) > sizeof(WarpParts<D, kSmallWarps>)
                                  ? kSmemKeys * sizeof(uint32_t) : sizeof(WarpParts<D, kSmallWarps>);

// Clusters of `ranks` CTAs that the current device holds at once (asked once per device and size); 0 if unknown.
template <int D>
int resident_clusters(int ranks) {
    static std::atomic<int> known[64][kSmallCluster + 1];    // 1 + the number
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev][ranks].load(std::memory_order_acquire);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ranks);
        cfg.blockDim = dim3(kSmallThreads);
        cfg.dynamicSmemBytes = kSmallSmem<D>;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ranks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (smem_opt_in<sparse_small_kernel<D>>(kSmallSmem<D>) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&clusters, sparse_small_kernel<D>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        n = 1 + clusters;
        known[dev][ranks].store(n, std::memory_order_release);
    }
    return n - 1;
}

template <int D>
cudaError_t launch(const SelectArgs& a, const AttendArgs& t, int ranks, cudaStream_t st) {
    const size_t keys = (size_t)a.max_pages * sizeof(uint32_t), parts = sizeof(WarpParts<D, kSmallWarps>);
    const size_t smem = keys > parts ? keys : parts;
    const cudaError_t e = smem_opt_in<sparse_small_kernel<D>>(kSmallSmem<D>);
    if (e != cudaSuccess) return e;
    return launch_dependent(sparse_small_kernel<D>, dim3((unsigned)(a.batch * a.h_kv * ranks)), dim3(kSmallThreads), smem,
                            st, ranks, a, t, a.max_pages);
}

}  // namespace

int sparse_small_ranks(const Shape& s, int num_sms, int batch, int max_pages, int top) {
    const long long units = (long long)batch * s.h_kv;
    const int take = top < max_pages ? top : max_pages, all = sparse_capacity(s, top);
    int ranks = 1;                                   // a page a warp in all, and a tile of 16 scores
    while (ranks < kSmallCluster && (ranks * kSmallWarps < (all < max_pages ? all : max_pages) ||
                                     ranks * kSmallThreads / 2 < max_pages) && 2 * ranks * units <= num_sms)
        ranks *= 2;
    // Few selected pages and few tiles a warp, and every cluster on the card at once. 100,000 tokens, eight heads: 384
    // pages 22.2 us against 22.6 with separate kernels, 512 24.1 and 22.7, 1,000 33.2 and 26.1; 4 x 100,000 with 128
    // pages 24.9 and 29.5, 8 x 60,000 with 64 27.8 and 28.9; 250,000 tokens 26.6 and 29.0. d = 64, two heads, 256 pages:
    // 14.8 and 13.9, for the one launch.
    if (max_pages == 0 || units * ranks > num_sms || take > ranks * kSmallWarps * kSmallPages ||
        max_pages > ranks * kSmallThreads * 4 || max_pages > kSmemKeys)
        return 0;
    const int fit = s.d == 128 ? resident_clusters<128>(ranks) : resident_clusters<64>(ranks);
    return units <= fit ? ranks : 0;
}

cudaError_t launch_sparse_small(const SelectArgs& a, const AttendArgs& t, int d, int ranks, cudaStream_t st) {
    return d == 128 ? launch<128>(a, t, ranks, st) : launch<64>(a, t, ranks, st);
}

}  // namespace oscar
