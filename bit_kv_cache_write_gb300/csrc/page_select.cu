// The selection of a sparse decode's pages as a kernel: one cluster per (sequence, KV head), see page_select.cuh.
#include "page_select.cuh"

namespace oscar {
namespace {

template <int D, int T>
__global__ void __launch_bounds__(T, 1024 / T) select_kernel(SelectArgs a, int smem_keys) {
    __shared__ __align__(16) QueryCodes<D> codes;
    __shared__ SelectShared s;
    extern __shared__ uint32_t key_store[];
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const Scored u = score_unit<D, T, true>(a, smem_keys, codes, s, key_store, [&](const Scored& u) {
        if (rank != 0) return;                           // everything but the selected pages
        int32_t* list = a.chosen + (int64_t)u.unit * a.cap;
        const int recent = u.recent(), total = u.total();
        for (int i = threadIdx.x; i < u.w.sink; i += T) list[i] = i;
        for (int i = threadIdx.x; i < recent; i += T) list[u.w.sink + u.take + i] = u.w.pages - recent + i;
        for (int i = total + threadIdx.x; i < a.cap; i += T) list[i] = -1;
        if (threadIdx.x == 0) a.n_chosen[u.unit] = total;
    });
    cluster.sync();
    if (rank != 0) return;
    int32_t* list = a.chosen + (int64_t)u.unit * a.cap;
    list_selected<T>(u, s, [&](int i, int p) { list[u.w.sink + i] = u.w.sink + p; });
}

template <int D, int T>
cudaError_t launch(SelectArgs a, int num_sms, cudaStream_t st) {
    const long long units = (long long)a.batch * a.h_kv;
    // CTAs of a cluster: as many as the card holds at once (1,024 threads an SM) with a tile of 16 pages for every
    // warp, and twice as many where each still has kLongShare pages, so that long sequences among short ones spread
    // out. 16 sequences of 4k to 131k (128 units): 76 us with four CTAs, 85 with two, 84 with eight; 16 of 32k: 56 with
    // four, 50 with two, 55 with one; 64 of 32k 159 with two, 150 with one.
    int cluster = 1;
    while (cluster < kSelectMaxCluster && 2 * cluster * (T / 2) <= a.max_pages) {
        const long long threads = 2 * cluster * units * T;
        if (threads > 1024LL * num_sms && (threads > 2048LL * num_sms || a.max_pages < 2 * cluster * kLongShare)) break;
        cluster *= 2;
    }
    // Where not all clusters run at once the longest sequences go first: that mixed batch 76 us against 82. More than
    // kSortedBatch sequences keep their order: each CTA counts the longer ones, which has not been measured for more.
    a.sorted = cluster > 1 && a.batch <= kSortedBatch && cluster * units * T > 1024LL * num_sms;
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
    // Few sequences: larger CTAs, so that one has the threads for the selection. Mixed batch of 16 (128 units): 76 us
    // with 512 threads, 88 with 256; 64 of 32k (512 units) 154 and 150.
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
