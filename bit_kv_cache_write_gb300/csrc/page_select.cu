// The pages that a sparse decode reads (oscar_decode_bf16_sparse): a cheap score per page, and the largest.
//
// Score of page p for KV head h: max over the head's g query heads of 2^e S with
// S = sum_c max(u_c lo_c, u_c hi_c), u the query's integer codes in the steps of the key bounds [lo, hi]. It
// bounds the logits of the page's keys (up to the rounding of u and to clipped codes). S is an integer below
// 2^23 and the scale a power of two, so the score is exact in fp32 and the choice does not depend on the
// order of any sum. sum max(u lo, u hi) = sum min(u, 0) lo + max(u, 0) hi: two runs of dp4a.
//
// Bounds of a (page, KV head) are 2 d bytes, a 32nd of its K and V.
#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kScorePages = 128;                 // pages of a CTA
constexpr int kSelectThreads = 1024;

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

// Integer codes of the g query heads of KV head h as dp4a words: min(u, 0) for the lower bounds in words
// [0, D / 4), max(u, 0) for the upper ones behind them. One warp a head.
template <int D>
__device__ void query_codes(const SelectArgs& a, int b, int h, int8_t (*codes)[2 * D], int* exponent) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < a.g; i += kScoreThreads / 32) {
        const uint16_t* q = a.q + b * a.q_stride + (int64_t)(h * a.g + i) * D;
        float x[D / 32], top = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const int c = lane + 32 * j, step = max(-100, min(100, (int)a.steps[h * D + c]));
            x[j] = __uint_as_float((uint32_t)q[c] << 16) * __int_as_float((127 + step) << 23);
            if (!isfinite(x[j])) x[j] = 0.0f;
            top = fmaxf(top, fabsf(x[j]));
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

template <int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(SelectArgs a) {
    __shared__ __align__(16) int8_t codes[8][2 * D];
    __shared__ int exponent[8];
    const int chunks = (a.max_pages + kScorePages - 1) / kScorePages;
    const int chunk = blockIdx.x % chunks, unit = blockIdx.x / chunks, h = unit % a.h_kv, b = unit / a.h_kv;
    grid_wait();
    grid_release();
    const int len = checked_len(a.seq_len[b], a.max_len, 0, a.dbg);
    const Window w = window_of(a, len);
    const int lo = max(w.sink, chunk * kScorePages), hi = min(w.first, (chunk + 1) * kScorePages);
    if (lo >= hi || w.first - w.sink <= a.top) return;   // no candidates, or all of them are taken
    query_codes<D>(a, b, h, codes, exponent);
    __syncthreads();
    const int t = threadIdx.x & 3;                       // four lanes a page
    for (int p = lo + (threadIdx.x >> 2); p - (threadIdx.x >> 2) < hi; p += kScoreThreads / 4) {
        const bool inside = p < hi;
        int id = inside ? a.tables[(int64_t)b * a.stride + p] : -1;
        const bool real = id >= 0 && id < a.pages;
        if (inside && !real && a.debug && t == 0) record_error(&a.dbg->kind, &a.dbg->index, 2, id);
        const int8_t* src = a.bounds + ((int64_t)(real ? id : 0) * a.h_kv + h) * (2 * D);
        uint4 x[2 * D / 64];
#pragma unroll
        for (int j = 0; j < 2 * D / 64; ++j) x[j] = ldg_stream(src + 64 * j + 16 * t);
        float best = -INFINITY;
        for (int i = 0; i < a.g; ++i) {
            int s = 0;
#pragma unroll
            for (int j = 0; j < 2 * D / 64; ++j) {
                const uint4 u = *reinterpret_cast<const uint4*>(&codes[i][64 * j + 16 * t]);
                s = __dp4a((int)x[j].x, (int)u.x, s);
                s = __dp4a((int)x[j].y, (int)u.y, s);
                s = __dp4a((int)x[j].z, (int)u.z, s);
                s = __dp4a((int)x[j].w, (int)u.w, s);
            }
            s += __shfl_xor_sync(~0u, s, 1);
            s += __shfl_xor_sync(~0u, s, 2);
            best = fmaxf(best, (float)s * __int_as_float((127 + exponent[i]) << 23));
        }
        if (inside && t == 0) a.scores[(int64_t)unit * a.max_pages + p] = real ? best : -INFINITY;
    }
}

// Sum of v over the threads before this one; the CTA's total in *total.
__device__ int scan_before(int v, int* total, int* warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = 0, sum = 0;
    for (int w = 0; w < kSelectThreads / 32; ++w) {
        if (w == warp) before = sum;
        sum += warp_sum[w];
    }
    *total = sum;
    return before + x - v;
}

// One CTA per (sequence, KV head): the top-th largest key by a radix search of 8 bits a pass, then the list
// in ascending order; of equal keys the lowest pages are taken.
__global__ void __launch_bounds__(kSelectThreads) select_kernel(SelectArgs a) {
    __shared__ int hist[256], warp_sum[kSelectThreads / 32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    const int unit = blockIdx.x, b = unit / a.h_kv, tid = threadIdx.x;
    grid_wait();
    grid_release();
    const int len = checked_len(a.seq_len[b], a.max_len, 0, a.dbg);
    const Window w = window_of(a, len);
    const int cand = max(w.first - w.sink, 0), take = min(a.top, cand);
    const float* scores = a.scores + (int64_t)unit * a.max_pages;
    uint32_t prefix = 0;                                 // the threshold's bits that are known
    int left = take;                                     // taken among the keys that share them
    const bool all = take == cand;
    if (!all && take > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
            for (int p = w.sink + tid; p < w.first; p += kSelectThreads) {
                const uint32_t k = ordered(scores[p]);
                if ((k & mask) == (prefix & mask)) atomicAdd(&hist[k >> shift & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int bin = 255, n = left;
                while (bin > 0 && hist[bin] < n) n -= hist[bin--];
                s_prefix = prefix | (uint32_t)bin << shift;
                s_left = n;
            }
            __syncthreads();
            prefix = s_prefix;
            left = s_left;
            __syncthreads();
        }
    }
    int32_t* list = a.chosen + (int64_t)unit * a.cap;
    int written = 0, ties = 0;                           // list entries and equal keys before this chunk
    for (int p0 = 0; p0 < w.pages; p0 += kSelectThreads) {
        const int p = p0 + tid;
        bool in = false, tie = false;
        if (p < w.pages) {
            if (p < w.sink || p >= w.first) in = true;
            else if (all) in = true;
            else if (take > 0) {
                const uint32_t k = ordered(scores[p]);
                in = k > prefix;
                tie = k == prefix;
            }
        }
        int total, chunk_ties;
        const int before = scan_before(tie, &chunk_ties, warp_sum);
        if (tie && ties + before < left) in = true;
        const int at = scan_before(in, &total, warp_sum);
        if (in) list[written + at] = p;
        written += total;
        ties += chunk_ties;
    }
    for (int i = written + tid; i < a.cap; i += kSelectThreads) list[i] = -1;
    if (tid == 0) a.n_chosen[unit] = written;
}

}  // namespace

size_t select_workspace_bytes(const Shape& s, int batch, int max_pages) {
    return ((size_t)batch * s.h_kv * max_pages * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_select(const SelectArgs& a, int d, cudaStream_t st) {
    const int chunks = (a.max_pages + kScorePages - 1) / kScorePages;
    const long long ctas = (long long)chunks * a.h_kv * a.batch;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t e = cudaSuccess;
    if (ctas > 0)
        e = d == 128 ? launch_dependent(score_kernel<128>, dim3((unsigned)ctas), dim3(kScoreThreads), 0, st, 1, a)
                     : launch_dependent(score_kernel<64>, dim3((unsigned)ctas), dim3(kScoreThreads), 0, st, 1, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(select_kernel, dim3(a.batch * a.h_kv), dim3(kSelectThreads), 0, st, 1, a);
}

}  // namespace oscar
