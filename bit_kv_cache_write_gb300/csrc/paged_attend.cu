// Attention of one new token over BF16 pages (oscar_decode_bf16, oscar_decode_bf16_sparse).
//
// o = sum_t p_t v_t / sum_t p_t with p_t = 2^(l_t - m), l_t = sm_scale log2(e) q.k_t and a running reference m:
// one pass over the pages, split over the length, the splits' (m, l, acc) joined afterwards.
//
// One warp takes one 16-token page of a (sequence, KV head) at a time, for all g <= 8 query heads, with
// mma.sync m16n8k16 on operands that go from HBM straight to registers:
//   logits  S[heads, tokens] = Q[16 (8 used), d] K^T: lane (gid, t) loads 16 bytes, channels 32 j + 8 t ..
//           + 7 of token gid, which hold its part of two k-steps (the contraction's order is free, Q is
//           permuted alike);
//   output  O^T[channels, heads] = V^T[channels, 16 tokens] P^T: lane (gid, t) loads 8 channels of the tokens
//           2t, 2t+1, 2t+8, 2t+9, and byte permutations pair the tokens. S leaves the first product in the
//           layout that P^T has to enter the second one in.
// Weights enter as three bf16 pieces (24 bits), products of bf16 are exact, and each page's sums are added to
// the fp32 accumulators with rounded additions, so nothing is lost to the bf16 operands.
#include <cooperative_groups.h>

#include "paged_device.cuh"

namespace oscar {
namespace {

namespace cg = cooperative_groups;

// Warps that share a split: four for the long splits of a dense decode, two for the short ones of a sparse one
// (batch 64 at 32k, 148 pages a head: 154 us against 161 with four and 157 with one).
constexpr int attend_warps(bool sparse) { return sparse ? 2 : 4; }
constexpr int kClusterWarps = 8;         // of a split that a cluster joins
constexpr int kMaxCluster = 8;
constexpr int kMaxSplitPages = 256;      // pages of a split at most
constexpr int kSplitCost = 6;            // pages' time that a split costs apart from its pages
// Resident CTAs an SM, by registers (168 and 128 a thread).
constexpr int attend_ctas(int d, int warps) { return (d == 128 ? 12 : 16) / warps; }
constexpr float kNoLogit = -1e30f;       // running reference before any token
constexpr float kHeadroom = 8.0f;        // the reference is raised when a logit passes it by this much (log2)

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two fp32 to packed bf16 (first argument in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// One output value from its accumulator and the sum of its weights; zeros where there is no token.
__device__ __forceinline__ void store_out(const AttendArgs& a, int64_t i, float acc, float sum) {
    const float r = sum == 0.0f ? 0.0f : acc / sum;
    if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16(r);
    else static_cast<float*>(a.out)[i] = r;
}

template <int D>
struct Page {
    uint4 k[2][D / 32];                  // tokens gid, gid + 8
    uint4 v[4][D / 64];                  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
};

template <int D>
__device__ __forceinline__ void load_k(Page<D>& p, const uint16_t* page, int gid, int t) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) p.k[n][j] = ldg_stream(page + (gid + 8 * n) * D + 32 * j + 8 * t);
}
template <int D>
__device__ __forceinline__ void load_v(Page<D>& p, const uint16_t* page, int gid, int t) {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int f = 0; f < D / 64; ++f)
            p.v[n][f] = ldg_stream(page + kPage * D + (2 * t + (n & 1) + 8 * (n >> 1)) * D + 64 * f + 8 * gid);
}

// W warps share a split. CLUSTER: the splits of a (sequence, KV head) are a cluster that joins them itself.
template <int D, bool SPARSE, int W, bool CLUSTER>
__global__ void __launch_bounds__(W * 32, CLUSTER ? 1 : attend_ctas(D, W)) attend_kernel(AttendArgs a) {
    constexpr int kTiles = D / 16;       // m-tiles of the output product
    __shared__ float warp_m[W][8], warp_l[W][8];
    __shared__ float warp_acc[W][8][D];
    __shared__ float cta_m[8], cta_l[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % a.splits;
    const int unit = blockIdx.x / a.splits, h = unit % a.h_kv, b = unit / a.h_kv;
    grid_wait();
    grid_release();
    const int32_t* table = a.tables + (int64_t)b * a.stride;
    const int32_t* list = SPARSE ? a.chosen + (int64_t)unit * a.cap : nullptr;
    // This warp's pages are first + warp, + W, ...; lane l holds the id and the valid tokens of the
    // l-th of every 32 of them, so that a page's address waits for no load. The first 32 logical pages are asked
    // for together with the length.
    const int first = split * a.pages_per_split;
    int lane_logical = first + warp + W * lane;
    if (SPARSE) lane_logical = lane_logical < a.cap ? list[lane_logical] : -1;
    int lane_id = lane_logical >= 0 && lane_logical < a.stride ? table[lane_logical] : -1;
    const int len = checked_len(a.seq_len[b], a.max_len, a.debug && split == 0 && threadIdx.x == 0, a.dbg);
    const int listed = SPARSE ? a.n_chosen[unit] : (len + kPage - 1) / kPage;
    const int last = min(listed, first + a.pages_per_split);
    if (!CLUSTER && first >= last && a.splits > 1) return;      // the join skips empty splits by the same rule

    // Q as the A operand: rows gid (heads), the upper eight rows are empty.
    uint4 q[D / 32];
    const uint16_t* qrow = a.q + b * a.q_stride + (int64_t)(h * a.g + gid) * D;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
        q[j] = gid < a.g ? *reinterpret_cast<const uint4*>(qrow + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);

    float m = kNoLogit, l = 0.0f;        // head gid (l: this lane's tokens)
    float acc[kTiles][4] = {};           // channels of gid, heads 2t and 2t + 1

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
        const int valid = __shfl_sync(~0u, lane_valid, n & 31);
        Page<D> p;
        load_k<D>(p, page, gid, t);
        load_v<D>(p, page, gid, t);

        float s[2][4] = {};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                mma_bf16(s[n], q[j].x, 0, q[j].y, 0, p.k[n][j].x, p.k[n][j].y);
                mma_bf16(s[n], q[j].z, 0, q[j].w, 0, p.k[n][j].z, p.k[n][j].w);
            }
        float x[4];                      // tokens 2t, 2t + 1, 2t + 8, 2t + 9 of head gid
#pragma unroll
        for (int n = 0; n < 4; ++n) x[n] = s[n >> 1][n & 1] * a.scale_log2;
        if (valid < kPage) {             // masked tokens: no weight, and their V cannot carry a NaN in
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (2 * t + (n & 1) + 8 * (n >> 1) >= valid) {
                    x[n] = -INFINITY;
#pragma unroll
                    for (int f = 0; f < D / 64; ++f) p.v[n][f] = make_uint4(0, 0, 0, 0);
                }
        }
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        if (__any_sync(~0u, top > m + kHeadroom)) {
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const float m_new = fmaxf(m, top), f = exp2f(m - m_new);
            m = m_new;
            l *= f;
            const float f0 = __shfl_sync(~0u, f, 8 * t), f1 = __shfl_sync(~0u, f, 8 * t + 4);
#pragma unroll
            for (int i2 = 0; i2 < kTiles; ++i2) {
                acc[i2][0] *= f0; acc[i2][1] *= f1; acc[i2][2] *= f0; acc[i2][3] *= f1;
            }
        }
        uint32_t w[3][2];                // pieces of the weights as the B operand
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float p0 = exp2f(x[2 * n] - m), p1 = exp2f(x[2 * n + 1] - m);
            l += p0 + p1;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                w[k][n] = pack_bf16(p0, p1);
                p0 -= bf16_lo(w[k][n]);
                p1 -= bf16_hi(w[k][n]);
            }
        }
#pragma unroll
        for (int f = 0; f < D / 64; ++f)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t v0 = (&p.v[0][f].x)[u], v1 = (&p.v[1][f].x)[u], v2 = (&p.v[2][f].x)[u],
                               v3 = (&p.v[3][f].x)[u];
                const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632),
                               a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
                float c[4] = {};
#pragma unroll
                for (int k = 2; k >= 0; --k) mma_bf16(c, a0, a1, a2, a3, w[k][0], w[k][1]);
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[4 * f + u][k] += c[k];
            }
    }

    // Join the warps: reference and sum per head, accumulators through shared memory.
    l += __shfl_xor_sync(~0u, l, 1);
    l += __shfl_xor_sync(~0u, l, 2);
    if (t == 0) { warp_m[warp][gid] = m; warp_l[warp][gid] = l; }
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)      // rows gid and gid + 8 of m-tile (f, u) are channels 64 f + 8 gid + 2 u and + 1
            warp_acc[warp][2 * t + (k & 1)][64 * (i / 4) + 8 * gid + 2 * (i % 4) + (k >> 1)] = acc[i][k];
    __syncthreads();
    const int64_t row0 = (int64_t)b * a.h_kv * a.g + h * a.g;
    for (int x = threadIdx.x; x < a.g * D; x += W * 32) {
        const int head = x / D, c = x % D;
        float mm = warp_m[0][head];
#pragma unroll
        for (int w = 1; w < W; ++w) mm = fmaxf(mm, warp_m[w][head]);
        float ll = 0.0f, o = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = exp2f(warp_m[w][head] - mm);
            ll += f * warp_l[w][head];
            o += f * warp_acc[w][head][c];
        }
        if (CLUSTER) {
            warp_acc[0][head][c] = o;                    // read by this thread alone so far
            if (c == 0) { cta_m[head] = mm; cta_l[head] = ll; }
        } else if (a.splits == 1) {
            store_out(a, (row0 + head) * D + c, o, ll);
        } else {
            a.split_acc[((row0 + head) * a.splits + split) * D + c] = o;
            if (c == 0) a.split_ml[(row0 + head) * a.splits + split] = make_float2(mm, ll);
        }
    }
    if (CLUSTER) {                                       // each CTA joins its share of the outputs
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        const int share = (a.g * D + a.splits - 1) / a.splits, end = min(a.g * D, (split + 1) * share);
        for (int x = split * share + threadIdx.x; x < end; x += W * 32) {
            const int head = x / D, c = x % D;
            float rm[kMaxCluster], mm = kNoLogit, ll = 0.0f, o = 0.0f;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                rm[r] = r < a.splits ? *cluster.map_shared_rank(&cta_m[head], r) : kNoLogit;
                mm = fmaxf(mm, rm[r]);
            }
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                if (r >= a.splits) continue;
                const float f = exp2f(rm[r] - mm);
                ll += f * *cluster.map_shared_rank(&cta_l[head], r);
                o += f * *cluster.map_shared_rank(&warp_acc[0][head][c], r);
            }
            store_out(a, (row0 + head) * D + c, o, ll);
        }
        cluster.sync();                                  // the other CTAs have read this one's memory
    }
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
    // few splits: a warp per head; more: a CTA of 8 warps; hundreds (one long sequence, few heads): of 32
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
    // heads: 5.3 us on the GPU as with the join as a kernel, and 7.0 us of host time against 8.5. Clusters of 16 do
    // not all find their place at once (128 pages, eight heads: 13 us against 7.4).
    int ranks = 1;
    while (ranks < kMaxCluster && ranks * kClusterWarps < max_pages) ranks *= 2;
    if (max_pages > attend_warps(sparse) && units * ranks <= num_sms && max_pages <= 2 * ranks * kClusterWarps) {
        p.cluster = true;
        p.splits = ranks;
        p.pages_per_split = (max_pages + ranks - 1) / ranks;
        return p;
    }
    const int warps = attend_warps(sparse);
    const long long slots = (long long)attend_ctas(s.d, warps) * num_sms;     // resident CTAs
    const long long most = (max_pages + warps - 1) / warps;
    // Splits that fill w waves of CTAs, for the w whose waves take least: a CTA's pages and about kSplitCost pages'
    // time to start and join. No split is longer than kMaxSplitPages, so that sequences of several lengths share out.
    long long best = 0, splits = 1;
    for (int w = 1; w <= 16 && units > 0; ++w) {
        long long n = w * slots / units;
        n = n > most ? most : n;
        if (n < 1) n = 1;
        const long long pages = (max_pages + n - 1) / n, waves = (units * n + slots - 1) / slots;
        const long long cost = waves * (pages + kSplitCost);
        if (best == 0 || cost < best) { best = cost; splits = n; }
        if (n == most) break;
    }
    const long long by_len = (max_pages + kMaxSplitPages - 1) / kMaxSplitPages;
    if (splits < by_len) splits = by_len;
    p.pages_per_split = max_pages > 0 ? (int)((max_pages + splits - 1) / splits) : 1;
    p.splits = max_pages > 0 ? (max_pages + p.pages_per_split - 1) / p.pages_per_split : 1;
    const size_t parts = p.splits == 1 ? 0 : (size_t)batch * s.h_q * p.splits;
    p.ws_acc = (parts * s.d * sizeof(float) + 255) / 256 * 256;
    p.ws_total = p.ws_acc + (parts * sizeof(float2) + 255) / 256 * 256;
    return p;
}

cudaError_t launch_attend(const AttendArgs& a, int d, cudaStream_t st) {
    if (d == 128) return a.chosen ? launch<128, true>(a, st) : launch<128, false>(a, st);
    return a.chosen ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

}  // namespace oscar
