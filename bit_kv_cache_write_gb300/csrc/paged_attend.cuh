// Attention of one new token over BF16 pages (oscar_decode_bf16, oscar_decode_bf16_sparse).
//
// o = sum_t p_t v_t / sum_t p_t with p_t = 2^(l_t - m), l_t = sm_scale log2(e) q.k_t and a running reference m:
// one pass over the pages, split over the length, the splits' (m, l, acc) joined afterwards.
//
// One warp takes one 16-token page of a (sequence, KV head) at a time, for all g <= 8 query heads, with
// mma.sync m16n8k16 on operands that go from HBM straight to registers:
//   logits  S[heads, tokens] = Q[16 (8 used), d] K^T: lane (gid, t) loads 32 bytes, channels 64 j + 16 t ..
//           + 15 of token gid (16 bytes at d = 64), which hold its part of four k-steps (the contraction's order
//           is free, Q is permuted alike);
//   output  O^T[channels, heads] = V^T[channels, 16 tokens] P^T: lane (gid, t) loads d / 8 channels of the
//           tokens 2t, 2t+1, 2t+8, 2t+9, and byte permutations pair the tokens. S leaves the first product in
//           the layout that P^T has to enter the second one in.
// Weights enter as three bf16 pieces (24 bits), products of bf16 are exact, and each page's sums are added to
// the fp32 accumulators with rounded additions, so nothing is lost to the bf16 operands.
//
// HBM bounds it (g flops a byte): 12 warps an SM with up to 8 KB of a page on its way each. 100,000 tokens of 8 KV
// heads at batch 1 in 65 us, 93 % of the measured copy rate; 64 x 32,768 in 1.17 ms, 108 % (a copy is slower than
// reads alone). The tensor cores are a tenth busy; tcgen05 would want its operands in shared memory and 128 rows.
#pragma once

#include <cooperative_groups.h>

#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int kAttendMaxCluster = 8;
constexpr float kNoLogit = -3.402823466e38f; // running reference before any token: no finite logit is below it
constexpr float kHeadroom = 8.0f;        // the reference is raised when a logit passes it by this much (log2)

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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
    uint4 k[2][D / 32];                  // tokens gid, gid + 8: channels channel_of(j, t) ..
    uint4 v[4][D / 64];                  // tokens 2t, 2t + 1, 2t + 8, 2t + 9: channels d / 8 gid + 8 f ..
};

template <int D>
__device__ __forceinline__ void load_k(Page<D>& p, const uint16_t* page, int gid, int t) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const uint16_t* row = page + (gid + 8 * n) * D + 64 * j;
            if constexpr (D == 128) {
                ldg_stream32(p.k[n][2 * j], p.k[n][2 * j + 1], row + 16 * t);
            } else {
                p.k[n][2 * j] = ldg_stream(row + 8 * t);
                p.k[n][2 * j + 1] = ldg_stream(row + 32 + 8 * t);
            }
        }
}
template <int D>
__device__ __forceinline__ void load_v(Page<D>& p, const uint16_t* page, int gid, int t) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const uint16_t* row = page + kPage * D + (2 * t + (n & 1) + 8 * (n >> 1)) * D + D / 8 * gid;
        if constexpr (D == 128) ldg_stream32(p.v[n][0], p.v[n][1], row);
        else p.v[n][0] = ldg_stream(row);
    }
}

// What a warp has gathered of a (sequence, KV head): reference and sum of weights of head gid (the sum over this
// lane's tokens), and the outputs of heads 2t and 2t + 1 at the lane's channels.
template <int D>
struct Gathered {
    float m = kNoLogit, l = 0.0f;
    float acc[D / 16][4] = {};
};

// Channel from which lane t holds eight in piece j of a K row or of Q. At d = 128 pieces 2 j and 2 j + 1 are one
// 32-byte load; at d = 64 a row is one cache line, and 16-byte loads are faster (64 x 8,192 tokens 162 us against 170).
// From HBM the 32-byte ones take 1186 us against 1205 (64 x 32k); a cache that the last call left in the L2 is read
// faster by 16-byte ones (8 x 4,096 tokens 21.9 us against 28.4), but between two calls on it a model's other layers
// read theirs.
template <int D>
__device__ __forceinline__ int channel_of(int j, int t) {
    return D == 128 ? 64 * (j / 2) + 16 * t + 8 * (j % 2) : 32 * j + 8 * t;
}

// Q as the A operand: rows gid (heads), the upper eight rows are empty.
template <int D>
__device__ __forceinline__ void load_query(uint4 (&q)[D / 32], const AttendArgs& a, int b, int h, int gid, int t) {
    const uint16_t* row = a.q + b * a.q_stride + (int64_t)(h * a.g + gid) * D;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
        q[j] = gid < a.g ? *reinterpret_cast<const uint4*>(row + channel_of<D>(j, t)) : make_uint4(0, 0, 0, 0);
}

// Logits of a page's tokens 2t, 2t + 1, 2t + 8, 2t + 9 for head gid.
template <int D>
__device__ __forceinline__ void page_logits(float (&x)[4], const uint4 (&q)[D / 32], const Page<D>& p, float scale_log2) {
    float c2[2][4] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            mma_bf16(c2[n], q[j].x, 0, q[j].y, 0, p.k[n][j].x, p.k[n][j].y);
            mma_bf16(c2[n], q[j].z, 0, q[j].w, 0, p.k[n][j].z, p.k[n][j].w);
        }
#pragma unroll
    for (int n = 0; n < 4; ++n) x[n] = c2[n >> 1][n & 1] * scale_log2;
}

// V^T as the A operand: channels of m-tile 4 f + u, tokens 2t, 2t + 1 and 2t + 8, 2t + 9.
__device__ __forceinline__ void pair_tokens(uint32_t (&a)[4], uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
    a[0] = __byte_perm(v0, v1, 0x5410);
    a[1] = __byte_perm(v0, v1, 0x7632);
    a[2] = __byte_perm(v2, v3, 0x5410);
    a[3] = __byte_perm(v2, v3, 0x7632);
}

// One page of which the first `valid` tokens count.
template <int D>
__device__ __forceinline__ void attend_page(Gathered<D>& s, const uint4 (&q)[D / 32], const uint16_t* page, int valid,
                                            float scale_log2, int gid, int t) {
    Page<D> p;
    load_k<D>(p, page, gid, t);
    load_v<D>(p, page, gid, t);

    float x[4];
    page_logits<D>(x, q, p, scale_log2);
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
    if (__any_sync(~0u, top > s.m + kHeadroom)) {
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        const float m_new = fmaxf(s.m, top), f = exp2f(s.m - m_new);
        s.m = m_new;
        s.l *= f;
        const float f0 = __shfl_sync(~0u, f, 8 * t), f1 = __shfl_sync(~0u, f, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            s.acc[i][0] *= f0; s.acc[i][1] *= f1; s.acc[i][2] *= f0; s.acc[i][3] *= f1;
        }
    }
    uint32_t w[3][2];                // pieces of the weights as the B operand
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        float p0 = exp2f(x[2 * n] - s.m), p1 = exp2f(x[2 * n + 1] - s.m);
        s.l += p0 + p1;
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
            uint32_t a[4];
            pair_tokens(a, (&p.v[0][f].x)[u], (&p.v[1][f].x)[u], (&p.v[2][f].x)[u], (&p.v[3][f].x)[u]);
            float c[4] = {};
#pragma unroll
            for (int k = 2; k >= 0; --k) mma_bf16(c, a[0], a[1], a[2], a[3], w[k][0], w[k][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) s.acc[4 * f + u][k] += c[k];
        }
}

// Infinite values. The three pieces of a weight cannot carry them: a zero piece makes NaN of an infinity, a negative
// one the opposite infinity, and so does a weight or a factor that has shrunk to zero. But an infinity always ends as
// itself or as NaN, and a NaN stays: where an output is one, the warps go over their pages again. This time only V's
// infinities and NaN enter, with weight one for every token that has a weight, and a sum other than zero is the output,
// whatever the finite values add. Without a NaN this costs a comparison an output and a vote: 1,344 tokens of 2 KV heads
// take 4.5 us with and without it on one card, 4.3 and 4.1 on another; longer sequences the same.

// Two bf16, zeros in place of finite ones.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
    return ((x & 0x7f80u) == 0x7f80u ? x & 0xffffu : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? x & 0xffff0000u : 0u);
}

// What one page of which the first `valid` tokens count adds to those sums, laid out as Gathered::acc.
template <int D>
__device__ __forceinline__ void odd_page(float (&sum)[D / 16][4], const uint4 (&q)[D / 32], const uint16_t* page, int valid,
                                         float scale_log2, int gid, int t) {
    Page<D> p;
    load_k<D>(p, page, gid, t);
    float x[4];
    page_logits<D>(x, q, p, scale_log2);
    const auto counts = [&](int n) { return 2 * t + (n & 1) + 8 * (n >> 1) < valid; };
    uint32_t w[2];                   // 1 where the token has a weight; 0 makes NaN of an infinity, as it should
#pragma unroll
    for (int n = 0; n < 2; ++n)
        w[n] = (counts(2 * n) && x[2 * n] > -INFINITY ? 0x3f80u : 0u) |
               (counts(2 * n + 1) && x[2 * n + 1] > -INFINITY ? 0x3f800000u : 0u);
    load_v<D>(p, page, gid, t);
#pragma unroll
    for (int f = 0; f < D / 64; ++f)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint32_t v[4], a[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) v[n] = counts(n) ? not_finite((&p.v[n][f].x)[u]) : 0u;
            pair_tokens(a, v[0], v[1], v[2], v[3]);
            mma_bf16(sum[4 * f + u], a[0], a[1], a[2], a[3], w[0], w[1]);
        }
}

// A CTA's W warps side by side in shared memory. Channel D / 8 i + j of a head lies at 8 j + i, rows are D + 4
// apart: a warp's lanes (gid, t) write 32 banks.
template <int D>
__device__ __forceinline__ int place(int c) { return c % (D / 8) * 8 + c / (D / 8); }
template <int D, int W>
struct WarpParts {
    float acc[W][8][D + 4];
    float m[W][8], l[W][8];
    float cta_m[8], cta_l[8];            // of the CTA, for its cluster; its accumulators replace acc[0]
    int odd;                             // an accumulator of the CTA, its warps joined, is not finite
};

template <int D, int W>
__device__ __forceinline__ void put_sums(WarpParts<D, W>& w, const float (&sum)[D / 16][4], int warp, int gid, int t) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)      // rows gid and gid + 8 of m-tile i are channels D / 8 gid + 2 i and + 1
            w.acc[warp][2 * t + (k & 1)][8 * (2 * i + (k >> 1)) + gid] = sum[i][k];
}

template <int D, int W>
__device__ __forceinline__ void put_warp(WarpParts<D, W>& w, const Gathered<D>& s, int warp, int gid, int t) {
    float l = s.l;
    l += __shfl_xor_sync(~0u, l, 1);
    l += __shfl_xor_sync(~0u, l, 2);
    if (t == 0) { w.m[warp][gid] = s.m; w.l[warp][gid] = l; }
    put_sums<D, W>(w, s.acc, warp, gid, t);
}

// The warps' parts of one output value joined: its reference, sum of weights and accumulator.
template <int D, int W>
__device__ __forceinline__ void join_warps(const WarpParts<D, W>& w, int head, int c, float& m, float& l, float& o) {
    m = w.m[0][head];
#pragma unroll
    for (int i = 1; i < W; ++i) m = fmaxf(m, w.m[i][head]);
    l = o = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float f = exp2f(w.m[i][head] - m);
        l += f * w.l[i][head];
        o += f * w.acc[i][head][place<D>(c)];
    }
}

// The warps' sums of a second way over the pages: 0, an infinity or NaN.
template <int D, int W>
__device__ __forceinline__ float odd_sum(const WarpParts<D, W>& w, int head, int c) {
    float o = 0.0f;
    for (int i = 0; i < W; ++i) o += w.acc[i][head][place<D>(c)];
    return o;
}

// The cluster's CTAs join their parts, each its share of the unit's g x D outputs, and write them. RANKS: CTAs of a
// cluster at most. All threads of the cluster call it after put_warp; `again` takes a warp over its pages a second
// time, up to put_sums.
template <int D, int W, int RANKS, typename G>
__device__ __forceinline__ void join_cluster(const AttendArgs& a, WarpParts<D, W>& w, int64_t row0, int rank, int ranks,
                                             G again) {
    if (threadIdx.x == 0) w.odd = 0;
    __syncthreads();
    for (int x = threadIdx.x; x < a.g * D; x += W * 32) {
        const int head = x / D, c = x % D;
        float m, l, o;
        join_warps<D, W>(w, head, c, m, l, o);
        w.acc[0][head][place<D>(c)] = o;                    // read by this thread alone so far
        if (c == 0) { w.cta_m[head] = m; w.cta_l[head] = l; }
        if (!(fabsf(o) < INFINITY)) w.odd = 1;
    }
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    cluster.sync();
    const int share = (a.g * D + ranks - 1) / ranks, end = min(a.g * D, (rank + 1) * share);
    for (int x = rank * share + threadIdx.x; x < end; x += W * 32) {
        const int head = x / D, c = x % D;
        float rm[RANKS], m = kNoLogit, l = 0.0f, o = 0.0f;
#pragma unroll
        for (int r = 0; r < RANKS; ++r) {
            rm[r] = r < ranks ? *cluster.map_shared_rank(&w.cta_m[head], r) : kNoLogit;
            m = fmaxf(m, rm[r]);
        }
#pragma unroll
        for (int r = 0; r < RANKS; ++r) {
            if (r >= ranks) continue;
            const float f = exp2f(rm[r] - m);
            l += f * *cluster.map_shared_rank(&w.cta_l[head], r);
            o += f * *cluster.map_shared_rank(&w.acc[0][head][place<D>(c)], r);
        }
        store_out(a, (row0 + head) * D + c, o, l);
    }
    const int lane = threadIdx.x & 31;
    const bool odd = __any_sync(~0u, lane < ranks && *cluster.map_shared_rank(&w.odd, lane < ranks ? lane : 0));
    cluster.sync();                                      // the other CTAs have read this one's memory
    if (!odd) return;
    again();
    cluster.sync();
    for (int x = rank * share + threadIdx.x; x < end; x += W * 32) {
        const int head = x / D, c = x % D;
        float o = 0.0f, l = 0.0f;
        for (int r = 0; r < ranks; ++r) {
            o += odd_sum(*cluster.map_shared_rank(&w, r), head, c);
            l += *cluster.map_shared_rank(&w.cta_l[head], r);      // 0, NaN: a head without weight, without result
        }
        if (o != 0.0f) store_out(a, (row0 + head) * D + c, o, l);
    }
    cluster.sync();
}

}  // namespace
}  // namespace oscar
