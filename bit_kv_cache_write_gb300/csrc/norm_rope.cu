// Norm and rotation of new queries and keys (oscar_norm_rope).
//
// Per head x of d channels: y = w x / sqrt(mean(x^2) + eps) (y = x without weights), then pairs (a, b) of the first
// `rot` channels turn by the angle of their token's position p:
//   (a', b') = scale (a cos t - b sin t, b cos t + a sin t),   t = 2 pi frac(p * turn_i).
// turn_i is a 64-bit fixed-point fraction of a turn, so the integer product p * turn_i mod 2^64 is the angle's exact
// remainder however far the position, and one conversion to fp32 is its only rounding. Everything between the bf16
// loads and the bf16 store is fp32; each output is rounded once.
//
// HBM bounds it: each channel is read and written once. d / 8 lanes take a head, 8 channels a lane: the four pairs
// 4 l .. 4 l + 3 (channels 4 l .. and rot / 2 + 4 l .., or 8 l ..), and the lanes behind rot / 8 pass 8 channels on. All
// heads of a token turn by the same angles, so a lane forms its four sines and cosines once a token and uses them
// for every head that its warp takes. Four heads of a lane group in flight and CTAs of four warps: 131,072 tokens x 40
// heads of 128 in 433 us, 92 % of the measured copy rate (449 us with eight warps a CTA, 660 with eight heads in flight),
// 5,003 tokens x 72 heads of 64 in 14.8 us, 95 %; single tokens 3 us.
#include "chunk_internal.h"
#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeDepth = 4;                // heads that a lane group has in flight

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The request of row t: the last b with row_start[b] <= t, or -1 where t is in front of the first or behind the last
// request. All lanes of the warp call it with one t and probe 32 starts a round.
__device__ __forceinline__ int request_of(const int32_t* row_start, int batch, int t, int lane) {
    if (t < row_start[0] || t >= row_start[batch]) return -1;
    int lo = 0, n = batch;                   // row_start[lo] <= t < row_start[lo + n]
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + min((lane + 1) * step, n);
        const uint32_t above = __ballot_sync(0xffffffffu, row_start[at] > t);
        const int first = above ? __ffs(above) - 1 : 31;
        lo += first * step;
        n = min(step, n - first * step);
        if (n < 1) return batch - 1;         // starts that do not ascend
    }
    return lo;
}

// One batch of kRopeDepth heads a lane group: heads h0 + group, + kGroups, ... of the token's q heads, then k heads.
template <int D, bool Interleaved>
struct RopeBatch {
    static constexpr int kLanes = D / 8;             // lanes of a head
    static constexpr int kGroups = 32 / kLanes;      // heads of a warp at once
    static constexpr int kHeads = kGroups * kRopeDepth;
    uint2 a[kRopeDepth], b[kRopeDepth];

    __device__ __forceinline__ static const uint16_t* source(const RopeArgs& r, int64_t t, int h) {
        return h < r.q.heads ? r.q.in + t * r.q.in_stride + h * D : r.k.in + t * r.k.in_stride + (h - r.q.heads) * D;
    }
    __device__ __forceinline__ void load(const RopeArgs& r, int64_t t, int h0, int group, int ca, int cb) {
#pragma unroll
        for (int i = 0; i < kRopeDepth; ++i) {
            const int h = h0 + i * kGroups + group;
            if (h < r.q.heads + r.k.heads) {
                const uint16_t* p = source(r, t, h);
                a[i] = *reinterpret_cast<const uint2*>(p + ca);
                b[i] = *reinterpret_cast<const uint2*>(p + cb);
            } else {
                a[i] = b[i] = make_uint2(0, 0);
            }
        }
    }
    __device__ __forceinline__ void finish(const RopeArgs& r, int64_t t, int h0, int group, int ca, int cb, bool turn,
                                           const float (&cs)[4], const float (&sn)[4]) const {
#pragma unroll
        for (int i = 0; i < kRopeDepth; ++i) {
            const int h = h0 + i * kGroups + group;
            const bool mine = h < r.q.heads + r.k.heads, is_q = h < r.q.heads;
            float x[8] = {bf16_lo(a[i].x), bf16_hi(a[i].x), bf16_lo(a[i].y), bf16_hi(a[i].y),
                          bf16_lo(b[i].x), bf16_hi(b[i].x), bf16_lo(b[i].y), bf16_hi(b[i].y)};
            const float* w = is_q ? r.q.weight : r.k.weight;
            if (r.q.weight || r.k.weight) {          // the same branch for all lanes: they sum together
                float ss = 0.0f;
#pragma unroll
                for (int c = 0; c < 8; ++c) ss += x[c] * x[c];
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                float f = rsqrtf(ss * (1.0f / D) + r.eps);
                if (__any_sync(0xffffffffu, !(ss <= 3.0e38f))) {     // the sum may have passed fp32: in units of 2^64
                    float s2 = 0.0f;
#pragma unroll
                    for (int c = 0; c < 8; ++c) s2 += (x[c] * 0x1p-64f) * (x[c] * 0x1p-64f);
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
                    if (!(ss <= 3.0e38f)) f = rsqrtf(s2 * (1.0f / D) + r.eps * 0x1p-128f) * 0x1p-64f;
                }
                if (w) {
                    const float4 wa = *reinterpret_cast<const float4*>(w + ca), wb = *reinterpret_cast<const float4*>(w + cb);
                    x[0] *= f * wa.x; x[1] *= f * wa.y; x[2] *= f * wa.z; x[3] *= f * wa.w;
                    x[4] *= f * wb.x; x[5] *= f * wb.y; x[6] *= f * wb.z; x[7] *= f * wb.w;
                }
            }
            if (turn) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int ia = Interleaved ? 2 * j : j, ib = Interleaved ? 2 * j + 1 : 4 + j;
                    const float u = x[ia], v = x[ib];
                    x[ia] = u * cs[j] - v * sn[j];
                    x[ib] = v * cs[j] + u * sn[j];
                }
            }
            if (mine) {
                uint16_t* p = is_q ? r.q.out + t * r.q.out_stride + h * D
                                   : r.k.out + t * r.k.out_stride + (h - r.q.heads) * D;
                *reinterpret_cast<uint2*>(p + ca) = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
                *reinterpret_cast<uint2*>(p + cb) = make_uint2(bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
            }
        }
    }
};

// A warp takes `span` batches of heads of one token; `parts` warps take a token.
template <int D, bool Interleaved>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeArgs r, int parts, int span) {
    using B = RopeBatch<D, Interleaved>;
    const int lane = threadIdx.x % 32, group = lane / B::kLanes, l = lane % B::kLanes;
    const int64_t item = (int64_t)blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32;
    const int64_t t = item / parts;
    const int heads = r.q.heads + r.k.heads;
    int h0 = (int)(item % parts) * span * B::kHeads;
    const int end = min(heads, h0 + span * B::kHeads);
    const bool turn = 8 * l < r.rot;
    const int ca = Interleaved ? 8 * l : (turn ? 4 * l : 8 * l);
    const int cb = Interleaved ? ca + 4 : (turn ? r.rot / 2 + 4 * l : ca + 4);
    uint64_t step[4] = {0, 0, 0, 0};
    if (turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) step[j] = r.turns[4 * l + j];
    }
    grid_wait();
    if (t >= r.n) return;
    B now;
    now.load(r, t, h0, group, ca, cb);
    int64_t pos = 0;
    if (r.positions) {
        pos = r.positions[t];
    } else if (r.batch > 0) {
        const int b = request_of(r.row_start, r.batch, (int)t, lane);
        if (b < 0) return;
        pos = (int64_t)r.total_len[b] - r.row_start[b + 1] + t;
    } else {
        return;
    }
    float cs[4], sn[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // half turns in [-1, 1): the angle over pi
        const float x = (float)(int64_t)(step[j] * (uint64_t)pos) * 0x1p-63f;
        sincospif(x, &sn[j], &cs[j]);
        cs[j] *= r.scale;
        sn[j] *= r.scale;
    }
    for (;;) {
        const int next = h0 + B::kHeads;
        B ahead;
        if (next < end) ahead.load(r, t, next, group, ca, cb);
        now.finish(r, t, h0, group, ca, cb, turn, cs, sn);
        if (next >= end) break;
        now = ahead;
        h0 = next;
    }
}

template <int D>
cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t st) {
    using B = RopeBatch<D, false>;
    const int batches = (a.q.heads + a.k.heads + B::kHeads - 1) / B::kHeads;
    // A warp takes a batch of heads while that gives no more warps than run at once (256 tokens x 40 heads: 4.4 us, 9.6
    // with a token a warp), else a whole token's heads (131,072: 449 us, 658 with a batch a warp).
    const bool spread = (int64_t)a.n * batches <= (int64_t)num_sms * 32;
    const int parts = spread ? batches : 1, span = spread ? 1 : batches;
    const int64_t warps = (int64_t)a.n * parts, per = kRopeThreads / 32;
    return launch_dependent(a.interleaved ? norm_rope_kernel<D, true> : norm_rope_kernel<D, false>,
                            dim3((unsigned)((warps + per - 1) / per)), dim3(kRopeThreads), 0, st, 1, a, parts, span);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a, int d, int num_sms, cudaStream_t st) {
    return d == 128 ? launch_rope<128>(a, num_sms, st) : launch_rope<64>(a, num_sms, st);
}

}  // namespace oscar
