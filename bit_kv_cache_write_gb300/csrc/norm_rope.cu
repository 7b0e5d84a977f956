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
// heads of a token turn by the same angles, so a lane forms its four sines and cosines once a token, multiplies the
// norm's weights into them, and uses both for every head that its warp takes; two pairs go through one instruction
// (with the weights read and multiplied head by head the kernel was bound by its instructions: 433 us where it now takes
// 398). Four heads of a lane group in flight, CTAs of two warps, so that a token's warp leaves its place to another at
// once: 131,072 tokens x 40 heads of 128 in 399 us, 99 % of the measured copy rate (464 us with eight warps a CTA, 435
// with two heads in flight); 5,003 tokens x 72 heads of 64 in 12.7 us; single tokens 2.4 us.
#include "chunk_internal.h"
#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int kRopeThreads = 64;
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

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split_f32x2(uint64_t x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// A lane's four pairs (a, b), two at a time: a' = f (a aa - b ab), b' = f (b bb + a ba), with the norm's weights in the
// coefficients and f the head's reciprocal root; b' and a' alone where the lane's channels do not turn.
struct Turn {
    uint64_t aa[2], ab[2], ba[2], bb[2];

    __device__ __forceinline__ void set(const float* w, bool interleaved, int ca, int cb, bool turn, const float (&cs)[4],
                                        const float (&sn)[4]) {
        float wa[4] = {1, 1, 1, 1}, wb[4] = {1, 1, 1, 1};
        if (w) {
            const float4 x = *reinterpret_cast<const float4*>(w + ca), y = *reinterpret_cast<const float4*>(w + cb);
            wa[0] = x.x; wb[3] = y.w;
            wa[1] = interleaved ? x.z : x.y; wb[0] = interleaved ? x.y : y.x;
            wa[2] = interleaved ? y.x : x.z; wb[1] = interleaved ? x.w : y.y;
            wa[3] = interleaved ? y.z : x.w; wb[2] = interleaved ? y.y : y.z;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = 2 * j, l = 2 * j + 1;
            aa[j] = turn ? f32x2(wa[k] * cs[k], wa[l] * cs[l]) : f32x2(wa[k], wa[l]);
            bb[j] = turn ? f32x2(wb[k] * cs[k], wb[l] * cs[l]) : f32x2(wb[k], wb[l]);
            ab[j] = f32x2(-wb[k] * sn[k], -wb[l] * sn[l]);
            ba[j] = f32x2(wa[k] * sn[k], wa[l] * sn[l]);
        }
    }
};

// One batch of kRopeDepth heads a lane group: heads h0 + group, + kGroups, ... of a token's q or k heads.
template <int D, bool Interleaved>
struct RopeBatch {
    static constexpr int kLanes = D / 8;             // lanes of a head
    static constexpr int kGroups = 32 / kLanes;      // heads of a warp at once
    static constexpr int kHeads = kGroups * kRopeDepth;
    uint2 a[kRopeDepth], b[kRopeDepth];

    __device__ __forceinline__ void load(const RopeRows& r, int64_t t, int h0, int group, int ca, int cb) {
        const uint16_t* p = r.in + t * r.in_stride + (h0 + group) * D;
#pragma unroll
        for (int i = 0; i < kRopeDepth; ++i) {
            a[i] = b[i] = make_uint2(0, 0);
            if (h0 + i * kGroups + group < r.heads) {
                a[i] = *reinterpret_cast<const uint2*>(p + i * kGroups * D + ca);
                b[i] = *reinterpret_cast<const uint2*>(p + i * kGroups * D + cb);
            }
        }
    }
    __device__ __forceinline__ void finish(const RopeRows& r, float eps, int64_t t, int h0, int group, int ca, int cb, bool turn,
                                           const Turn& c) const {
        uint16_t* p = r.out + t * r.out_stride + (h0 + group) * D;
#pragma unroll
        for (int i = 0; i < kRopeDepth; ++i) {
            if (h0 + i * kGroups >= r.heads) break;          // none of the warp's
            // a's and b's of the pairs, two at a time
            uint64_t x[2], y[2];
            if (Interleaved) {
                x[0] = f32x2(bf16_lo(a[i].x), bf16_lo(a[i].y)); y[0] = f32x2(bf16_hi(a[i].x), bf16_hi(a[i].y));
                x[1] = f32x2(bf16_lo(b[i].x), bf16_lo(b[i].y)); y[1] = f32x2(bf16_hi(b[i].x), bf16_hi(b[i].y));
            } else {
                x[0] = f32x2(bf16_lo(a[i].x), bf16_hi(a[i].x)); x[1] = f32x2(bf16_lo(a[i].y), bf16_hi(a[i].y));
                y[0] = f32x2(bf16_lo(b[i].x), bf16_hi(b[i].x)); y[1] = f32x2(bf16_lo(b[i].y), bf16_hi(b[i].y));
            }
            float f = 1.0f;
            if (r.weight) {
                // sums from here on are right whatever their squares lost (or eps is above that)
                const float least = eps < 0x1p-60f ? D * 0x1p-60f : 0.0f;
                const uint32_t from = __float_as_uint(least), span = __float_as_uint(3.0e38f) - from;
                float lo, hi;
                split_f32x2(fma_f32x2(y[1], y[1], fma_f32x2(y[0], y[0], fma_f32x2(x[1], x[1], mul_f32x2(x[0], x[0])))), lo, hi);
                float ss = lo + hi;
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                f = rsqrtf(ss * (1.0f / D) + eps);
                if (__any_sync(0xffffffffu, __float_as_uint(ss) - from > span)) {       // not within [least, 3e38]
                    // The sum may have passed fp32, or its squares may be below it with an eps that does not hide that:
                    // the values in units of 2^72 or 2^-88, where neither is so. The root's unit goes to the values: the
                    // coefficients times it might not be a float.
                    const float unit = ss < least ? 0x1p88f : ss <= 3.0e38f ? 1.0f : 0x1p-72f;
                    const uint64_t by = f32x2(unit, unit);
                    uint64_t s = f32x2(0.0f, 0.0f);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint64_t u = mul_f32x2(x[k], by), v = mul_f32x2(y[k], by);
                        s = fma_f32x2(v, v, fma_f32x2(u, u, s));
                    }
                    split_f32x2(s, lo, hi);
                    float s2 = lo + hi;
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
                    if (unit != 1.0f) {
                        f = rsqrtf(s2 * (1.0f / D) + eps * unit * unit);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            x[k] = mul_f32x2(x[k], by);
                            y[k] = mul_f32x2(y[k], by);
                        }
                    }
                }
            }
            uint64_t u[2], v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                u[k] = mul_f32x2(x[k], c.aa[k]);
                v[k] = mul_f32x2(y[k], c.bb[k]);
                if (turn) {
                    u[k] = fma_f32x2(y[k], c.ab[k], u[k]);
                    v[k] = fma_f32x2(x[k], c.ba[k], v[k]);
                }
                if (r.weight) {
                    u[k] = mul_f32x2(u[k], f32x2(f, f));
                    v[k] = mul_f32x2(v[k], f32x2(f, f));
                }
            }
            float m[4], n[4];
            split_f32x2(u[0], m[0], m[1]); split_f32x2(u[1], m[2], m[3]);
            split_f32x2(v[0], n[0], n[1]); split_f32x2(v[1], n[2], n[3]);
            if (h0 + i * kGroups + group < r.heads) {
                uint16_t* to = p + i * kGroups * D;
                if (Interleaved) {
                    *reinterpret_cast<uint2*>(to + ca) = make_uint2(bf16_pair(m[0], n[0]), bf16_pair(m[1], n[1]));
                    *reinterpret_cast<uint2*>(to + cb) = make_uint2(bf16_pair(m[2], n[2]), bf16_pair(m[3], n[3]));
                } else {
                    *reinterpret_cast<uint2*>(to + ca) = make_uint2(bf16_pair(m[0], m[1]), bf16_pair(m[2], m[3]));
                    *reinterpret_cast<uint2*>(to + cb) = make_uint2(bf16_pair(n[0], n[1]), bf16_pair(n[2], n[3]));
                }
            }
        }
    }
};

// A warp takes `span` batches of heads of one token; `parts` warps take a token. Batches of q heads come first.
template <int D, bool Interleaved>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeArgs r, int parts, int span) {
    using B = RopeBatch<D, Interleaved>;
    const int lane = threadIdx.x % 32, group = lane / B::kLanes, l = lane % B::kLanes;
    const int64_t item = (int64_t)blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32;
    const int64_t t = item / parts;
    const int q_batches = (r.q.heads + B::kHeads - 1) / B::kHeads, all = q_batches + (r.k.heads + B::kHeads - 1) / B::kHeads;
    int at = (int)(item % parts) * span;
    const int end = min(all, at + span);
    const bool turn = 8 * l < r.rot;
    const int ca = Interleaved ? 8 * l : (turn ? 4 * l : 8 * l);
    const int cb = Interleaved ? ca + 4 : (turn ? r.rot / 2 + 4 * l : ca + 4);
    grid_wait();                             // the turns may be of the launch before too
    if (t >= r.n) return;
    uint64_t step[4] = {0, 0, 0, 0};
    if (turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) step[j] = r.turns[4 * l + j];
    }
    auto load = [&](B& b, int i) {
        if (i < q_batches)
            b.load(r.q, t, i * B::kHeads, group, ca, cb);
        else
            b.load(r.k, t, (i - q_batches) * B::kHeads, group, ca, cb);
    };
    B now;
    load(now, at);
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
    Turn c;
    c.set(at < q_batches ? r.q.weight : r.k.weight, Interleaved, ca, cb, turn, cs, sn);
    for (;;) {
        B ahead;
        if (at + 1 < end) load(ahead, at + 1);
        if (at < q_batches)
            now.finish(r.q, r.eps, t, at * B::kHeads, group, ca, cb, turn, c);
        else
            now.finish(r.k, r.eps, t, (at - q_batches) * B::kHeads, group, ca, cb, turn, c);
        if (++at >= end) break;
        now = ahead;
        if (at == q_batches) c.set(r.k.weight, Interleaved, ca, cb, turn, cs, sn);
    }
}

template <int D>
cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t st) {
    using B = RopeBatch<D, false>;
    const int batches = (a.q.heads + B::kHeads - 1) / B::kHeads + (a.k.heads + B::kHeads - 1) / B::kHeads;
    // A warp takes a batch of heads while that gives no more warps than run at once (256 tokens x 40 heads: 3.5 us, more
    // than twice that with a token a warp), else a whole token's heads (131,072: 398 us, half as much again with a batch
    // a warp).
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
