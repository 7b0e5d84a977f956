// New K/V rows into the BF16 pool, and the key bounds of their pages (oscar_append_bf16).
//
// A row is a copy of 2 d bytes. The bounds of a (page, KV head) are, per channel, the least and the largest
// of the keys' codes clamp(rint(k 2^-step), -127, 127). The code is monotone in k, so the minimum and maximum
// are taken over the bf16 keys of a run (adjacent tokens of one page), with packed bf16 instructions, and
// only the two results are turned into codes.
//
// A warp takes a few adjacent tokens of one KV head (two at d = 64): half of a head's lanes move K, the other
// half V, 16 bytes a lane, four rows at once. With bounds it takes the runs that begin in its tokens, to
// their end, so that a run has one owner and needs no atomics. The kernel does not let its successor start
// early: a decode prefetches pages.
//
// HBM bounds it: 131,072 tokens of 8 heads (d = 128) with bounds in 165 us, 97 % of the measured copy rate; 256
// single tokens take 1.9 us, a launch and two dependent loads.
#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t bf2_min(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// NaN keys count as zero in the bounds.
__device__ __forceinline__ uint32_t bf2_no_nan(uint32_t a) {
    const uint32_t lo = (a & 0x7fffu) > 0x7f80u ? 0u : a & 0xffffu;
    const uint32_t hi = (a & 0x7fff0000u) > 0x7f800000u ? 0u : a & 0xffff0000u;
    return lo | hi;
}
__device__ __forceinline__ int code_of(uint32_t bf16_bits, float inv_step) {
    const float x = __uint_as_float(bf16_bits << 16) * inv_step;
    return __float2int_rn(fminf(fmaxf(x, -127.0f), 127.0f));
}

// 2^-step, exactly; steps beyond +-100 count as that.
__device__ __forceinline__ float inv_pow2(int step) {
    return __int_as_float((127 - max(-100, min(100, step))) << 23);
}

// Widens a page's bounds of eight channels (old_lo and old_hi; none where the run begins the page) by a run's
// least and largest keys and writes them.
template <int D>
__device__ __forceinline__ void write_bounds(int8_t* b, uint2 steps, const uint32_t (&lo)[4], const uint32_t (&hi)[4],
                                             uint2 old_lo, uint2 old_hi) {
    uint32_t word[2][2] = {};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int at = 8 * (c & 3), half = 16 * (c & 1);
        const float inv = inv_pow2((int8_t)((c < 4 ? steps.x : steps.y) >> at));
        const int l = min(code_of(lo[c / 2] >> half & 0xffffu, inv), (int)(int8_t)((c < 4 ? old_lo.x : old_lo.y) >> at));
        const int u = max(code_of(hi[c / 2] >> half & 0xffffu, inv), (int)(int8_t)((c < 4 ? old_hi.x : old_hi.y) >> at));
        word[0][c / 4] |= (uint32_t)(l & 0xff) << at;
        word[1][c / 4] |= (uint32_t)(u & 0xff) << at;
    }
    *reinterpret_cast<uint2*>(b) = make_uint2(word[0][0], word[0][1]);
    *reinterpret_cast<uint2*>(b + D) = make_uint2(word[1][0], word[1][1]);
}

template <int D, bool BOUNDS>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(AppendArgs a, int tokens) {
    constexpr int kHalf = D / 8;                     // lanes that move one row of K (or V)
    constexpr int kHeads = 32 / (2 * kHalf);         // KV heads of a warp
    constexpr int kRows = 4;                         // rows in flight per lane (131,072 tokens: 165 us; with 8 189, with 16 253)
    grid_wait();
    const int lane = threadIdx.x & 31;
    const int groups = (a.h_kv + kHeads - 1) / kHeads;
    const long long unit = ((long long)blockIdx.x * kAppendThreads + threadIdx.x) / 32;
    const int h = (int)(unit % groups) * kHeads + lane / (2 * kHalf);
    const int part = lane / kHalf % 2, c0 = lane % kHalf * 8;
    const long long i0 = unit / groups * tokens;
    if (i0 >= a.n) return;

    // Lane l holds the page and the row of token i0 - 1 + l, page -1 where there is none to write.
    const long long i = i0 - 1 + lane;
    const int64_t slot = i >= 0 && i < a.n ? a.slots[i] : -1;
    const bool real = slot >= 0 && slot < a.pages * kPage;
    if (slot >= a.pages * kPage && a.debug) record_error(&a.dbg->kind, &a.dbg->index, 1, slot);
    const int page = real ? (int)(slot / kPage) : -1, row = (int)(slot % kPage);
    const int before = __shfl_up_sync(~0u, page, 1);
    const uint32_t live = __ballot_sync(~0u, real) & ~1u;                     // tokens that are written
    uint32_t starts = __ballot_sync(~0u, real && page != before) & ~1u;       // that begin a run
    const uint32_t own = (1u << (tokens + 1)) - 2;                            // that are this warp's
    if (!BOUNDS) starts = live;                                               // each token for itself
    const bool active = h < a.h_kv;
    const uint16_t* src = (part ? a.v : a.k) + (i0 - 1) * (part ? a.v_stride : a.k_stride) + (int64_t)(active ? h : 0) * D + c0;
    const int64_t stride = part ? a.v_stride : a.k_stride;
    uint16_t* dst = a.pool + ((int64_t)(active ? h : 0) * 2 + part) * kPage * D + c0;

    if (!BOUNDS) {
        for (uint32_t todo = starts & own; todo;) {
            uint4 x[kRows];
            uint16_t* to[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int l = todo ? __ffs(todo) - 1 : 0;
                to[k] = nullptr;
                const int p = __shfl_sync(~0u, page, l), r = __shfl_sync(~0u, row, l);
                if (todo && active) {
                    to[k] = dst + (int64_t)p * a.h_kv * 2 * kPage * D + r * D;
                    x[k] = ldg_stream(src + l * stride);
                }
                todo &= todo - 1;
            }
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                if (to[k]) *reinterpret_cast<uint4*>(to[k]) = x[k];
        }
        return;
    }
    const bool keeps = part == 0 && active;
    const uint2 steps = keeps ? *reinterpret_cast<const uint2*>(a.steps + h * D + c0) : make_uint2(0, 0);
    const uint2 none_lo = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu), none_hi = make_uint2(0x81818181u, 0x81818181u);
    const uint32_t ends = live & ~((live & ~starts) >> 1);                    // tokens that end a run
    uint32_t todo = starts & own;
    if ((todo & ends) == (live & own)) {             // each token a run (a decode step): two at a time
        while (todo) {
            int8_t* b[2];
            uint4 x[2];
            uint2 old_lo[2], old_hi[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int l = todo ? __ffs(todo) - 1 : 0;
                const int p = __shfl_sync(~0u, page, l), r = __shfl_sync(~0u, row, l);
                b[k] = nullptr;
                if (todo && active) {
                    x[k] = ldg_stream(src + l * stride);
                    b[k] = a.bounds + ((int64_t)p * a.h_kv + h) * 2 * D + c0;
                    old_lo[k] = none_lo;
                    old_hi[k] = none_hi;
                    if (keeps && r) {
                        old_lo[k] = *reinterpret_cast<const uint2*>(b[k]);
                        old_hi[k] = *reinterpret_cast<const uint2*>(b[k] + D);
                    }
                    *reinterpret_cast<uint4*>(dst + (int64_t)p * a.h_kv * 2 * kPage * D + r * D) = x[k];
                }
                todo &= todo - 1;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (b[k] && keeps) {
                    const uint32_t z[4] = {bf2_no_nan(x[k].x), bf2_no_nan(x[k].y), bf2_no_nan(x[k].z), bf2_no_nan(x[k].w)};
                    write_bounds<D>(b[k], steps, z, z, old_lo[k], old_hi[k]);
                }
        }
        return;
    }
    for (; todo; todo &= todo - 1) {
        const int first = __ffs(todo) - 1;
        // the run's tokens: up to the next one that begins another run or is not written
        const uint32_t stop = (starts | ~live) & ~((2u << first) - 1);
        const int end = stop ? __ffs(stop) - 1 : 32;
        const int p = __shfl_sync(~0u, page, first);
        uint16_t* to = dst + (int64_t)p * a.h_kv * 2 * kPage * D;
        const bool fresh = __any_sync(~0u, lane >= first && lane < end && row == 0);
        int8_t* b = a.bounds + ((int64_t)p * a.h_kv + (active ? h : 0)) * 2 * D + c0;
        uint32_t lo[4], hi[4];
        for (int l0 = first; l0 < end; l0 += kRows) {
            uint4 x[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                if (l0 + k < end && active) x[k] = ldg_stream(src + (l0 + k) * stride);
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int r = __shfl_sync(~0u, row, l0 + k);
                if (l0 + k >= end || !active) continue;
                *reinterpret_cast<uint4*>(to + r * D) = x[k];
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t z = bf2_no_nan(w[j]);
                    lo[j] = l0 + k == first ? z : bf2_min(lo[j], z);
                    hi[j] = l0 + k == first ? z : bf2_max(hi[j], z);
                }
            }
        }
        if (keeps) {
            const uint2 old_lo = fresh ? none_lo : *reinterpret_cast<const uint2*>(b);
            const uint2 old_hi = fresh ? none_hi : *reinterpret_cast<const uint2*>(b + D);
            write_bounds<D>(b, steps, lo, hi, old_lo, old_hi);
        }
    }
}

template <int D>
cudaError_t launch(const AppendArgs& a, int num_sms, cudaStream_t st) {
    constexpr int kHeads = 32 / (D / 4);
    const int groups = (a.h_kv + kHeads - 1) / kHeads;
    // One token a warp while those warps fit on the card about once, 16 (a page) beyond. Eight heads: 256 single rows
    // with bounds 2.3 us against 8.1 with 16, 4,864 17.5 and 14.0; without bounds 1.8 and 3.5, 9.2 and 4.9. In between
    // either may lose: 1,216 tokens of one request 8.4 and 6.2 us, 2,432 single rows 9.2 and 10.5.
    const int tokens = (long long)a.n * groups <= 64LL * num_sms ? 1 : kPage;
    const long long warps = ((long long)a.n + tokens - 1) / tokens * groups;
    const long long ctas = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)ctas), block(kAppendThreads);
    return a.bounds ? launch_dependent(append_kernel<D, true>, grid, block, 0, st, 1, a, tokens)
                    : launch_dependent(append_kernel<D, false>, grid, block, 0, st, 1, a, tokens);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int d, int num_sms, cudaStream_t st) {
    return d == 128 ? launch<128>(a, num_sms, st) : launch<64>(a, num_sms, st);
}

}  // namespace oscar
