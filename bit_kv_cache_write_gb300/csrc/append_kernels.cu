// New K/V rows into the BF16 pool, and the key bounds of their pages (oscar_append_bf16).
//
// A row is a copy of 2 d bytes. The bounds of a (page, KV head) are, per channel, the least and the largest
// of the keys' codes clamp(rint(k 2^-step), -127, 127). The code is monotone in k, so the minimum and maximum
// are taken over the bf16 keys of a run (adjacent tokens of one page), with packed bf16 instructions, and
// only the two results are turned into codes.
//
// A unit of 2 d / 8 lanes takes the runs that begin in its tokens, one KV head each: half of its lanes move
// K, the other half V, 16 bytes a lane. A run has one owner, so bounds need no atomics.
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

template <int D, bool BOUNDS>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a, int tokens_per_unit) {
    constexpr int kHalf = D / 8;                     // lanes that move one row of K (or V)
    constexpr int kUnit = 2 * kHalf;
    grid_wait();
    const long long unit = ((long long)blockIdx.x * kAppendThreads + threadIdx.x) / kUnit;
    const int lane = threadIdx.x % kUnit, part = lane / kHalf, c0 = lane % kHalf * 8;
    const int h = (int)(unit % a.h_kv);
    const long long i0 = unit / a.h_kv * tokens_per_unit;
    if (i0 >= a.n) return;
    const long long i1 = min(i0 + tokens_per_unit, (long long)a.n);
    const uint16_t* src = (part ? a.v : a.k) + (long long)h * D + c0;
    const int64_t src_stride = part ? a.v_stride : a.k_stride;
    const long long limit = a.pages * kPage;
    // The slot's page, or -1 for a token that is skipped.
    auto page_of = [&](long long i, long long& slot) -> long long {
        slot = a.slots[i];
        if (slot >= 0 && slot < limit) return slot / kPage;
        if (slot >= limit && a.debug) record_error(&a.dbg->kind, &a.dbg->index, 1, slot);
        return -1;
    };
    auto row_at = [&](long long page, long long slot) {
        return a.pool + (((page * a.h_kv + h) * 2 + part) * kPage + slot % kPage) * D + c0;
    };
    long long i = i0, slot;
    if (!BOUNDS) {
        for (; i < i1; ++i) {
            const long long page = page_of(i, slot);
            if (page >= 0)
                *reinterpret_cast<uint4*>(row_at(page, slot)) = ldg_stream(src + i * src_stride);
        }
        return;
    }
    if (i > 0) {                                     // the run that reaches into these tokens has its owner
        const long long before = page_of(i - 1, slot);
        while (i < i1 && before >= 0 && page_of(i, slot) == before) ++i;
    }
    while (i < i1) {
        const long long page = page_of(i, slot);
        if (page < 0) { ++i; continue; }
        bool fresh = false;
        uint32_t lo[4], hi[4];
        for (int first = 1; i < a.n; ++i, first = 0) {
            if (!first && page_of(i, slot) != page) break;
            fresh |= slot % kPage == 0;
            const uint4 x = ldg_stream(src + i * src_stride);
            *reinterpret_cast<uint4*>(row_at(page, slot)) = x;
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t z = bf2_no_nan(w[j]);
                lo[j] = first ? z : bf2_min(lo[j], z);
                hi[j] = first ? z : bf2_max(hi[j], z);
            }
        }
        if (part == 0) {
            int8_t* b = a.bounds + ((page * a.h_kv + h) * 2) * D + c0;
            const int8_t* steps = a.steps + h * D + c0;
            uint32_t word[2][2] = {};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float inv = inv_pow2(steps[c]);
                const int shift = 16 * (c & 1);
                int l = code_of(lo[c / 2] >> shift & 0xffffu, inv), u = code_of(hi[c / 2] >> shift & 0xffffu, inv);
                if (!fresh) { l = min(l, (int)b[c]); u = max(u, (int)b[D + c]); }
                word[0][c / 4] |= (uint32_t)(l & 0xff) << (8 * (c & 3));
                word[1][c / 4] |= (uint32_t)(u & 0xff) << (8 * (c & 3));
            }
            *reinterpret_cast<uint2*>(b) = make_uint2(word[0][0], word[0][1]);
            *reinterpret_cast<uint2*>(b + D) = make_uint2(word[1][0], word[1][1]);
        }
    }
}

template <int D>
cudaError_t launch(const AppendArgs& a, int num_sms, cudaStream_t st) {
    const int tokens = 1;
    const long long units = ((long long)a.n + tokens - 1) / tokens * a.h_kv;
    const long long ctas = (units * (2 * D / 8) + kAppendThreads - 1) / kAppendThreads;
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
