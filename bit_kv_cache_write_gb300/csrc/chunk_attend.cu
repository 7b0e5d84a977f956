// Attention of chunks of new tokens over a paged BF16 cache (oscar_extend_bf16).
//
//   out_i = sum_t w_t v_t / sum_t w_t,  w_t = 2^(c q_i.k_t - m),  t <= pos_i,  c = sm_scale log2(e)
// with a running reference m that is raised only when a logit passes it by 2^8 (the lazy online softmax of the
// decodes). The query rows of a (request, KV head) are its tokens times the g heads of the group, token by token, so
// that the group's heads share every K and V tile.
//
// One CTA an SM takes work items: 256 query rows (two blocks of 128) against a range of 128-token tiles of the cache.
//   warp 8      loads: K and V pages through TMA (page ids looked up four tiles at a time), 128-byte swizzle;
//   warp 9      issues tcgen05.mma: S = Q K^T (128 x 128 x d) into tensor memory, O += P V with P read from tensor
//               memory; at d = 128 a block's next S is issued behind its P V, so the softmax of one block runs under
//               the matrix products of the other, at d = 64 as soon as the last S is in registers;
//   warps 0..7  one warp group a block, a thread a row: the row's 128 logits in registers, weights rounded to bf16
//               over the logits' own columns or beside them, O scaled only where the reference rises.
// At d = 128 logits and outputs of two blocks are all of tensor memory (512 columns): P has to lie over S, and a block's
// next S to wait for its P V; at d = 64 there is room for P beside it. The weights' rounding to bf16 is the operand type
// of the product (a second piece would cost half again of the tensor time that bounds long prompts); their sum is of the
// unrounded ones, in fp32.
//
// What bounds it (32 query and 8 KV heads of 128 on one GB300): long prompts the tensor cores and the power, 8,192 tokens
// in 345 us in a graph of a few passes = 1.59 PFLOP/s, 84 % of the measured rate of a large matrix product, and 369 to 375
// in a loop of calls, where the card is at its power limit (77 %); the softmax of a block takes 1,250 cycles a tile, its
// two products 1,024, of two blocks' 2,048. At d = 64 (257 us) the softmax, of which two blocks share the ex2
// (1,024 cycles) and all else. Few rows HBM: 1 to 8 tokens of 32 requests of 4k to 32k in 280 us = 6.5 TB/s, 97 % of the
// measured copy rate; a lone row block (8 tokens at 100,000, 74 us) 82 %, by the parts' writing and join and the items'
// starts. Short ones the chain of launch, plan, loads, softmax and join: 11 us.
//
// Items of requests with long caches and few rows are cut along the cache, by a plan from the lengths on the device, so
// that the items fill the SMs evenly: for few row blocks every loader plans for itself, for many chunk_plan_kernel does;
// chunk_join_kernel adds the parts of cut items.
//
// A weight of 0 does not undo an infinity or NaN in the value of a token that a row must not see (0 x inf): rows whose
// accumulator is not finite are marked, and chunk_join_kernel looks at them again, with the tokens that they see alone.
//
// Every wait is bounded: a role that gives up records kind 4 and sets a flag, the others stop, copies and matrix
// products in flight are waited for (bounded too), tensor memory is freed.
#include <cudaTypedefs.h>

#include "chunk_internal.h"
#include "paged_device.cuh"
#include "tc_device.cuh"

namespace oscar {
namespace {

constexpr int kBlock = 128;                      // query rows of a block
constexpr int kTilePages = kChunkTile / kPage;
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = 384;                    // two softmax warp groups, one of loader and issuer
constexpr int kItemRing = 4;                     // items that the loader may be ahead with the others
constexpr int kMaskRing = 16;                    // tiles whose page masks are kept: more than the loader is ahead
constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;
constexpr int kSelfUnits = 80;                   // row blocks and requests up to which each loader plans for itself
constexpr int kJoinThreads = 256;
constexpr float kNoReference = -3.402823466e38f; // reference before any token: no finite logit is below it
constexpr float kHeadroom = 8.0f;                // the reference rises when a logit passes it by this much (log2)
constexpr int kFold = 512;                       // tiles whose products the tensor core adds up (see Fold)

// A work item: rows r0 .. r0 + rows of request b's row space against cache tiles [kv0, kv1).
struct alignas(16) Item {
    int b, head, tok0, r0;        // tok0: the request's first row of q
    int rows, pos0, kv0, kv1;     // pos0: position of the request's first new token (below 0 where it has no room)
    int total, part, piece, pieces;   // part: first row of its partial results, or -1
    // its number, and how far the next piece's is; piece p's parts begin p * step rows behind piece 0's, which lie `lead`
    // rows further
    int self, stride, step, lead;
};
static_assert(sizeof(Item) == 64, "copied as four words of 16 bytes");

struct Header {
    int items, next;              // next: item after the CTAs' first ones
    int cut;                      // whether any item is
};

struct Work {
    int self, sms;                // each CTA's loader plans for itself, for this many
    int unit_cap, item_cap, part_cap;     // as in ChunkPlan
    Header* head;
    int* tiles;                   // [batch + 1] first row block of each request
    int2* units;                  // per row block: request, cache tiles and rows (unit_word)
    Item* items;
    uint32_t* odd;                // [items][8] rows to look at again, a word for each softmax warp
    int* marked;                  // [SMs] whether a CTA has marked any
    float2* part_ml;              // per row of a cut item: reference and sum
    float* part_acc;              // [rows][d]
    int fold_rows;                // of a CTA
    float2* fold_ml;              // [SMs][fold_rows] the same of what the tensor core no longer holds (see Fold)
    float* fold_acc;              // [SMs][fold_rows][d]
};

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// The request's rows of q and the position of its first new token.
struct Request {
    int tok0, count, total, pos0;
};
__device__ __forceinline__ Request request(const ChunkArgs& a, int b) {
    Request r;
    r.tok0 = clamp_int(a.row_start[b], 0, a.n);
    r.count = clamp_int(a.row_start[b + 1], r.tok0, a.n) - r.tok0;
    r.total = checked_len(a.total_len[b], a.stride * kPage, a.debug, a.dbg);
    r.pos0 = r.total - r.count;
    return r;
}

// Cached tokens that row r of a request's row space sees.
__device__ __forceinline__ int limit_of(int r, int pos0, int g_log2) { return max(pos0 + (r >> g_log2) + 1, 0); }

// ---- plan ---------------------------------------------------------------------------------------------------

// Exclusive sum over the block; every thread gets the total too.
__device__ int block_scan(int x, int* shared, int& total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) shared[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int w = shared[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        shared[lane] = w;
    }
    __syncthreads();
    total = shared[31];
    return s - x + (warp ? shared[warp - 1] : 0);
}

// The last i in [0, n) with at[i] <= x; at[0] <= x.
__device__ __forceinline__ int last_at_most(const int* at, int n, int x) {
    int lo = 0;
    while (n > 1) {
        const int half = n / 2;
        if (at[lo + half] <= x) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

// Cutting every row block's tiles into pieces of at most L gives items whose time on `sms` SMs is at most
// min(waves * (L + s), all / sms + L + s), s the cost of starting an item, and parts whose rows are written and read
// again. The i-th L that a plan looks at: an SM's share of all tiles times 2^(1 - i / 15), the last one without a cut. A
// cut item costs its share of the join, hence no L below half an SM's share.
constexpr int kStart = 3;                        // tiles' worth of starting an item
constexpr float kJoined = 1.0f / 65536;          // tiles' worth of a part's element
__device__ __forceinline__ int piece_length(int i, int share, int longest) {
    return i == 31 ? max(longest, 1) : max(1, (int)ceilf((float)share * exp2f(1.0f - (float)i / 15.0f)));
}
__device__ __forceinline__ int pieces_of(int tiles, int len) { return max(1, (tiles + len - 1) / len); }
// The same for what a plan costs, by 1 / len: exact below 2^21 tiles, one off at most beyond.
__device__ __forceinline__ int about_pieces(int tiles, int len, float inv) { return max(1, (int)(((float)(tiles + len - 1) + 0.5f) * inv)); }
__device__ __forceinline__ float cost_of(int pieces, int parts, int len, float all, const ChunkArgs& a, int sms) {
    const float one = (float)(len + kStart);
    return fminf((float)((pieces + sms - 1) / sms) * one, (all + (float)kStart * (float)pieces) / (float)sms + one) +
           (float)parts * (float)a.d * kJoined;
}
// An SM's share of all tiles, a tile more at most.
__device__ __forceinline__ int share_of(float all, int sms) { return (int)(all / (float)sms) + 1; }

// The lane with the least cost, of equal ones the last: the one with the longest pieces, or without a cut.
__device__ __forceinline__ int cheapest(float cost, int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, cost, o);
        const int where = __shfl_xor_sync(0xffffffffu, lane, o);
        if (other < cost || (other == cost && where > lane)) {
            cost = other;
            lane = where;
        }
    }
    return lane;
}

// A row block's tiles (at most 2^23: 24 bits) and rows less one (8 bits) in a word.
__device__ __forceinline__ int unit_word(const Request& r, int block, int g, int g_log2) {
    const int rows = min(kChunkRows, r.count * g - block * kChunkRows);
    const int tiles = (limit_of(block * kChunkRows + rows - 1, r.pos0, g_log2) + kChunkTile - 1) / kChunkTile;
    return (int)((unsigned)(rows - 1) << 24) | tiles;
}
__device__ __forceinline__ int tiles_of(int word) { return word & 0xffffff; }
__device__ __forceinline__ int rows_of(int word) { return (int)((unsigned)word >> 24) + 1; }

// A row block: `block` of request b.
struct Unit {
    int b, block, word, tok0, pos0, total;
};
// Piece rest / H_kv of head rest % H_kv of a row block in p pieces; part: first row of its parts.
__device__ __forceinline__ Item item_of(const ChunkArgs& a, const Unit& u, int p, int rest, int part, int part_cap, int self) {
    Item it{};
    const int tiles = tiles_of(u.word);
    it.b = u.b;
    it.head = rest % a.h_kv;
    it.tok0 = u.tok0;
    it.r0 = u.block * kChunkRows;
    it.rows = rows_of(u.word);
    it.pos0 = u.pos0;
    it.piece = rest / a.h_kv;
    it.pieces = p;
    // at most 2^23 tiles in two pieces an SM and one: below 2^32 up to 255 SMs
    it.kv0 = p > 1 ? (int)((unsigned)tiles * it.piece / (unsigned)p) : 0;
    it.kv1 = p > 1 ? (int)((unsigned)tiles * (it.piece + 1) / (unsigned)p) : tiles;
    it.total = u.total;
    it.part = p > 1 ? min(part + (it.head * p + it.piece) * it.rows, part_cap - it.rows) : -1;
    it.self = self;
    it.stride = a.h_kv;
    it.step = it.rows;
    return it;
}

// Work items from the lengths; each warp tries one L. Requests and row blocks are held in shared memory where they fit, else
// read again. Every CTA makes the whole plan (and writes the same words of it), but only its share of the items: an SM takes
// 3 us to write a thousand.
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkArgs a, const Work w) {
    __shared__ int shared[32];
    __shared__ long long sum;
    __shared__ int longest;
    __shared__ float cost[32];
    __shared__ int first_item[kPlanThreads], first_part[kPlanThreads];
    __shared__ Request s_request[kPlanThreads];
    __shared__ int s_tiles[kPlanThreads + 1];
    __shared__ int2 s_units[kPlanThreads];
    __shared__ int s_block[kPlanThreads];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, sms = w.sms;
    const int g_log2 = 31 - __clz(a.g), unit_cap = w.unit_cap;
    grid_release();
    if (tid == 0) { sum = 0; longest = 0; }
    const bool held = a.batch <= kPlanThreads;
    int* const first_block = held ? s_tiles : w.tiles;
    auto request_at = [&](int b) { return held ? s_request[b] : request(a, b); };
    grid_wait();

    // row blocks of each request, numbered through; a request's last block, which sees the most, comes first
    int base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int blocks = 0;
        if (b < a.batch) {
            const Request r = request(a, b);
            blocks = (int)(((long long)r.count * a.g + kChunkRows - 1) / kChunkRows);
            if (held) s_request[b] = r;
        }
        int total;
        const int at = block_scan(blocks, shared, total);
        if (b < a.batch) first_block[b] = min(base + at, unit_cap);
        base = min(base + total, unit_cap);      // more only where the starts do not ascend
    }
    if (tid == 0) first_block[a.batch] = base;
    const int units = base;
    int2* const unit = units <= kPlanThreads ? s_units : w.units;
    __syncthreads();
    int my_longest = 0;
    long long my_sum = 0;
    for (int u = tid; u < units; u += kPlanThreads) {
        const int b = last_at_most(first_block, a.batch, u);
        const int word = unit_word(request_at(b), first_block[b + 1] - 1 - u, a.g, g_log2);
        unit[u] = make_int2(b, word);
        my_longest = max(my_longest, tiles_of(word));
        my_sum += tiles_of(word);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        my_longest = max(my_longest, __shfl_xor_sync(0xffffffffu, my_longest, o));
        my_sum += __shfl_xor_sync(0xffffffffu, my_sum, o);
    }
    if (lane == 0) {
        atomicMax(&longest, my_longest);
        atomicAdd(reinterpret_cast<unsigned long long*>(&sum), (unsigned long long)my_sum);
    }
    __syncthreads();
    const float all = (float)(sum * a.h_kv);
    const int share = share_of(all, sms);
    {
        const int len = min(piece_length(warp, share, longest), max(longest, 1));
        const float inv = 1.0f / (float)len;
        int pieces = 0, parts = 0;
        for (int u = lane; u < units; u += 32) {
            const int p = about_pieces(tiles_of(unit[u].y), len, inv);
            pieces += p;
            if (p > 1) parts += p * rows_of(unit[u].y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            pieces += __shfl_xor_sync(0xffffffffu, pieces, o);
            parts += __shfl_xor_sync(0xffffffffu, parts, o);
        }
        if (lane == 0) cost[warp] = cost_of(pieces * a.h_kv, parts * a.h_kv, len, all, a, sms);
    }
    __syncthreads();
    const int len = piece_length(cheapest(cost[lane], lane), share, longest);

    // the longest pieces first, where the row blocks are held: what comes last is short
    const bool sorted = units <= kPlanThreads;
    if (sorted) {
        int2 mine = make_int2(0, 0);
        int length = 0, rank = 0;
        if (tid < units) {
            mine = s_units[tid];
            length = tiles_of(mine.y) / pieces_of(tiles_of(mine.y), len);
            first_item[tid] = length;
        }
        __syncthreads();
        if (tid < units) {
            for (int v = 0; v < units; ++v) rank += first_item[v] > length || (first_item[v] == length && v < tid);
            s_units[rank] = mine;
            s_block[rank] = first_block[mine.x + 1] - 1 - tid;
        }
        __syncthreads();
    }

    int item_base = 0, part_base = 0;
    for (int u0 = 0; u0 < units; u0 += kPlanThreads) {
        const int u = u0 + tid;
        int pieces = 0, rows = 0;
        if (u < units) {
            const int word = unit[u].y;
            pieces = pieces_of(tiles_of(word), len);
            rows = pieces > 1 ? pieces * a.h_kv * rows_of(word) : 0;
        }
        int items, parts;
        first_item[tid] = block_scan(pieces * a.h_kv, shared, items);
        first_part[tid] = block_scan(rows, shared, parts);
        __syncthreads();
        items = min(items, w.item_cap - item_base);
        for (int i = (warp * gridDim.x + blockIdx.x) * 32 + lane; i < items; i += kPlanThreads * gridDim.x) {
            const int at = last_at_most(first_item, min(kPlanThreads, units - u0), i);
            const int2 here = unit[u0 + at];
            const Request r = request_at(here.x);
            w.items[item_base + i] = item_of(a, Unit{here.x, sorted ? s_block[at] : first_block[here.x + 1] - 1 - (u0 + at), here.y,
                                                  r.tok0, r.pos0, r.total},
                                             pieces_of(tiles_of(here.y), len), i - first_item[at],
                                             part_base + first_part[at], w.part_cap, item_base + i);
        }
        item_base += items;
        part_base += parts;
        __syncthreads();
    }
    if (tid == 0 && blockIdx.x == 0) *w.head = Header{item_base, 0, part_base > 0};
}

// ---- attention ----------------------------------------------------------------------------------------------

// Shared memory of a CTA, by addresses: `base` and constants, so that a role keeps one register for all of it.
template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;                     // blocks of 64 channels, 128 bytes a row
    static constexpr int kHalfBytes = kChunkTile * 128;        // such a block of a K or V tile, or of a query block
    static constexpr int kTileBytes = kHalves * kHalfBytes;
    static constexpr int kStages = D == 128 ? 5 : 8;           // K and V tiles in turn
    static constexpr int kOffKv = 2 * kTileBytes;              // behind the two query blocks
    static constexpr int kOffItem = kOffKv + kStages * kTileBytes;
    static constexpr int kOffBar = kOffItem + kItemRing * (int)sizeof(Item);
    static constexpr int kBars = 2 * kStages + 2 * 5 + 1 + 2 * kItemRing;
    static constexpr int kOffMask = kOffBar + 8 * kBars;
    static constexpr int kOffTmem = kOffMask + 4 * kMaskRing;
    static constexpr int kOffFail = kOffTmem + 4;
    static constexpr int kOffMarked = kOffFail + 4;
    static constexpr int kOffPlan = kOffFail + 12;
    static constexpr int kBytes = kOffPlan + 28 * kSelfUnits + 24;
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
    // Columns of tensor memory: logits of the two blocks, outputs, and weights, beside the logits where there is room
    static constexpr bool kBeside = 2 * kChunkTile + 2 * D + kChunkTile <= 512;
    __device__ static constexpr int s_col(int t) { return t * kChunkTile; }
    __device__ static constexpr int o_col(int t) { return 2 * kChunkTile + t * D; }
    __device__ static constexpr int p_col(int t) { return kBeside ? 2 * kChunkTile + 2 * D + t * (kChunkTile / 2) : s_col(t); }

    uint32_t base;
    __device__ uint32_t q(int t) const { return base + t * kTileBytes; }
    __device__ uint32_t kv(int slot) const { return base + kOffKv + slot % kStages * kTileBytes; }
    __device__ uint32_t item(int i) const { return base + kOffItem + i % kItemRing * (int)sizeof(Item); }
    __device__ uint32_t mask(int tile) const { return base + kOffMask + 4 * (tile % kMaskRing); }
    __device__ uint32_t tmem() const { return base + kOffTmem; }
    __device__ uint32_t fail() const { return base + kOffFail; }
    __device__ uint32_t marked() const { return base + kOffMarked; }
    // mbarriers; those of a ring come with the phase of its i-th turn
    __device__ uint32_t bar(int i) const { return base + kOffBar + 8 * i; }
    __device__ uint32_t kv_full(int slot) const { return bar(slot % kStages); }
    __device__ uint32_t kv_empty(int slot) const { return bar(kStages + slot % kStages); }
    __device__ static uint32_t kv_phase(int slot) { return slot / kStages & 1; }
    __device__ uint32_t q_full(int t) const { return bar(2 * kStages + t); }
    __device__ uint32_t s_full(int t) const { return bar(2 * kStages + 2 + t); }
    __device__ uint32_t p_full(int t) const { return bar(2 * kStages + 4 + t); }
    __device__ uint32_t o_done(int t) const { return bar(2 * kStages + 6 + t); }
    __device__ uint32_t s_read(int t) const { return bar(2 * kStages + 8 + t); }
    __device__ uint32_t last() const { return bar(2 * kStages + 10); }
    __device__ uint32_t item_full(int i) const { return bar(2 * kStages + 11 + i % kItemRing); }
    __device__ uint32_t item_empty(int i) const { return bar(2 * kStages + 11 + kItemRing + i % kItemRing); }
    __device__ static uint32_t item_phase(int i) { return i / kItemRing & 1; }

    // A role that gives up: the others stop at their next wait.
    __device__ void give_up(const ChunkArgs& a, int where) const {
        sts32(fail(), 1);
        record_error(&a.dbg->kind, &a.dbg->index, 4, where);
    }
    // False once the wait has run out or another role has given up; the same for all lanes of the warp.
    __device__ __forceinline__ bool wait(uint32_t at, uint32_t phase, const ChunkArgs& a, int where) const {
        if (__all_sync(0xffffffffu, mbar_test(at, phase))) return true;
        return wait_longer(at, phase, a, where);
    }
    __device__ __forceinline__ bool wait_longer(uint32_t at, uint32_t phase, const ChunkArgs& a, int where) const {
        const uint32_t t0 = cycles();
        bool ok;
        while (!(ok = mbar_test(at, phase)) && !lds32(fail())) {
            if (cycles() - t0 > a.wait_ticks) {
                give_up(a, where);
                break;
            }
        }
        return __all_sync(0xffffffffu, ok);
    }
    // For what is in flight when a role stops: nobody is told.
    __device__ void drain(uint32_t at, uint32_t phase) const {
        const uint32_t t0 = cycles();
        while (!mbar_test(at, phase))
            if (cycles() - t0 > kChunkWait) return;
    }
    __device__ Item read_item(int i) const {
        Item it;
        lds128(item(i), reinterpret_cast<uint32_t*>(&it));
        lds128(item(i) + 16, reinterpret_cast<uint32_t*>(&it) + 4);
        lds128(item(i) + 32, reinterpret_cast<uint32_t*>(&it) + 8);
        lds128(item(i) + 48, reinterpret_cast<uint32_t*>(&it) + 12);
        return it;
    }
};

// The tiles of a block: how many of the item's cache tiles its rows see.
struct Blocks {
    int rows[2], count[2];
};
__device__ __forceinline__ Blocks blocks_of(const Item& it, int g_log2) {
    Blocks r;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        r.rows[t] = clamp_int(it.rows - kBlock * t, 0, kBlock);
        const int tiles = r.rows[t] ? (limit_of(it.r0 + kBlock * t + r.rows[t] - 1, it.pos0, g_log2) + kChunkTile - 1) / kChunkTile : 0;
        r.count[t] = max(min(it.kv1, tiles) - it.kv0, 0);
    }
    return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split_f32x2(uint64_t x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void store32(void* p, const uint32_t* u) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]) : "memory");
}

// A loader's own plan, in shared memory: the row blocks of few requests, and how they are cut.
struct SelfPlan {
    Unit unit[kSelfUnits];
    int first_item[kSelfUnits];
    int units, items, len, cut;
    int stream, all;                             // CTAs that share all tiles evenly, or 0; all tiles
};
static_assert(sizeof(SelfPlan) == 28 * kSelfUnits + 24, "as much as Layout reserves");

// The plan kernel's work by one warp.
__device__ __forceinline__ void plan_here(const ChunkArgs& a, SelfPlan* plan, int unit_cap, int sms, int lane) {
    auto found = [&](int units, int items, int len, int cut, int stream, int all) {
        if (lane == 0) {
            plan->units = units; plan->items = items; plan->len = len; plan->cut = cut; plan->stream = stream; plan->all = all;
        }
        __syncwarp();
    };
    const int g_log2 = 31 - __clz(a.g);
    int units = 0, longest = 0, most = 0;        // most: rows of a block at most
    long long sum = 0;
    bool even = true;                            // no two row blocks share tiles, none is without
#pragma unroll 1
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        Request r{};
        if (b < a.batch) r = request(a, b);
        const int blocks = (r.count * a.g + kChunkRows - 1) / kChunkRows;
        even = even && blocks <= 1;
        int at = blocks;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += y;
        }
        const int all = __shfl_sync(0xffffffffu, at, 31);
        at += units - blocks;
#pragma unroll 1
        for (int k = 0; k < blocks && at + k < unit_cap; ++k) {          // the last block, which sees the most, first
            const int word = unit_word(r, blocks - 1 - k, a.g, g_log2);
            plan->unit[at + k] = Unit{b, blocks - 1 - k, word, r.tok0, r.pos0, r.total};
            longest = max(longest, tiles_of(word));
            sum += tiles_of(word);
            even = even && tiles_of(word) > 0;
            most = max(most, rows_of(word));
        }
        units += all;
    }
    units = min(units, unit_cap);                // more only where the starts do not ascend
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    __syncwarp();
    const long long all = sum * a.h_kv;
    const int share = share_of((float)all, sms);
    int len = min(piece_length(lane, share, longest), max(longest, 1));
    int pieces = 0, parts = 0;
    for (int u = 0; u < units; ++u) {
        const int p = pieces_of(tiles_of(plan->unit[u].word), len);
        pieces += p;
        if (p > 1) parts += p * rows_of(plan->unit[u].word);
    }
    const float cost = cost_of(pieces * a.h_kv, parts * a.h_kv, len, (float)all, a, sms);
    const int at = cheapest(cost, lane);
    const float best = __shfl_sync(0xffffffffu, cost, at);
    len = __shfl_sync(0xffffffffu, len, at);
    parts = __shfl_sync(0xffffffffu, parts, at);
    // or equal stretches of all tiles in a line, which may begin and end within an item each
    const int ctas = (int)min((long long)gridDim.x, all);
    if (__all_sync(0xffffffffu, even) && all > 0 && (all + 1) * sms < 0x7fffffff &&       // products of both in 32 bits
        (float)(share + 2 * kStart) + 2.0f * (float)(ctas * most) * (float)a.d * kJoined < best) {
        int pos = 0;
#pragma unroll 1
        for (int u0 = 0; u0 < units; u0 += 32) {
            const int u = u0 + lane, mine = u < units ? tiles_of(plan->unit[u].word) * a.h_kv : 0;
            int s = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            if (u < units) plan->first_item[u] = pos + s - mine;     // here: its first tile of all
            pos += __shfl_sync(0xffffffffu, s, 31);
        }
        return found(units, units * a.h_kv + ctas - 1, 0, ctas > 1, ctas, (int)all);
    }
    // more items than CTAs: the longest pieces first, so that what follows them evens the CTAs out
    if (__shfl_sync(0xffffffffu, pieces, at) * a.h_kv > (int)gridDim.x) {
        auto length = [&](int u) {
            const int tiles = tiles_of(plan->unit[u].word);
            return tiles / pieces_of(tiles, len);
        };
        constexpr int kMine = (kSelfUnits + 31) / 32;
        Unit mine[kMine];
        int rank[kMine] = {};
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
            const int u = 32 * k + lane;
            if (u < units) mine[k] = plan->unit[u];
            if (u < units) plan->first_item[u] = length(u);
        }
        __syncwarp();
        for (int v = 0; v < units; ++v) {
            const int other = plan->first_item[v];
#pragma unroll
            for (int k = 0; k < kMine; ++k) {
                const int u = 32 * k + lane;
                if (u < units) rank[k] += other > plan->first_item[u] || (other == plan->first_item[u] && v < u);
            }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kMine; ++k)
            if (32 * k + lane < units) plan->unit[rank[k]] = mine[k];
        __syncwarp();
    }
    int items = 0;
#pragma unroll 1
    for (int u0 = 0; u0 < units; u0 += 32) {
        const int u = u0 + lane;
        const int mine = u < units ? pieces_of(tiles_of(plan->unit[u].word), len) * a.h_kv : 0;
        int s = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (u < units) plan->first_item[u] = items + s - mine;
        items += __shfl_sync(0xffffffffu, s, 31);
    }
    found(units, items, len, parts > 0, 0, 0);
}

// Item `item` of that plan.
__device__ __forceinline__ Item item_here(const ChunkArgs& a, const SelfPlan* plan, int item, int part_cap, int lane) {
    const int at = last_at_most(plan->first_item, plan->units, item);
    int parts = 0;                               // rows of the cut units before it
    for (int u = lane; u < at; u += 32) {
        const int p = pieces_of(tiles_of(plan->unit[u].word), plan->len);
        if (p > 1) parts += p * a.h_kv * rows_of(plan->unit[u].word);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) parts += __shfl_xor_sync(0xffffffffu, parts, o);
    return item_of(a, plan->unit[at], pieces_of(tiles_of(plan->unit[at].word), plan->len), item - plan->first_item[at], parts,
                   part_cap, item);
}

// Where row blocks share no tiles, all tiles stand in one line (row block by row block, head by head) and each CTA takes
// an equal stretch of it. The item at tile `at` of the line, up to the end of its (row block, head) or of the CTA's
// stretch. Its number is that of its (row block, head) plus the CTA's; a stretch that begins with a (row block, head)
// leaves a number out, which `gap` is then (else -1).
__device__ __forceinline__ int stretch(int cta, const SelfPlan* plan) {
    return (int)((unsigned)plan->all * min(cta, plan->stream) / (unsigned)plan->stream);
}
__device__ __forceinline__ Item item_in_line(const ChunkArgs& a, const SelfPlan* plan, int at, int end, int cta,
                                             int slot_rows, int& gap) {
    const int u = last_at_most(plan->first_item, plan->units, at);
    const int tiles = tiles_of(plan->unit[u].word), head = (at - plan->first_item[u]) / tiles;
    const int begin = plan->first_item[u] + head * tiles, number = u * a.h_kv + head;
    auto cta_of = [&](int x) { return (int)(((unsigned)(x + 1) * plan->stream - 1) / (unsigned)plan->all); };
    const int c0 = cta_of(begin), pieces = cta_of(begin + tiles - 1) - c0 + 1;
    Item it = item_of(a, plan->unit[u], 1, head, 0, 0, number + cta);
    it.kv0 = at - begin;
    it.kv1 = min(tiles, end - begin);
    it.piece = cta - c0;
    it.pieces = pieces;
    // a CTA has at most two pieces of cut items: the rest of one, and the beginning of one
    it.stride = 1;
    it.step = 2 * slot_rows;
    it.lead = slot_rows;
    it.part = pieces > 1 ? 2 * slot_rows * cta + (it.piece == 0 ? slot_rows : 0) : -1;
    gap = it.piece == 0 && cta > 0 && at == stretch(cta, plan) ? number + cta - 1 : -1;
    return it;
}

// Item `item` of the loader's own plan (or the one at tile `item` of the line, whose stretch ends at `end`) to the CTA's
// ring and to the list that the join reads. Out of line: the loader's registers are short.
__device__ __noinline__ void put_own_item(const ChunkArgs& a, const Work& w, const SelfPlan* plan, uint32_t to, int item, int end) {
    const int lane = threadIdx.x % 32;
    int gap = -1;
    const Item it = plan->stream ? item_in_line(a, plan, item, end, blockIdx.x, w.part_cap / (4 * w.sms), gap)
                                 : item_here(a, plan, item, w.part_cap, lane);
    if (lane == 0) {
        const uint4* from = reinterpret_cast<const uint4*>(&it);
#pragma unroll
        for (int c = 0; c < 4; ++c) sts128(to + 16 * c, from[c]);
        w.items[it.self] = it;
    }
    if (gap >= 0) {
        Item none{};
        none.part = -1;
        if (lane == 0) w.items[gap] = none;
        if (lane < 8) w.odd[(int64_t)gap * 8 + lane] = 0;
    }
}

// Loader: work items to the other roles, K and V pages to the ring.
template <int D>
__device__ __forceinline__ void load_role(const ChunkArgs& a, const Work& w, const CUtensorMap* map, const Layout<D> sm,
                                          SelfPlan* plan, int lane) {
    using L = Layout<D>;
    constexpr int kBoxes = kTilePages * L::kHalves;          // TMA boxes of a K or V tile: 16 tokens x 64 channels
    const int g_log2 = 31 - __clz(a.g);
    const int blocks = (int)(a.pages * a.h_kv * 2);          // a block id behind the pool reads as zeros
    int n_items;
    if (w.self) {
        plan_here(a, plan, w.unit_cap, w.sms, lane);
        n_items = min(plan->items, w.item_cap);
        if (blockIdx.x == 0 && lane == 0) *w.head = Header{n_items, 0, plan->cut};
    } else {
        n_items = w.head->items;
    }
    int slot = 0, tile = 0;                                  // ring positions, counted through
    // item: its number, or the tile of the line where it begins
    const bool in_line = w.self && plan->stream;
    int item = in_line ? stretch(blockIdx.x, plan) : blockIdx.x;
    if (in_line) n_items = stretch(blockIdx.x + 1, plan);
    bool ok = true;
    for (int i = 0; ok; ++i) {
        // asked for ahead of its use; the few items of an own plan go round to and fro
        int next = !w.self && lane == 0 ? atomicAdd(&w.head->next, 1) + (int)gridDim.x : 0;
        if (w.self) next = (i + 1) * (int)gridDim.x + (i % 2 ? (int)blockIdx.x : (int)(gridDim.x - 1 - blockIdx.x));
        const bool stop = item >= n_items;
        ok = sm.wait(sm.item_empty(i), sm.item_phase(i) ^ 1, a, i);
        if (!ok) break;
        if (!stop && w.self) {
            put_own_item(a, w, plan, sm.item(i), item, n_items);
        } else if (lane < 4) {                   // 16 bytes a lane; no rows: the end
            uint4 x = make_uint4(lane == 1 ? 0xffffffffu : 0, 0, 0, 0);
            if (!stop) x = reinterpret_cast<const uint4*>(w.items + item)[lane];
            sts128(sm.item(i) + 16 * lane, x);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.item_full(i));
        if (stop) break;
        const Item it = sm.read_item(i);
        if (in_line) next = item + it.kv1 - it.kv0;
        const Blocks bl = blocks_of(it, g_log2);
        const bool lost = a.lost_loads && blockIdx.x % 2;    // what a test asks for: some tiles of this item, then no more
        const int count = min(max(bl.count[0], bl.count[1]), lost ? (int)blockIdx.x / 2 % 4 : 0x7fffffff);
        const int32_t* table = a.tables + (int64_t)it.b * a.stride;
        // page ids of four tiles a load, asked for four tiles ahead; -1 where there is no page to read
        const int last_page = min((it.total + kPage - 1) / kPage, (it.kv0 + count) * kTilePages);
        auto look_up = [&](int j) {
            const int page = (it.kv0 + j) * kTilePages + lane;
            return page < last_page ? table[page] : -1;
        };
        int ids = -1, ahead = count ? look_up(0) : -1;
        for (int j = 0; j < count && ok; ++j) {
            if (j % 4 == 0) {
                ids = ahead;
                ahead = look_up(j + 4);
                if (ids < 0 || ids >= a.pages) {
                    if (a.debug && (it.kv0 + j) * kTilePages + lane < last_page) record_error(&a.dbg->kind, &a.dbg->index, 2, ids);
                    ids = -1;
                }
            }
            const uint32_t there = __ballot_sync(0xffffffffu, ids >= 0);
            const int box = lane % kBoxes;                   // lanes beyond the boxes only follow
            const int page = box / L::kHalves, half = box % L::kHalves;
            const int id = __shfl_sync(0xffffffffu, ids, j % 4 * kTilePages + page);
            const int z = id >= 0 ? (id * a.h_kv + it.head) * 2 : blocks;
            if (lane == 0) sts32(sm.mask(tile), (there >> (j % 4 * kTilePages)) & 0xff);
            __syncwarp();
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {           // K, then V
                ok = sm.wait(sm.kv_empty(slot), sm.kv_phase(slot) ^ 1, a, 1000 + i);
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(sm.kv_full(slot), L::kTileBytes);
                __syncwarp();
                if (lane < kBoxes)
                    tma_load_3d(sm.kv(slot) + half * L::kHalfBytes + page * (kPage * 128), map, 64 * half, 0,
                                id >= 0 ? z + kind : blocks, sm.kv_full(slot));
                ++slot;
            }
            ++tile;
        }
        if (lost) break;
        item = __shfl_sync(0xffffffffu, next, 0);
    }
    // what was asked for lands before the CTA may leave
    for (int s = max(slot - L::kStages, 0); s < slot; ++s) sm.drain(sm.kv_full(s), sm.kv_phase(s));
}

// Issuer of the matrix products.
template <int D>
__device__ __forceinline__ void issue_role(const ChunkArgs& a, const Layout<D> sm, uint32_t tmem, int lane) {
    using L = Layout<D>;
    constexpr uint32_t kScores = idesc_bf16(kBlock, kChunkTile, false), kValues = idesc_bf16(kBlock, D, true);
    const int g_log2 = 31 - __clz(a.g);
    const uint32_t leader = elected();
    int slot = 0;
    uint32_t q_phase[2] = {0, 0};
    int steps[2] = {0, 0};                                   // of each block, before the item
    bool ok = true, issued = false;
    auto scores = [&](int t, int k_slot) {                   // S of block t
        const uint32_t qd = sw128_desc(sm.q(t), 0), kd = sw128_desc(sm.kv(k_slot), 0);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks / 4) * L::kHalfBytes + (ks % 4) * 32) >> 4;
            umma_ss(leader, tmem + L::s_col(t), qd + off, kd + off, kScores, ks > 0);
        }
        umma_commit(leader, sm.s_full(t));
    };
    auto values = [&](int t, int v_slot, int j) {            // O of block t: tile j of the item
        const uint32_t vd = sw128_desc(sm.kv(v_slot), L::kHalfBytes), p = tmem + L::p_col(t);
#pragma unroll
        for (int k16 = 0; k16 < kTilePages; ++k16)
            umma_ts(leader, tmem + L::o_col(t), p + k16 * 8, vd + k16 * (2048 >> 4), kValues, j % kFold > 0 || k16 > 0);
        umma_commit(leader, sm.o_done(t));
    };
    // V of tile j, without what may lie behind the sequence on its last page
    auto clean_values = [&](const Item& it, int v_slot, int j) {
        const int tail = it.total % kPage;
        if (tail && it.kv0 + j == it.total / kChunkTile) {
            const int left = kPage - tail;
            const uint32_t to = sm.kv(v_slot) + it.total % kChunkTile * 128;
            for (int c = lane; c < left * 8 * L::kHalves; c += 32)
                sts128(to + c / (left * 8) * L::kHalfBytes + c % (left * 8) * 16, make_uint4(0, 0, 0, 0));
            fence_async();
            __syncwarp();
        }
    };
    for (int i = 0; ok; ++i) {
        ok = sm.wait(sm.item_full(i), sm.item_phase(i), a, 2000 + i);
        if (!ok) break;
        const Item it = sm.read_item(i);
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.item_empty(i));
        if (it.rows < 0) break;
        const Blocks bl = blocks_of(it, g_log2);
        const int count = max(bl.count[0], bl.count[1]);
        if (count == 0) continue;
        // S of the first tile
        const int k0 = slot++;
        ok = sm.wait(sm.kv_full(k0), sm.kv_phase(k0), a, 3000 + i);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (!ok || bl.count[t] == 0) continue;
            ok = sm.wait(sm.q_full(t), q_phase[t], a, 4000 + i);
            q_phase[t] ^= 1;
            if (!ok) break;
            tc_fence_after();
            scores(t, k0);
            issued = true;
        }
        if (!ok) break;
        umma_commit(leader, sm.kv_empty(k0));
        if constexpr (L::kBeside) {
            // A block's next logits follow once the last ones are in registers, and its outputs half a step behind the
            // other block's (8,192 tokens of 32 heads of 64: 254 us, 292 in the order below).
            int vs = 0, v_last = 0;                          // V of this tile and of the one before
            for (int j = 0; j <= count && ok; ++j) {
                v_last = vs;
                if (j < count) vs = slot++;
                const bool more = j + 1 < count;
                const int kn = more ? slot++ : 0;
                if (more) ok = sm.wait(sm.kv_full(kn), sm.kv_phase(kn), a, 6000 + i);
                if (ok && j + 1 < bl.count[0]) {
                    ok = sm.wait(sm.s_read(0), steps[0] + j & 1, a, 7000 + i);
                    if (!ok) break;
                    tc_fence_after();
                    scores(0, kn);
                }
                if (ok && j > 0 && j <= bl.count[1]) {
                    ok = sm.wait(sm.p_full(1), steps[1] + j + 1 & 1, a, 7000 + i);
                    if (!ok) break;
                    tc_fence_after();
                    values(1, v_last, j - 1);
                }
                if (ok && j > 0) umma_commit(leader, sm.kv_empty(v_last));
                if (ok && j + 1 < bl.count[1]) {
                    ok = sm.wait(sm.s_read(1), steps[1] + j & 1, a, 7000 + i);
                    if (!ok) break;
                    tc_fence_after();
                    scores(1, kn);
                }
                if (ok && more) umma_commit(leader, sm.kv_empty(kn));
                if (!ok || j == count) break;
                ok = sm.wait(sm.kv_full(vs), sm.kv_phase(vs), a, 5000 + i);
                if (!ok) break;
                clean_values(it, vs, j);
                if (j < bl.count[0]) {
                    ok = sm.wait(sm.p_full(0), steps[0] + j & 1, a, 7000 + i);
                    if (!ok) break;
                    tc_fence_after();
                    values(0, vs, j);
                }
            }
        } else {
            for (int j = 0; j < count && ok; ++j) {
                const int vs = slot++;
                ok = sm.wait(sm.kv_full(vs), sm.kv_phase(vs), a, 5000 + i);
                if (!ok) break;
                clean_values(it, vs, j);
                const bool more = j + 1 < count;
                const int kn = more ? slot++ : 0;
                bool here = false;                           // K of the next tile
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (j < bl.count[t]) {
                        ok = sm.wait(sm.p_full(t), steps[t] + j & 1, a, 7000 + i);
                        if (!ok) break;
                        tc_fence_after();
                        values(t, vs, j);
                    }
                    if (t == 1) umma_commit(leader, sm.kv_empty(vs));
                    if (j + 1 < bl.count[t]) {
                        if (!here) ok = sm.wait(sm.kv_full(kn), sm.kv_phase(kn), a, 6000 + i);
                        here = true;
                        if (!ok) break;
                        tc_fence_after();
                        scores(t, kn);
                    }
                }
                if (ok && more) umma_commit(leader, sm.kv_empty(kn));
            }
        }
        steps[0] += bl.count[0];
        steps[1] += bl.count[1];
    }
    // the last matrix products are done before tensor memory is freed
    if (issued) {
        umma_commit(leader, sm.last());
        __syncwarp();
        sm.drain(sm.last(), 0);
    }
}

// Asks for a block's queries, 16 bytes at a time, into the swizzled layout; zeros behind the last row. There after
// async_copies_done.
template <int D>
__device__ __forceinline__ void ask_queries(const ChunkArgs& a, const Item& it, const Layout<D> sm, int t, int rows,
                                            int thread, int g_log2) {
    using L = Layout<D>;
    const int c = thread % (D / 8);
    const uint16_t* from = a.q + (int64_t)it.tok0 * a.q_stride + (it.head << g_log2) * D + c * 8;
    const int r0 = it.r0 + kBlock * t;
#pragma unroll 4
    for (int row = thread / (D / 8); row < kBlock; row += kBlock * 8 / D) {
        const int r = r0 + row;
        const uint16_t* at = from + (row < rows ? (int64_t)(r >> g_log2) * a.q_stride + (r & (a.g - 1)) * D : 0);
        async_copy16(sm.q(t) + c / 8 * L::kHalfBytes + row * 128 + (((c % 8) ^ (row % 8)) * 16), at, row < rows);
    }
}

// Logits of 32 tokens that the row does not see count as -infinity: from `seen` on, and those of absent pages.
__device__ __forceinline__ void hide(uint32_t (&u)[32], int seen, int mask) {
#pragma unroll
    for (int c = 0; c < 32; ++c)
        if (c >= seen || !(mask >> (c / kPage) & 1)) u[c] = 0xff800000u;
}

// The largest of 32 logits and `top`.
__device__ __forceinline__ float max32(const uint32_t (&u)[32], float top) {
    float m[4] = {top, __uint_as_float(u[0]), __uint_as_float(u[1]), __uint_as_float(u[2])};
#pragma unroll
    for (int c = 3; c < 31; c += 2) m[c / 2 % 4] = fmax3(m[c / 2 % 4], __uint_as_float(u[c]), __uint_as_float(u[c + 1]));
    m[0] = fmax3(m[0], m[1], __uint_as_float(u[31]));
    return fmax3(m[0], m[2], m[3]);
}

// Weights 2^(scale u - m) of a row's 128 tokens, in bf16 to pk, and the sum of the unrounded ones. In stages of 32 that
// overlap by hand (a warp issues in order, and ex2 has its result long after its issue): all in the logits' registers.
// 128 ex2 of 4 cycles each bound it, 512 cycles a warp.
__device__ __forceinline__ float weigh128(uint32_t (&u)[4][32], uint64_t scale, uint64_t less, uint32_t (&pk)[2][32]) {
    uint64_t sum[2] = {0, 0};
    auto scaled = [&](int c) {
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            float x, y;
            split_f32x2(fma_f32x2(f32x2(__uint_as_float(u[c][k]), __uint_as_float(u[c][k + 1])), scale, less), x, y);
            u[c][k] = __float_as_uint(x);
            u[c][k + 1] = __float_as_uint(y);
        }
    };
    auto power = [&](int c, int k) { u[c][k] = __float_as_uint(exp2_approx(__uint_as_float(u[c][k]))); };
    auto packed = [&](int c, int k) {
        const float x = __uint_as_float(u[c][k]), y = __uint_as_float(u[c][k + 1]);
        pk[c / 2][c % 2 * 16 + k / 2] = bf16_pair(x, y);
        sum[k / 2 % 2] = add_f32x2(sum[k / 2 % 2], f32x2(x, y));
    };
    scaled(0);
#pragma unroll
    for (int k = 0; k < 32; ++k) power(0, k);
#pragma unroll
    for (int c = 1; c < 4; ++c) {
        scaled(c);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            power(c, k);
            power(c, k + 1);
            packed(c - 1, k);
        }
    }
#pragma unroll
    for (int k = 0; k < 32; k += 2) packed(3, k);
    float x, y;
    split_f32x2(add_f32x2(sum[0], sum[1]), x, y);
    return x + y;
}

// The tensor core cuts off what its fp32 accumulator does not hold, so a sum of one sign falls short, a little more with each
// of a tile's eight additions: by 0.6 % after 8,192 tiles and 2.6 % after 32,768 (measured: 2^-23.3 of the final sum an
// addition). Every kFold tiles the outputs are therefore added, rounded to nearest, to a row in the workspace, and begin
// anew; at the end they come back. An accumulator is short by 0.04 % then (by that rate), and 512 tiles take some 600 us,
// the addition some 5.
//
// Instructions on tensor memory want the warp's lanes together: where some have a row and others none, they meet again
// in front of each (here and where outputs are stored).
//
// Adds a thread's row of outputs (reference m, sum) to its folded ones, the first time over them. `there`: whether the
// thread has a row; tensor memory is read by the whole warp.
template <int D>
__device__ __noinline__ void fold_row(float2* ml, float* acc, uint32_t o_col, float m, float sum, bool first, bool there) {
    const float2 old = first || !there ? make_float2(m, 0.0f) : *ml;
    const float f = exp2_approx(old.x - m);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        __syncwarp();
        tmem_read32(o_col + c, o);
        if (there) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                float4* at = reinterpret_cast<float4*>(acc + c + k);
                float4 x = first ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *at;
                x.x = fmaf(x.x, f, __uint_as_float(o[k])); x.y = fmaf(x.y, f, __uint_as_float(o[k + 1]));
                x.z = fmaf(x.z, f, __uint_as_float(o[k + 2])); x.w = fmaf(x.w, f, __uint_as_float(o[k + 3]));
                *at = x;
            }
        }
    }
    if (there) *ml = make_float2(m, fmaf(old.y, f, sum));
}
// Adds a thread's folded row to its outputs in tensor memory, whose reference is m; returns the folded sum.
template <int D>
__device__ __noinline__ float unfold_row(const float2* ml, const float* acc, uint32_t o_col, float m, bool there) {
    const float2 old = there ? *ml : make_float2(m, 0.0f);
    const float f = exp2_approx(old.x - m);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        __syncwarp();
        tmem_read32(o_col + c, o);
        if (there) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                const float4 x = *reinterpret_cast<const float4*>(acc + c + k);
                o[k] = __float_as_uint(fmaf(x.x, f, __uint_as_float(o[k])));
                o[k + 1] = __float_as_uint(fmaf(x.y, f, __uint_as_float(o[k + 1])));
                o[k + 2] = __float_as_uint(fmaf(x.z, f, __uint_as_float(o[k + 2])));
                o[k + 3] = __float_as_uint(fmaf(x.w, f, __uint_as_float(o[k + 3])));
            }
        }
        __syncwarp();
        tmem_st32(o_col + c, o);
    }
    tmem_wait_st();
    return old.y * f;
}

// Softmax of block t: one thread a row.
template <int D>
__device__ __forceinline__ void softmax_role(const ChunkArgs& a, const Work& w, const Layout<D> sm, uint32_t tmem, int t,
                                             int warp, int lane) {
    const int g_log2 = 31 - __clz(a.g), in_block = warp * 32 + lane;
    using L = Layout<D>;
    const uint32_t s_col = tmem + ((uint32_t)(32 * warp) << 16) + L::s_col(t);
    const uint32_t o_col = tmem + ((uint32_t)(32 * warp) << 16) + L::o_col(t);
    const uint32_t p_col = tmem + ((uint32_t)(32 * warp) << 16) + L::p_col(t);
    int tile = 0, step = 0;                      // tiles of the CTA, steps of this block, counted through
    auto mine = [&](const Item& it) { return kBlock * t + in_block < it.rows; };     // the thread has a row
    auto fold_at = [&] { return (int64_t)blockIdx.x * w.fold_rows + kBlock * t + in_block; };
    // Waits for item i and asks for its queries, once the products with the last ones are done; says that they are there.
    bool asked = false;
    auto ask = [&](int i) {
        if (!sm.wait(sm.item_full(i), sm.item_phase(i), a, 8000 + i)) return false;
        const Item it = sm.read_item(i);
        if (it.rows < 0) return true;
        const Blocks bl = blocks_of(it, g_log2);
        asked = (t ? bl.count[1] : bl.count[0]) > 0;
        if (asked) ask_queries<D>(a, it, sm, t, t ? bl.rows[1] : bl.rows[0], in_block, g_log2);
        return true;
    };
    auto there = [&] {
        if (!asked) return;
        async_copies_done();
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.q_full(t));
        asked = false;
    };
    if (!ask(0)) return;
    there();
    for (int i = 0;; ++i) {
        int count, seen;
        bool working;
        const int tile0 = tile;
        {
            const Item it = sm.read_item(i);
            if (it.rows < 0) return;
            const Blocks bl = blocks_of(it, g_log2);
            const int rows = t ? bl.rows[1] : bl.rows[0];
            count = t ? bl.count[1] : bl.count[0];
            tile += max(bl.count[0], bl.count[1]);
            working = 32 * warp < rows;
            // rows behind the last one see everything: their zeros need no mask
            seen = in_block < rows ? limit_of(it.r0 + kBlock * t + in_block, it.pos0, g_log2) - it.kv0 * kChunkTile : 0x7fffffff;
        }
        float m = kNoReference, sum = 0.0f;
        bool early = false;
        for (int j = 0; j < count; ++j, ++step, seen -= kChunkTile) {
            if (!sm.wait(sm.s_full(t), step & 1, a, 9000 + i)) return;
            // the last logits: the next item's queries travel while their weights are formed and the products end. Not
            // waited for here: the loader may need these weights to get that far.
            if (j + 1 == count && __all_sync(0xffffffffu, mbar_over(sm.item_full(i + 1), sm.item_phase(i + 1)))) {
                if (!ask(i + 1)) return;
                early = true;
            }
            // The block's products before these logits, which read the weights and add to the outputs: done with the
            // logits where those were asked for behind them, else waited for.
            auto done = [&] { return !L::kBeside || j == 0 || sm.wait(sm.o_done(t), (step - 1) & 1, a, 10000 + i); };
            if (!working) {                      // no row of this warp is any: what its lanes hold as weights reaches nothing
                if (L::kBeside && lane == 0) mbar_arrive(sm.s_read(t));
                if (!done()) return;             // nor may it be a step ahead
                if (lane == 0) mbar_arrive(sm.p_full(t));
                continue;
            }
            tc_fence_after();
            if (j % kFold == 0 && j > 0) {
                if (!done()) return;
                tc_fence_after();
                fold_row<D>(w.fold_ml + fold_at(), w.fold_acc + fold_at() * D, o_col, m, sum, j == kFold, mine(sm.read_item(i)));
                sum = 0.0f;
            }
            uint32_t u[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, u[c]);
            const int mask = lds32(sm.mask(tile0 + j));
            const bool hidden = __any_sync(0xffffffffu, seen < kChunkTile || mask != 0xff);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_wait(u[c]);
            if (L::kBeside) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sm.s_read(t));
            }
            if (hidden) {
#pragma unroll
                for (int c = 0; c < 4; ++c) hide(u[c], seen - 32 * c, mask >> 2 * c);
                __syncwarp();
            }
            float high = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) high = max32(u[c], high);
            high *= a.scale_log2;
            // Here, not where the weights are stored: that keeps the blocks apart, one finding its largest logits while the
            // other forms weights (8,192 tokens of 32 heads of 64: 254 us; 284 to 288 with the wait at the store or in
            // front of the logits, where both blocks fall into step)
            if (!done()) return;
            if (L::kBeside) tc_fence_after();
            const bool rise = high > m + kHeadroom;
            if (__any_sync(0xffffffffu, rise)) {
                const float to = rise ? high : m, f = exp2_approx(m - to);
                m = to;
                sum *= f;
                if (j > 0) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 8) tmem_scale8(o_col + c, f);
                }
            }
            uint32_t pk[2][32];
            sum += weigh128(u, f32x2(a.scale_log2, a.scale_log2), f32x2(-m, -m), pk);
            tmem_st32(p_col, pk[0]);             // at most over logits that the thread has read
            tmem_st32(p_col + 32, pk[1]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sm.p_full(t));
        }
        // a block without tokens waits for the loader through all of the other block's: a wait's limit for 2^18 of them
        for (int k = count ? 0 : (tile - tile0) >> 18; k > 0 && !lds32(sm.fail()) && !mbar_over(sm.item_full(i + 1), sm.item_phase(i + 1)); --k)
            sm.drain(sm.item_full(i + 1), sm.item_phase(i + 1));
        if (!early && !ask(i + 1)) return;
        there();
        if (count > 0 && !sm.wait(sm.o_done(t), (step - 1) & 1, a, 10000 + i)) return;
        uint32_t again = 0;
        if (working) {
            tc_fence_after();
            if (count > kFold) sum += unfold_row<D>(w.fold_ml + fold_at(), w.fold_acc + fold_at() * D, o_col, m, mine(sm.read_item(i)));
            const Item it = sm.read_item(i);
            const int r = it.r0 + kBlock * t + in_block;                 // row of the request
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const int64_t row = (int64_t)(it.tok0 + (r >> g_log2)) * (a.h_kv << g_log2) + (it.head << g_log2) + (r & (a.g - 1));
            const int part = it.part + r - it.r0;
            if (it.part >= 0 && mine(it)) w.part_ml[part] = make_float2(m, sum);
            uint64_t probe = 0;                  // 0 * x of all channels: NaN where one is infinite or NaN
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                __syncwarp();
                if (count > 0) {
                    tmem_read32(o_col + c, o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0;
                }
#pragma unroll
                for (int k = 0; k < 32; k += 2) probe = fma_f32x2(f32x2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), 0ull, probe);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = inv == 0.0f ? 0 : o[k];    // no token with a weight: zeros, whatever values are
                if (mine(it) && it.part >= 0) {  // a part of a cut item, as it is
                    float* to = w.part_acc + (int64_t)part * D + c;
#pragma unroll
                    for (int k = 0; k < 32; k += 8) store32(to + k, o + k);
                } else if (mine(it)) {
                    uint32_t y[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float lo, hi;
                        split_f32x2(mul_f32x2(f32x2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), f32x2(inv, inv)), lo, hi);
                        y[k] = bf16_pair(lo, hi);
                    }
                    uint16_t* to = a.out + row * D + c;
                    store32(to, y);
                    store32(to + 16, y + 8);
                }
            }
            __syncwarp();
            tc_fence_before();
            float lo, hi;
            split_f32x2(probe, lo, hi);
            // a sum of NaN is a row of NaN, none a row of zeros; but a part without a weight may hold infinities of its row
            again = __ballot_sync(0xffffffffu, lo + hi != 0.0f && mine(it) && inv == inv && (inv != 0.0f || it.part >= 0));
        }
        if (lane == 0) w.odd[(int64_t)sm.read_item(i).self * 8 + 4 * t + warp] = again;
        if (lane == 0 && again) sts32(sm.marked(), 1);
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.item_empty(i));
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_attend_kernel(const __grid_constant__ ChunkArgs a,
                                                                   const __grid_constant__ Work w,
                                                                   const __grid_constant__ CUtensorMap map) {
    using L = Layout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];        // the tiles' swizzle wants them on 1,024 bytes
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x % 32;    // uniform for the compiler too
    const L sm{smem_u32(smem)};
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(sm.kv_full(s), 1);
            mbar_init(sm.kv_empty(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(sm.q_full(t), kSoftmaxWarps / 2);
            mbar_init(sm.s_full(t), 1);
            mbar_init(sm.p_full(t), kSoftmaxWarps / 2);
            mbar_init(sm.o_done(t), 1);
            mbar_init(sm.s_read(t), kSoftmaxWarps / 2);
        }
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(sm.item_full(i), 1);
            mbar_init(sm.item_empty(i), kSoftmaxWarps + 1);
        }
        mbar_init(sm.last(), 1);
        sts32(sm.fail(), 0);
        sts32(sm.marked(), 0);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    if (warp == kSoftmaxWarps + 1) {             // all of tensor memory: S of two blocks, O of two blocks
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(sm.tmem()), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, lds32(sm.tmem()), 0);
    grid_wait();
    grid_release();

    // registers: 384 x 168 at launch; 256 x 192 + 128 x 112 = 63,488 of those 64,512
    if (warp < kSoftmaxWarps) {
        more_registers<192>();
        softmax_role<D>(a, w, sm, tmem, warp / 4, warp % 4, lane);
    } else {
        fewer_registers<112>();
        if (warp == kSoftmaxWarps) load_role<D>(a, w, &map, sm, reinterpret_cast<SelfPlan*>(smem + L::kOffPlan), lane);
        if (warp == kSoftmaxWarps + 1) issue_role<D>(a, sm, tmem, lane);
    }
    async_copies_done();                         // of a role that stopped
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) w.marked[blockIdx.x] = lds32(sm.marked());
    if (warp == kSoftmaxWarps + 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512) : "memory");
    }
}

// ---- join ---------------------------------------------------------------------------------------------------

template <int N>
__device__ __forceinline__ void store_bf16(uint16_t* to, const float (&x)[N], float f) {
#pragma unroll
    for (int c = 0; c < N; c += 2) *reinterpret_cast<uint32_t*>(to + c) = bf16_pair(x[c] * f, x[c + 1] * f);
}

// ---- rows that are not finite
//
// An infinity or NaN in V reaches every row of its tile, through a weight of 0 those too that must not see it; and a sum of
// finite values may pass fp32. A CTA of the join takes up to 32 such rows (of one request and KV head) at a time:
//   look_again goes over V once for all of them, finds the tokens with an infinity or NaN, and adds those values by
//   themselves, with weight one for every token that has a weight, however small (0 makes NaN of an infinity, as it
//   should): a channel that has any is that sum, whatever its finite values add;
//   form_rows forms what is left, infinite or NaN without such a value among those that the row sees, from the first token.
// An 8,192-token prompt (32 / 8 heads of 128, 345 us) takes 3.3 ms with an infinite value of token 10 in every head, 1.2 with
// one in one head, 5.8 with one of token 8,190, whose tile's rows are formed, and 121 where every row's sum passes fp32
// (3.7 s where a warp formed all rows of four items, a token's values at a time). Loops stay rolled up: a kernel's
// instructions take the next one's place in the instruction cache even where they do not run. With as many of them again,
// eight tokens at 100,000 took 80 us instead of 74, all of it at the start of the next call.
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kScanPages = 32 * kJoinWarps;      // pages of a stretch of V, a lane's table entry each

template <int D>
struct Again {
    // tokens of a step of form_rows; the stride lets eight lanes read 16 bytes of a token each without a bank twice
    alignas(16) uint16_t k[32][D + 8], v[32][D + 8];
    float acc[32][D];                            // of each row: infinities and NaN; then what form_rows adds
    const uint16_t* q[32];                       // of each row: its queries, its outputs, the tokens that it sees (0: no row)
    uint16_t* out[32];
    int seen[32];
    float m[32], sum[32];
    uint32_t words[kJoinThreads];                // marked rows, 32 each: of whole items, or the first eight of a cut one
    uint32_t bad[kScanPages];                    // per page: tokens with an infinity or NaN
    uint32_t todo, left;                         // rows to form, now and in another turn
    uint8_t want[32][32];                        // per row and lane: channels to form
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The channels want[k] of the rows k of s.todo, by the whole CTA: 32 tokens a step, whose K and V go to shared memory. A
// warp takes every eighth row, a lane a token's logit, then some channels of all tokens. The values are added as they are
// (unit 1), so that the smallest count; the channels whose sum passes fp32 are left for a second turn, where they are added
// in units of 2^31, more than there are tokens.
template <int D>
__device__ __forceinline__ void form_rows(const ChunkArgs& a, const int32_t* table, int head, int end, float unit, Again<D>& s, int lane, int warp) {
    constexpr int kChannels = D / 32, kChunks = D / 8;
#pragma unroll 1
    for (int i = threadIdx.x; i < 32 * D; i += kJoinThreads) {
        s.acc[0][i] = 0.0f;
        s.m[i / D] = kNoReference;
        s.sum[i / D] = 0.0f;
    }
#pragma unroll 1
    for (int t0 = 0; t0 < end; t0 += 32) {
        auto page = [&](int t) {
            const int id = t0 + t < end ? table[(t0 + t) / kPage] : -1;
            return id < a.pages ? id : -1;
        };
#pragma unroll 1
        for (int i = threadIdx.x; i < 32 * kChunks; i += kJoinThreads) {
            const int c = i % kChunks * 8, t = i / kChunks, id = page(t);
            const uint16_t* from = a.pool + (((int64_t)max(id, 0) * a.h_kv + head) * 2 * kPage + t % kPage) * D + c;
            async_copy16(smem_u32(&s.k[t][c]), from, id >= 0);
            async_copy16(smem_u32(&s.v[t][c]), from + kPage * D, id >= 0);
        }
        const bool there = page(lane) >= 0;
        async_copies_done();
        __syncthreads();
#pragma unroll 1
        for (int k = warp; k < 32; k += kJoinWarps) {
            const int seen = s.seen[k] - t0;
            if (!(s.todo >> k & 1) || seen <= 0) continue;
            const uint16_t* q = s.q[k];
            float x = 0.0f;
#pragma unroll 1
            for (int c = 0; c < D; c += 8) {
                const uint4 u = *reinterpret_cast<const uint4*>(q + c), v = *reinterpret_cast<const uint4*>(&s.k[lane][c]);
                x += bf16_lo(u.x) * bf16_lo(v.x) + bf16_hi(u.x) * bf16_hi(v.x) + bf16_lo(u.y) * bf16_lo(v.y) +
                     bf16_hi(u.y) * bf16_hi(v.y) + bf16_lo(u.z) * bf16_lo(v.z) + bf16_hi(u.z) * bf16_hi(v.z) +
                     bf16_lo(u.w) * bf16_lo(v.w) + bf16_hi(u.w) * bf16_hi(v.w);
            }
            x = there && lane < seen ? x * a.scale_log2 : -INFINITY;
            float m = fmaxf(x, s.m[k]);
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            // rounded for the product and summed unrounded, as in the attention
            const float f = exp2_approx(s.m[k] - m), e = exp2_approx(x - m), p = bf16_lo(bf16_pair(e, 0.0f));
            const float sum = s.sum[k] * f + warp_sum(e);
            float acc[kChannels] = {};               // of the step alone: a sum of 2^24 would take no more ones
#pragma unroll 1
            for (int i = 0; i < min(seen, 32); ++i) {
                const float pi = __shfl_sync(0xffffffffu, p, i) * unit;
#pragma unroll
                for (int c = 0; c < kChannels; c += 2) {
                    const uint32_t v = *reinterpret_cast<const uint32_t*>(&s.v[i][lane * kChannels + c]);
                    acc[c] += pi * bf16_lo(v);
                    acc[c + 1] += pi * bf16_hi(v);
                }
            }
#pragma unroll
            for (int c = 0; c < kChannels; ++c) {
                float& to = s.acc[k][lane * kChannels + c];
                to = (f == 0.0f ? 0.0f : to * f) + acc[c];
            }
            __syncwarp();                            // all lanes have read them
            s.sum[k] = sum;
            s.m[k] = m;
            __syncwarp();
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) s.left = 0;
    __syncthreads();
#pragma unroll 1
    for (int k = warp; k < 32; k += kJoinWarps) {
        if (!(s.todo >> k & 1)) continue;
        const float inv = s.sum[k] == 0.0f ? 0.0f : 1.0f / (s.sum[k] * unit);
        uint32_t want = s.want[k][lane];
#pragma unroll 1
        for (int c = 0; c < kChannels; ++c) {
            const float y = s.acc[k][lane * kChannels + c] * inv;
            if (!(want >> c & 1) || (unit == 1.0f && !(fabsf(y) < INFINITY))) continue;
            s.out[k][lane * kChannels + c] = (uint16_t)bf16_pair(y, 0.0f);
            want &= ~(1u << c);
        }
        s.want[k][lane] = (uint8_t)want;
        if (want) atomicOr(&s.left, 1u << k);
    }
    __syncthreads();
    if (threadIdx.x == 0) s.todo = s.left;
    __syncthreads();
}

// The rows `from` + k of an item, for the bits k of `marked`, by the whole CTA; their outputs are there, infinities and NaN
// among them, and they have a weight.
template <int D>
__device__ __noinline__ void look_again(const ChunkArgs& a, const Item* item, int from, uint32_t marked, Again<D>& s) {
    constexpr int kChannels = D / 32, kLanes = D / 8, kRounds = kPage * kLanes / 32;         // 16 bytes a lane
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, behind = item->rows - from, head = item->head;
    if (behind < 32) marked &= behind > 0 ? (1u << behind) - 1 : 0;
    if (!marked) return;
    const int32_t* table = a.tables + (int64_t)item->b * a.stride;
    if (threadIdx.x < 32) {
        const int r = item->r0 + from + lane, g_log2 = 31 - __clz(a.g), channel = (head * a.g + (r & (a.g - 1))) * D;
        const int64_t token = item->tok0 + (r >> g_log2);
        s.q[lane] = a.q + token * a.q_stride + channel;
        s.out[lane] = a.out + token * (a.h_kv * a.g * D) + channel;
        s.seen[lane] = marked >> lane & 1 ? min(limit_of(r, item->pos0, g_log2), item->total) : 0;
        if (lane == 0) s.todo = 0;
    }
#pragma unroll 1
    for (int i = threadIdx.x; i < 32 * D; i += kJoinThreads) s.acc[0][i] = 0.0f;
    __syncthreads();
    const int end = s.seen[31 - __clz(marked)];
#pragma unroll 1
    for (int p0 = 0; p0 * kPage < end; p0 += kScanPages) {
        const int mine = p0 + (int)threadIdx.x, ids = mine * kPage < end ? table[mine] : -1;
        bool found = false;
        s.bad[threadIdx.x] = 0;
        __syncwarp();
#pragma unroll 1
        for (int j = 0; j < 32; ++j) {           // the page of each lane
            const int id = __shfl_sync(0xffffffffu, ids, j);
            if (id < 0 || id >= a.pages) continue;
            const uint4* v = reinterpret_cast<const uint4*>(a.pool + (((int64_t)id * a.h_kv + head) * 2 + 1) * kPage * D) + lane;
#pragma unroll 4
            for (int i = 0; i < kRounds; ++i) {
                const uint4 x = v[32 * i];
                // an exponent of ones carries into the bit above it
                const auto carry = [](uint32_t u) { return (u & 0x7f807f80u) + 0x00800080u; };
                if ((carry(x.x) | carry(x.y) | carry(x.z) | carry(x.w)) & 0x80008000u) {
                    found = true;
                    atomicOr(&s.bad[warp * 32 + j], 1u << ((32 * i + lane) / kLanes));
                }
            }
        }
        if (!__syncthreads_or(found)) continue;
#pragma unroll 1
        for (int j = 0; j < kScanPages; ++j) {
#pragma unroll 1
            for (uint32_t bad = s.bad[j]; bad; bad &= bad - 1) {
                const int local = __ffs(bad) - 1;
                const uint16_t* key = a.pool + (((int64_t)table[p0 + j] * a.h_kv + head) * 2 * kPage + local) * D + lane * kChannels;
#pragma unroll 1
                for (int k = warp; k < 32; k += kJoinWarps) {
                    if ((p0 + j) * kPage + local >= s.seen[k]) continue;
                    float dot = 0.0f;
#pragma unroll 1
                    for (int c = 0; c < kChannels; ++c) dot += bf16_lo(s.q[k][lane * kChannels + c]) * bf16_lo(key[c]);
                    const float one = warp_sum(dot) * a.scale_log2 > -INFINITY ? 1.0f : 0.0f;
#pragma unroll 1
                    for (int c = 0; c < kChannels; ++c) {
                        const float v = bf16_lo(key[kPage * D + c]);
                        if (!(fabsf(v) < INFINITY)) s.acc[k][lane * kChannels + c] += one * v;
                    }
                }
            }
        }
        __syncthreads();                         // before the next stretch's pages
    }
#pragma unroll 1
    for (int k = warp; k < 32; k += kJoinWarps) {
        if (s.seen[k] == 0) continue;
        uint32_t want = 0;
#pragma unroll 1
        for (int c = 0; c < kChannels; ++c) {
            uint16_t& to = s.out[k][lane * kChannels + c];
            const float odd = s.acc[k][lane * kChannels + c];
            if (odd != 0.0f)
                to = (uint16_t)bf16_pair(odd, 0.0f);
            else if ((to & 0x7f80) == 0x7f80)
                want |= 1u << c;
        }
        s.want[k][lane] = (uint8_t)want;
        if (want) atomicOr(&s.todo, 1u << k);
    }
    __syncthreads();
#pragma unroll 1
    for (float unit = 1.0f; s.todo; unit = 0x1p-31f) form_rows<D>(a, table, head, end, unit, s, lane, warp);
    __syncthreads();
}

// Whether an item's indexes lie within the call's buffers: a CTA that gave up leaves entries of the list unwritten.
__device__ __forceinline__ bool sane(const ChunkArgs& a, const Work& w, const Item& it, int item, int g_log2) {
    if (it.b < 0 || it.b >= a.batch || it.head < 0 || it.head >= a.h_kv || it.tok0 < 0 || it.tok0 >= a.n || it.r0 < 0 ||
        it.rows < 1 || it.rows > kChunkRows || it.r0 > (a.n << g_log2) || it.tok0 + ((it.r0 + it.rows - 1) >> g_log2) >= a.n ||
        it.total < 0 || it.total > a.stride * kPage)
        return false;
    if (it.part < 0) return true;
    if (it.pieces < 2 || it.pieces > min(w.item_cap, 1 << 22) || it.piece < 0 || it.piece >= it.pieces || it.step < 1 || it.lead < 0 ||
        it.step > w.part_cap || it.lead > w.part_cap || it.stride < 1 || it.stride > a.h_kv)
        return false;
    const long long base = it.part - (long long)it.piece * it.step - (it.piece ? 0 : it.lead);
    const long long first = item - (long long)it.piece * it.stride, last = first + (long long)(it.pieces - 1) * it.stride;
    return base >= 0 && base + (long long)(it.pieces - 1) * it.step + it.rows <= w.part_cap && base + it.lead + it.rows <= w.part_cap &&
           first >= 0 && last < w.item_cap;
}

// Whole items' marked rows, a word of 32 each. Rows side by side are marked together, hence a CTA's words, one of each
// thread, lie far apart, and where there are fewer words than CTAs `shares` of them take some rows of each.
template <int D>
__device__ __noinline__ void look_at_words(const ChunkArgs& a, const Work& w, int items, Again<D>& s) {
    const unsigned count = (unsigned)items * 8, shares = clamp_int((int)(gridDim.x / max(count, 1u)), 1, 32);
#pragma unroll 1
    for (unsigned u0 = 0; u0 < count * shares; u0 += gridDim.x * kJoinThreads) {
        const unsigned mine = u0 + threadIdx.x * gridDim.x + blockIdx.x;
        uint32_t word = mine / shares < count ? w.odd[mine / shares] : 0;
#pragma unroll 1
        for (unsigned i = 0; word && i < 32; ++i)
            if (i % shares != mine % shares) word &= ~(1u << i);
        s.words[threadIdx.x] = word;
        if (!__syncthreads_or(word != 0)) continue;
#pragma unroll 1
        for (int i = 0; i < kJoinThreads; ++i) {
            if (!s.words[i]) continue;
            const unsigned at = (u0 + i * gridDim.x + blockIdx.x) / shares;
            const Item it = w.items[at / 8];
            if (it.part < 0 && sane(a, w, it, (int)(at / 8), 31 - __clz(a.g))) look_again<D>(a, w.items + at / 8, 32 * (int)(at % 8), s.words[i], s);
        }
        __syncthreads();
    }
}

// Adds the parts of cut items, in their order: a piece's CTA takes its share of the rows, a warp a row. Rows that are
// marked, in any of the pieces too, or whose parts' sum is not finite are looked at again.
template <int D>
__global__ void __launch_bounds__(kJoinThreads, D == 64 ? 4 : 2) chunk_join_kernel(const __grid_constant__ ChunkArgs a,
                                                                  const __grid_constant__ Work w) {
    constexpr int kChannels = D / 32, kDepth = 8;
    __shared__ Again<D> again;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g_log2 = 31 - __clz(a.g);
    grid_release();
    again.words[threadIdx.x] = 0;
    __syncthreads();
    grid_wait();
    Header head = *w.head;
    int marked = 0;
    for (int i = threadIdx.x; i < w.sms; i += kJoinThreads) marked |= w.marked[i];
    head.items = clamp_int(head.items, 0, w.item_cap);
    // with more CTAs than items, `per` of them share an item's rows
    const int per = max((int)gridDim.x / max(head.items, 1), 1), sub = (int)blockIdx.x / max(head.items, 1);
    const int first = !head.cut || sub >= per ? head.items : per > 1 ? (int)blockIdx.x % head.items : (int)blockIdx.x;
#pragma unroll 1
    for (int item = first; item < head.items; item += gridDim.x) {
        const Item it = w.items[item];
        if (it.part < 0 || !sane(a, w, it, item, g_log2)) continue;
        const int base = it.part - it.piece * it.step - (it.piece ? 0 : it.lead);
        auto part_of = [&](int p, int local) { return base + p * it.step + (p ? 0 : it.lead) + local; };
        const int end = it.rows * (it.piece + 1) / it.pieces;
        bool look = false;
#pragma unroll 1
        for (int local = it.rows * it.piece / it.pieces + sub * kJoinWarps + warp; local < end;
             local += per * kJoinWarps) {
            float m = kNoReference, sum = 0.0f, acc[kChannels] = {};
            bool odd = false, nan = false;
#pragma unroll 1
            for (int p0 = 0; p0 < it.pieces; p0 += 32) {
                const int p = p0 + lane;
                float2 ml = make_float2(kNoReference, 0.0f);
                if (p < it.pieces) {
                    ml = w.part_ml[part_of(p, local)];
                    nan |= ml.y != ml.y;
                    odd |= w.odd[(int64_t)(item + (p - it.piece) * it.stride) * 8 + local / 32] >> (local % 32) & 1;
                }
                float top = ml.y != 0.0f ? fmaxf(m, ml.x) : m;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float back = exp2_approx(m - top);
                m = top;
                sum *= back;
#pragma unroll
                for (int c = 0; c < kChannels; ++c) acc[c] *= back;
                const float f = ml.y == 0.0f ? 0.0f : exp2_approx(ml.x - m);
                const int count = min(32, it.pieces - p0);
#pragma unroll 1
                for (int q0 = 0; q0 < count; q0 += kDepth) {
                    float x[kDepth][kChannels];
#pragma unroll
                    for (int k = 0; k < kDepth; ++k) {
                        const float* from = w.part_acc + (unsigned)(part_of(p0 + min(q0 + k, count - 1), local) * D + lane * kChannels);
#pragma unroll
                        for (int c = 0; c < kChannels; c += 2) *reinterpret_cast<float2*>(&x[k][c]) = *reinterpret_cast<const float2*>(from + c);
                    }
#pragma unroll
                    for (int k = 0; k < kDepth; ++k) {
                        // no weight: what the part holds does not count
                        const float fp = __shfl_sync(0xffffffffu, f, q0 + k), lp = __shfl_sync(0xffffffffu, ml.y, q0 + k);
                        if (q0 + k >= count || fp == 0.0f) continue;
                        sum += fp * lp;
#pragma unroll
                        for (int c = 0; c < kChannels; ++c) acc[c] += fp * x[k][c];
                    }
                }
            }
            const int r = it.r0 + local;
            float probe = 0.0f;                  // NaN where the parts' sum is infinite
#pragma unroll
            for (int c = 0; c < kChannels; ++c) probe += acc[c] * 0.0f;
            if (__any_sync(0xffffffffu, nan)) sum = NAN;
            if (__any_sync(0xffffffffu, odd || probe != 0.0f) && fabsf(sum) > 0.0f) {       // a number other than 0
                look = true;
                if (lane == 0) atomicOr(&again.words[local / 32], 1u << (local % 32));
            }
            const int64_t row = (int64_t)(it.tok0 + (r >> g_log2)) * (a.h_kv << g_log2) + (it.head << g_log2) + (r & (a.g - 1));
            store_bf16(a.out + row * D + lane * kChannels, acc, sum == 0.0f ? 0.0f : 1.0f / sum);
        }
        if (!__syncthreads_or(look)) continue;
#pragma unroll 1
        for (int k = 0; k < kChunkRows / 32; ++k) look_again<D>(a, w.items + item, 32 * k, again.words[k], again);
        if (threadIdx.x < kChunkRows / 32) again.words[threadIdx.x] = 0;
        __syncthreads();
    }
    if (__syncthreads_or(marked)) look_at_words<D>(a, w, head.items, again);
}

// ---- host ---------------------------------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// The pool as [pages H_kv 2][16 tokens][d], boxes of one page's 16 tokens x 64 channels, 128-byte swizzle.
bool make_pool_map(CUtensorMap* map, const ChunkArgs& a, int d) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, kPage, (cuuint64_t)a.pages * a.h_kv * 2};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)kPage * d * 2};
    const cuuint32_t box[3] = {64, kPage, 1}, step[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.pool), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const ChunkArgs& a, const ChunkPlan& plan, void* workspace, int num_sms, cudaStream_t st) {
    using L = Layout<D>;
    CUtensorMap map;
    if (!make_pool_map(&map, a, D)) return cudaErrorInvalidValue;
    cudaError_t e = smem_opt_in<chunk_attend_kernel<D>>(L::kBytes);
    if (e != cudaSuccess) return e;
    char* base = static_cast<char*>(workspace);
    // Few row blocks: every loader plans by itself, 2 us for a few (five tokens at 1,344: 10.5 us in all, 16.5 with the
    // kernel in front); its loops grow with them, and it has shared memory for 80. The kernel takes 7 to 9 us for 100
    // to 200 row blocks, and its items go to whichever CTA is free.
    const Work w{plan.unit_cap <= kSelfUnits && a.batch <= kSelfUnits, num_sms, plan.unit_cap, plan.item_cap, plan.part_cap,
                 reinterpret_cast<Header*>(base), reinterpret_cast<int*>(base + plan.tiles),
                 reinterpret_cast<int2*>(base + plan.units), reinterpret_cast<Item*>(base + plan.items),
                 reinterpret_cast<uint32_t*>(base + plan.odd), reinterpret_cast<int*>(base + plan.marked), reinterpret_cast<float2*>(base + plan.part_ml), reinterpret_cast<float*>(base + plan.part_acc),
                 plan.fold_rows, reinterpret_cast<float2*>(base + plan.fold_ml), reinterpret_cast<float*>(base + plan.fold_acc)};
    const int grid = num_sms < plan.item_cap ? num_sms : plan.item_cap;
    if (!w.self) {
        e = launch_dependent(chunk_plan_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0, st, 1, a, w);
        if (e != cudaSuccess) return e;
    }
    e = launch_dependent(chunk_attend_kernel<D>, dim3(grid), dim3(kThreads), L::kBytes, st, 1, a, w, map);
    if (e != cudaSuccess) return e;
    // rows that may be cut, a warp each; at least a CTA an SM, at most four (seven prompts of heads of 64: 25.5 us, 26.0 with
    // eight, and 24.7 with two, which costs 16 mixed requests 1.3 us and 32 drafts 2)
    const int64_t rows = (int64_t)a.n * a.g * a.h_kv, per = kJoinThreads / 32;
    const int joins = rows > 4 * per * num_sms ? 4 * num_sms : rows > per * num_sms ? (int)((rows + per - 1) / per) : num_sms;
    return launch_dependent(chunk_join_kernel<D>, dim3(joins), dim3(kJoinThreads), 0, st, 1, a, w);
}

}  // namespace

ChunkPlan plan_chunk(const Shape& s, int num_sms, int batch, int n) {
    const int g = s.h_q / s.h_kv;
    const int64_t rows = (int64_t)n * g;
    ChunkPlan p{};
    p.unit_cap = (int)((rows + kChunkRows - 1) / kChunkRows) + (batch < n ? batch : n);
    // cutting at L tiles makes all / L more items at most, L half an SM's share or more; the pieces of cut items are
    // longer than L / 2
    p.item_cap = p.unit_cap * s.h_kv + 2 * num_sms;
    p.fold_rows = (int)(rows < kChunkRows ? rows : kChunkRows);
    p.part_cap = 4 * num_sms * p.fold_rows;
    size_t at = 0;
    auto place = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    place(sizeof(Header));
    p.tiles = place(((size_t)batch + 1) * sizeof(int));
    p.units = place((size_t)p.unit_cap * sizeof(int2));
    p.items = place((size_t)p.item_cap * sizeof(Item));
    p.odd = place((size_t)p.item_cap * 8 * sizeof(uint32_t));
    p.marked = place((size_t)num_sms * sizeof(int));
    p.part_ml = place((size_t)p.part_cap * sizeof(float2));
    p.part_acc = place((size_t)p.part_cap * s.d * sizeof(float));
    p.fold_ml = place((size_t)num_sms * p.fold_rows * sizeof(float2));
    p.fold_acc = place((size_t)num_sms * p.fold_rows * s.d * sizeof(float));
    p.total = at;
    return p;
}

cudaError_t launch_chunk(const ChunkArgs& a, const ChunkPlan& plan, void* workspace, int d, int num_sms, cudaStream_t st) {
    return d == 128 ? launch<128>(a, plan, workspace, num_sms, st) : launch<64>(a, plan, workspace, num_sms, st);
}

}  // namespace oscar
