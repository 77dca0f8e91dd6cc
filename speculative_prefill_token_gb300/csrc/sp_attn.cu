// Attention of new tokens over a block-paged cache ("SpecPrefill —
// Implementation Guide", §How It Works / Sparse Prefill: the target's
// attention over the kept tokens, and its decode steps after them), on
// fifth-generation tensor cores.
//
// For a query row (token i of request b, head h) with visible cache indices
// [lo, hi), and KV head g = h / G,
//   out = sum_j exp2(y_j - m) v_j / sum_j exp2(y_j - m),  y_j = scale log2(e) <q, k_j>,
// in one pass over the keys: m is a reference at most 8 below the running
// maximum, and sum and accumulator are scaled by exp2(m_old - m_new) when it
// moves.
//
// Work. The G heads that share a KV head are rows of one query tile: 128 / G
// tokens x G heads, so a decode step reads each key once for all of them. An
// item is the query tiles of one request and KV head that one CTA holds at a
// time (two tiles of 128 rows for d <= 128, one for d = 256, whose
// accumulator fills the tensor memory); its unit is a tile of 128 keys. All
// units of all items are cut into equal contiguous ranges, one for each CTA
// (one CTA per SM), whatever the mix of lengths. The lengths live on the
// device: every CTA lays out a small batch itself, a one-CTA kernel before it a
// larger one. An item cut between CTAs leaves a part in the workspace for each
// of them (reference, sum and accumulator of each row), and another kernel
// joins the parts in their order, so results do not depend on timing. (Joined
// by the last CTA to finish instead, the 76 parts of a single long chunk were
// read by two CTAs: 244 us in place of 60 for 8 tokens over 32K, 24 now.)
//
// Roles (384 threads):
//   warps 0-7  two softmax warpgroups. A thread owns one row of a 128 x 128
//              logits tile: reads it from tensor memory, takes the maximum,
//              writes the weights back as 16-bit values in its place, keeps
//              the sum, and writes or joins the result at the item's end.
//   warp 8     K and V boxes by TMA (lane j issues box j of a slot)
//   warp 9     tcgen05.mma issuer and TMEM owner
//   warp 10    query tiles by TMA
//   warp 11    looks for infinities and NaN among values that some rows of an
//              item are masked from; CTA 0: the list of cut items for the join
// Two streams keep the tensor cores busy while the other stream's softmax
// runs: with two query tiles, one tile each; with one (decode steps, short
// chunks), even and odd key tiles, with an accumulator each for d <= 128
// (joined from tensor memory at the end) and one accumulator for d = 256.
//
// What bounds it (of 6,693 GB/s of a copy, 7,200 of a plain read of 2.6 GB and
// 1,908 TFLOP/s measured):
//   decode steps    the stream of keys and values: 64 requests of 2K to 32K
//                   tokens, 16 + 4 heads of 128, 366 to 376 us, 6.9 to 7.1 TB/s;
//                   16 of 4K to 16K, 8 + 2 heads of 256, 57 us, 5.3 TB/s (of it
//                   4.5 us until the first copy, and 2 to 5 us of the join)
//   d = 128, long   the chain logits -> softmax (some 1,700 cycles) -> weights
//                   of a tile, which two streams do not hide in full: 4,096
//                   tokens over 39K, 16 + 4 heads, 860 to 897 us, 1,395 to
//                   1,455 TFLOP/s by the machine's clock under power
//   d = 256         shared memory: operands of both products and the copies
//                   take 2,560 cycles of its bandwidth a tile, the products
//                   2,048: 4,916 tokens, 8 + 2 heads, 95 us, 1,045 TFLOP/s (10 of
//                   them the join, some 4 each of a CTA's two items' ends)
//   d = 64          latency of the softmax's chain: two of its warps on each
//                   scheduler, each tensor-memory load, maximum, exponentials and
//                   store in turn. No pipe is full: a prompt of 2,700 tokens, 8 +
//                   2 heads, has an instruction in 24 % of the issue slots, the
//                   tensor and exponential pipes busy 15 % each
//   single rows     latency: 9.0 to 9.5 us for a token over 512
//
// Every mbarrier wait is bounded; a wait that gives up records SP_ERR_TIMEOUT
// in the workspace status, and the CTA drains its copies and MMAs in flight
// and frees its tensor memory before it returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sp_device.cuh"
#include "sp_internal.h"
#include "sp_paged.h"
#include "sp_ptx.cuh"
#include "sp_ptx_attn.cuh"

namespace sp {
namespace {

constexpr int kKeys = 128;                 // keys of a tile (a unit of work)
constexpr int kRows = 128;                 // rows of a query tile
constexpr uint32_t kChunk = 16384;         // bytes of 128 rows x 64 elements
constexpr int kWarps = 12;
constexpr int kAttnThreads = 32 * kWarps;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kQWarp = 10, kListWarp = 11;
constexpr int kPlanThreads = 1024;
constexpr int64_t kDrainSpin = int64_t(1) << 22;
constexpr float kSlack = 8.0f;             // log2 units the reference may lag behind the maximum

constexpr float kLn2 = 0.6931471805599453f;

// fp16 weights are scaled by 2^6: their subnormals then start 20 binary
// orders below the maximum, and the largest weight is 2^14.
__host__ __device__ constexpr float weight_bias(bool bf16) { return bf16 ? 0.0f : 6.0f; }

// Whether weights and values are bf16: of bf16 queries, but for the values of a 4-bit cache (kOver),
// which fp16 holds as exactly and whose weights then keep three bits more (the long chunk's error of 0.0023
// relative to 64 bits becomes 0.0017, that of the result's own rounding).
__host__ __device__ constexpr bool bf16_values(bool bf16, bool over) { return bf16 && !over; }

__host__ __device__ constexpr int tiles_per_item(int d) { return d <= 128 ? 2 : 1; }
// A ring slot holds a whole K or V tile (d = 256: half of one): the MMA warp
// waits once for each. (16 KB slots at d = 128: a wait before every four MMAs,
// 100 cycles that the MMA queue is too short to hide.)
__host__ __device__ constexpr int slots_per_tile(int d) { return d == 256 ? 2 : 1; }
__host__ __device__ constexpr int ring_slots(int d) { return d == 64 ? 12 : 5; }

// One item: rows of `ntok` tokens from row tok0 of q, the first at cache
// index pos0; keys [klo, khi) are seen by some row, in tiles
// [tile0, tile0 + ntiles).
struct alignas(16) Item {
    int32_t b, tok0, ntok, pos0, klo, khi, tile0, ntiles;
};

// Where a CTA's range starts (and the one before it ends): key tile `off` of
// item `item` of KV head g.
struct alignas(16) Start {
    int32_t item, g, off, pad;
};

// A cut item: its parts lie with CTAs c0 .. c0 + parts - 1.
struct alignas(16) Job {
    int32_t c0, parts, g, c0_head;      // c0_head: CTA c0 starts with the item
    int32_t tok0, ntok;
    int32_t task0;                      // tasks of the join kernel before it
    int32_t pad;
};

struct PlanHead {
    int32_t items;    // of one KV head; 0: nothing to do
    int32_t jobs, tasks, pad;
    int64_t units;    // cost of one KV head
};

struct AttnArgs {
    const int32_t* q_off;
    const int32_t* kv_len;
    const int32_t* table;
    const int32_t* only;   // with kOver, [B]: requests below 0 are left out
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* out;
    float* lse;
    int32_t* status;
    PlanHead* head;
    Item* items;
    int64_t* pre;       // cost before each item, [items + 1]
    int32_t* req_item;  // first item of each request, [B + 1]
    Start* starts;      // [grid + 1]
    Job* jobs;          // [grid]
    float* part_o;      // [grid * 2][tiles][128][d]
    float2* part_ml;    // [grid * 2][tiles][128] (reference, sum)
    int64_t q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh, pool_tokens, spin;
    int B, hk, G, tq, bs, table_stride, cap, causal, window, grid, item_cost;
    int wide_out;        // 32-byte stores of out are aligned
    int local_plan;      // every CTA lays out the batch itself
    int hk_shift, hv_shift;  // rows of a K and of a V box, as powers of two
    uint32_t q_bytes;    // of one 64-element chunk of a query tile
    float scale2;
    float out_scale;     // with kOver: factor of the result
};

// kOver, of the kernels below: called over the 16-bit copy of a 4-bit cache (sp_fp4_attn.cu). Kernels of
// their own, as the choice at run time took the others 0.2 of 9.5 us for one token over 512
// and 0.4 of 50.9 for 24 mixed requests.

// ------------------------------------------------------------ plan

constexpr int kMaxCtas = 256;
constexpr int kLocalItems = 384;   // items and requests of a plan made by every CTA
// Cost of an item besides its key tiles, in tiles: loading the queries,
// filling the pipeline and writing the rows. (Without it the CTAs with the
// shortest items of a prompt finish last: 8,200 cycles at d = 256, where a tile
// takes 3,100, 5,300 at d = 64 and 2,700. At 1, 2, 3 and 4: 4,916 tokens at
// d = 256 118, 101, 98, 100 us; 24 mixed requests at d = 64 57, 53, 54, 55 us.)
constexpr int item_cost(int d) { return d == 256 ? 3 : 2; }
constexpr int kJoinFew = 4;        // parts held in registers at once
constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 3;     // of an SM, all resident (80 registers a thread)
constexpr int kJoinGroups = kJoinThreads / 16;   // of 16 threads: 64 columns of a row
// Rows of two parts that a group has in flight: their latency is the join of a
// prompt, whose items are mostly cut once. (4,916 tokens at d = 256, whole call:
// one row and four blocks an SM 104 us, two and three 101, four and two 101.)
constexpr int kJoinRows = 2;

// Whether the groups of a join block share a row and its parts, or take a row
// each: with few rows the parts' latency counts, with many (of some parts) the
// blocks. (8 tokens over 32K, 76 parts: 25 us of the whole call shared, 45 a row
// each; 702 tokens of one request, 5 parts: 18 us a row each, 23.5 shared.)
__device__ __forceinline__ bool join_shares(int parts, int row_chunks) {
    return parts > 16 || (parts > kJoinFew && row_chunks <= 128);
}

template <typename T>
__device__ __forceinline__ T range_start(T total, int ctas, int c) { return total * c / ctas; }

// The CTA whose range holds unit u of `total`.
__device__ __forceinline__ int range_owner(int64_t total, int ctas, int64_t u) {
    return static_cast<int>(((u + 1) * ctas - 1) / total);
}

// Exclusive sums over the block's NT threads, and their total.
template <int NT, typename T>
__device__ __forceinline__ T block_scan(T v, T* sums, T* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    const T mine = lane < NT / 32 ? sums[lane] : 0;
    T all = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T x = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += x;
    }
    *total = __shfl_sync(0xffffffffu, all, 31);
    return __shfl_sync(0xffffffffu, all - mine, warp) + incl - v;
}

// The item that begins at token `first` of a request's nq new ones.
__device__ __forceinline__ Item make_item(const AttnArgs& a, int b, int q0, int nq, int kv, int first, int tpi) {
    Item it;
    it.b = b;
    it.tok0 = q0 + first;
    it.ntok = min(nq - first, tpi);
    it.pos0 = kv - nq + first;
    it.khi = a.causal ? max(0, min(kv, it.pos0 + it.ntok)) : kv;
    it.klo = a.window > 0 ? max(0, it.pos0 - a.window + 1) : 0;
    it.tile0 = it.klo / kKeys;
    it.ntiles = it.khi > it.klo ? (it.khi + kKeys - 1) / kKeys - it.tile0 : 0;
    return it;
}

// Last index i in [0, n) with v[i] <= x (v[0] <= x).
template <typename T, typename U>
__device__ __forceinline__ int last_at_most(const T* v, int n, U x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// Start of CTA c's range: ranges of equal cost; a cut inside an item's fixed
// cost falls on the item's start.
template <typename T>
__device__ __forceinline__ Start make_start(const AttnArgs& a, const T* pre, int items, T units, int c) {
    const T all = units * a.hk;
    const int ctas = static_cast<int>(min(static_cast<T>(a.grid), all));
    Start s{0, a.hk, 0, 0};   // the end of everything
    if (c < ctas) {
        const T begin = range_start(all, ctas, c);
        s.g = static_cast<int32_t>(begin / units);
        const T u = begin - s.g * units;
        s.item = last_at_most(pre, items, u);
        s.off = static_cast<int32_t>(max(u - pre[s.item] - a.item_cost, static_cast<T>(0)));
    }
    return s;
}

// The same, not inlined: for the list of all starts, which CTA 0 makes beside its work. (The loop's
// instructions between the start and the streams' loops moved the long chunk at d = 128 from 851 to 864 us.)
template <typename T>
__device__ __noinline__ Start listed_start(const AttnArgs& a, const T* pre, int items, T units, int c) {
    return make_start(a, pre, items, units, c);
}

// (cache indices stay below 2^30, so that no sum of two of them leaves 31 bits)
__device__ __forceinline__ bool bad_request(const AttnArgs& a, int64_t lo, int64_t hi, int64_t kv) {
    return hi < lo || hi > a.cap || kv < 0 || kv > kMaxCached || (kv + a.bs - 1) / a.bs > a.table_stride;
}

// Requests that the caller computes elsewhere. It has looked at their lengths: their
// contexts may be longer than this call's table holds.
template <bool kOver>
__device__ __forceinline__ bool left_out(const AttnArgs& a, int b) {
    if constexpr (kOver) return a.only[b] < 0;
    else return false;
}

// Lays out a batch of any size, by one block of its own: items with their
// costs, and the CTAs' ranges. Bound by the latency of its scans.
template <bool kOver>
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const AttnArgs a, int tiles) {
    __shared__ int64_t sums[32];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    const int tpi = a.tq * tiles;   // tokens per item
    int bad = tid == 0 ? a.q_off[0] != 0 : 0;
    int64_t items = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int64_t n = 0;
        if (b < a.B) {
            const int64_t lo = a.q_off[b], hi = a.q_off[b + 1];
            if (!left_out<kOver>(a, b)) {
                if (bad_request(a, lo, hi, a.kv_len[b])) bad = 1;
                else n = (hi - lo + tpi - 1) / tpi;
            }
        }
        int64_t total;
        const int64_t at = items + block_scan<kPlanThreads>(n, sums, &total);
        if (b < a.B) a.req_item[b] = static_cast<int32_t>(at);
        items += total;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
        items = 0;
    }
    int64_t units = 0;
    for (int64_t i0 = 0; i0 < items; i0 += kPlanThreads) {
        const int64_t i = i0 + tid;
        int64_t n = 0;
        if (i < items) {
            // the last request whose first item is at or before i: requests
            // without new tokens share the next one's first item
            const int b = last_at_most(a.req_item, a.B, i);
            const int q0 = a.q_off[b];
            const Item it = make_item(a, b, q0, a.q_off[b + 1] - q0, a.kv_len[b],
                                      static_cast<int>(i - a.req_item[b]) * tpi, tpi);
            n = it.ntiles + a.item_cost;
            a.items[i] = it;
        }
        int64_t total;
        const int64_t at = units + block_scan<kPlanThreads>(n, sums, &total);
        if (i < items) a.pre[i] = at;
        units += total;
    }
    if (tid == 0) {
        a.pre[items] = units;
        PlanHead h = {};
        h.items = static_cast<int32_t>(items);
        h.units = units;
        *a.head = h;
    }
    __syncthreads();
    for (int c = tid; c <= a.grid; c += kPlanThreads)
        a.starts[c] = make_start(a, a.pre, static_cast<int>(items), units, c);
}

// The same of a small batch (at most kLocalItems items and requests, costs of
// 32 bits), by every CTA of the attention kernel for itself: no launch before
// it, and its own range and first item are at hand. (By this and by the plan
// kernel: one token 9.9 and 12.0 us, 16 decodes 57.6 and 60.2, 24 mixed requests
// 52.6 and 55.7; a prompt of 4,916 tokens the same.)
struct LocalPlan {
    int32_t sums[32];
    int32_t q0[kLocalItems], nq[kLocalItems], kv[kLocalItems], req_item[kLocalItems], pre[kLocalItems + 1];
};

// What a CTA starts from.
struct alignas(16) Range {
    Start begin, end;
};

template <bool kOver>
__device__ __forceinline__ int local_plan(const AttnArgs& a, int tiles, LocalPlan& p, Range* range) {
    const int t = threadIdx.x;
    const int tpi = a.tq * tiles;
    int bad = 0, n = 0;
    if (t < a.B) {
        const int lo = a.q_off[t], hi = a.q_off[t + 1], kv = a.kv_len[t];
        const bool out = left_out<kOver>(a, t);
        bad = (!out && bad_request(a, lo, hi, kv)) || (t == 0 && lo != 0);
        if (!bad && !out) n = (hi - lo + tpi - 1) / tpi;
        p.q0[t] = lo;
        p.nq[t] = hi - lo;
        p.kv[t] = kv;
    }
    if (__syncthreads_or(bad)) {
        if (t == 0) {
            atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
            if (blockIdx.x == 0) a.head->items = 0;
        }
        return 0;
    }
    int items, units;
    const int at = block_scan<kAttnThreads>(n, p.sums, &items);
    if (t < a.B) p.req_item[t] = at;
    __syncthreads();
    n = 0;
    if (t < items) {
        const int b = last_at_most(p.req_item, a.B, t);
        const Item it = make_item(a, b, p.q0[b], p.nq[b], p.kv[b], (t - p.req_item[b]) * tpi, tpi);
        n = it.ntiles + a.item_cost;
        a.items[t] = it;   // (every CTA writes the same; each reads what it wrote)
    }
    const int before = block_scan<kAttnThreads>(n, p.sums, &units);
    if (t < items) p.pre[t] = before;
    if (t == 0) p.pre[items] = units;
    __syncthreads();
    if (items > 0 && t < 2) {
        const Start s = make_start(a, p.pre, items, units, static_cast<int>(blockIdx.x) + t);
        if (t == 0) range->begin = s;
        else range->end = s;
    }
    if (blockIdx.x == 0) {   // for the list of cut items
        for (int c = t; c <= a.grid && items > 0; c += kAttnThreads) a.starts[c] = listed_start(a, p.pre, items, units, c);
        for (int i = t; i <= items; i += kAttnThreads) a.pre[i] = p.pre[i];
        if (t == 0) {
            a.head->items = items;
            a.head->units = units;
        }
    }
    return items;
}

// The cut items, listed for the join kernel by one warp of CTA 0 while the
// others work.
__device__ __forceinline__ void list_cuts(const AttnArgs& a, int chunks, int lane) {
    constexpr unsigned kAll = 0xffffffffu;
    const int items = __ldcg(&a.head->items);
    const int64_t units = __ldcg(&a.head->units), all = units * a.hk;
    const int ctas = items > 0 ? static_cast<int>(min(static_cast<int64_t>(a.grid), all)) : 0;
    int jobs = 0, tasks = 0;
    for (int x0 = 1; x0 < ctas; x0 += 32) {
        const int x = x0 + lane;
        Job j = {};
        int mine = 0;
        if (x < ctas) {
            const int4 s = __ldcg(reinterpret_cast<const int4*>(a.starts + x));
            const int4 b = __ldcg(reinterpret_cast<const int4*>(a.starts + x - 1));
            const bool same = b.x == s.x && b.y == s.y;   // (item, g, off)
            if (s.z > 0 && !(same && b.z > 0)) {          // the first cut inside the item
                const int64_t last = s.y * units + __ldcg(a.pre + s.x + 1) - 1;
                j.c0 = x - 1;
                j.parts = range_owner(all, ctas, last) - j.c0 + 1;
                j.g = s.y;
                j.c0_head = same;
                j.tok0 = __ldcg(&a.items[s.x].tok0);
                j.ntok = __ldcg(&a.items[s.x].ntok);
                mine = j.ntok * a.G * chunks;
                if (!join_shares(j.parts, mine)) mine = (mine + kJoinGroups * kJoinRows - 1) / (kJoinGroups * kJoinRows);
            }
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned who = __ballot_sync(kAll, mine > 0);
        j.task0 = tasks + incl - mine;
        if (mine > 0) a.jobs[jobs + __popc(who & ((1u << lane) - 1))] = j;
        jobs += __popc(who);
        tasks += __shfl_sync(kAll, incl, 31);
    }
    if (lane == 0) {
        a.head->jobs = jobs;
        a.head->tasks = tasks;
    }
}

// ------------------------------------------------------------ segments

// A CTA's part of one item: key tiles [first, first + n) (n = 0 for an item
// that sees no key), and whether other CTAs hold the rest.
struct Segment {
    Item it;
    int g, first, n;
    bool split, head;   // head: the CTA's first segment
};

// Walks a CTA's range; every role takes the same steps.
struct Walk {
    int item, g, off, items;
    int end_item, end_g, end_off;
    bool head;
    __device__ __forceinline__ Walk(const Range* r, int n_items) {
        item = r->begin.item;
        g = r->begin.g;
        off = r->begin.off;
        end_item = r->end.item;
        end_g = r->end.g;
        end_off = r->end.off;
        items = n_items;
        head = true;
    }
    __device__ __forceinline__ bool next(const AttnArgs& a, Segment& s) {
        if (g > end_g || (g == end_g && (item > end_item || (item == end_item && off >= end_off)))) return false;
        const int4* p = reinterpret_cast<const int4*>(a.items + item);
        const int4 x = __ldcg(p), y = __ldcg(p + 1);
        s.it = Item{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        s.g = g;
        s.first = s.it.tile0 + off;
        s.n = (g == end_g && item == end_item ? end_off : s.it.ntiles) - off;
        s.split = s.n < s.it.ntiles;
        s.head = head;
        head = false;
        off = 0;
        if (++item == items) {
            item = 0;
            ++g;
        }
        return true;
    }
};

// Two query tiles, each with its own stream, or one tile whose key tiles
// alternate between the streams.
__device__ __forceinline__ bool two_tiles(const AttnArgs& a, const Segment& s, int d) {
    return d <= 128 && s.it.ntok > a.tq;
}

// Ring order of a segment's tiles: K0 V0 K1 V1 ... with two query tiles,
// K0 K1 V0 K2 V1 ... with alternating key tiles. Position of V_j:
__device__ __forceinline__ int v_position(bool two, int j, int n) {
    return two ? 2 * j + 1 : min(2 * j + 2, 2 * n - 1);
}

// ------------------------------------------------------------ shared memory

template <int D>
struct Smem {
    static constexpr int kTiles = tiles_per_item(D);
    static constexpr int kChunks = D / 64;         // 64-element chunks of a row
    static constexpr int kParts = slots_per_tile(D);
    static constexpr int kSlots = ring_slots(D);
    static constexpr uint32_t kSlot = kChunks / kParts * kChunk;   // bytes
    static constexpr int kSlotChunks = kChunks / kParts;           // of a K slot (128 keys)
    static constexpr int kSlotKeys = kKeys / kParts;               // of a V slot (all chunks)
    static constexpr uint32_t q = 0;
    static constexpr uint32_t ring = kTiles * kChunks * kChunk;
    static constexpr uint32_t stat = ring + kSlots * kSlot;   // [2][128] float2
    static constexpr uint32_t range = stat + 2 * kRows * 8;
    static constexpr uint32_t bars = range + sizeof(Range);
    static constexpr uint32_t full = bars;
    static constexpr uint32_t empty = full + 8 * kSlots;
    static constexpr uint32_t qfull = empty + 8 * kSlots;
    static constexpr uint32_t qempty = qfull + 8;
    static constexpr uint32_t sfull = qempty + 8;     // [2] logits written
    static constexpr uint32_t pfull = sfull + 16;     // [2] weights written
    static constexpr uint32_t odone = pfull + 16;     // [2] weights of a stream buffer in the accumulator
    static constexpr uint32_t oempty = odone + 16;    // [2] accumulator read
    static constexpr uint32_t statfull = oempty + 16; // [2] second stream's sums written
    static constexpr uint32_t drain = statfull + 16;
    static constexpr uint32_t tmem = drain + 8;
    static constexpr uint32_t abort = tmem + 8;
    static constexpr uint32_t odd = abort + 4;        // [3] a value of the segment is no number; of any segment
    static constexpr uint32_t checked = odd + 12;     // [2] that flag is written
    static constexpr uint32_t seen = checked + 16;    // [2] and read
    static constexpr uint32_t total = seen + 16;
};

static_assert(Smem<64>::total <= 232448 && Smem<128>::total <= 232448 && Smem<256>::total <= 232448,
              "shared memory of one CTA");

struct Ctx {
    uint8_t* smem;
    uint32_t base;
    volatile int* abort_flag;
    int32_t* status;
    int64_t spin;
    const Range* range;
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
        if (mbar_wait_bounded(base + bar, parity & 1, spin, abort_flag)) return true;
        *abort_flag = 1;
        atomicCAS(status, 0, static_cast<int32_t>(SP_ERR_TIMEOUT));
        return false;
    }
};

// ------------------------------------------------------------ loads

// K and V boxes of the CTA's segments, by the whole warp. Boxes outside the
// item's keys [klo, khi) are not loaded (their blocks may be gone); the
// softmax warps zero the V rows outside before they are used.
template <int D>
__device__ __forceinline__ void load_keys(const Ctx& c, const AttnArgs& a, const CUtensorMap* mk,
                                          const CUtensorMap* mv, int items, int lane) {
    using L = Smem<D>;
    constexpr unsigned kAll = 0xffffffffu;
    constexpr int P = L::kParts, kPer = L::kSlotKeys;
    // (few instructions per slot: the warp shares its scheduler with two softmax
    // warps, and at 120 instructions a slot its own arithmetic set the rate)
    const int nk = kKeys >> a.hk_shift, hk = 1 << a.hk_shift;   // K boxes of a tile, their rows
    const int sub = kPer >> a.hv_shift, hv = 1 << a.hv_shift;   // V boxes of a slot
    const uint32_t k_dst = c.base + L::ring + static_cast<uint32_t>(lane << a.hk_shift) * (L::kSlotChunks * 128u);
    const uint32_t v_dst = c.base + L::ring + static_cast<uint32_t>(lane << a.hv_shift) * (L::kChunks * 128u);
    const int key_v = lane << a.hv_shift;    // this lane's V box, within its slot
    const int per_block = a.bs >> 7;         // tiles of a block (0: blocks of a tile)
    int slot = 0;
    uint32_t turn = 0;
    bool ok = true;

    // pool row / 8 of this lane's K box of a tile; -1 outside the item's keys
    auto lookup = [&](const Segment& s, int tile) -> int {
        const int key = tile * kKeys + (lane << a.hk_shift);
        if (lane >= nk || key >= s.it.khi || key + hk <= s.it.klo) return -1;
        const int blk = per_block > 1 ? tile / per_block : per_block ? tile : tile * nk + lane;
        const int within = per_block > 1 ? (tile - blk * per_block) * kKeys : 0;
        const int id = a.table[static_cast<int64_t>(s.it.b) * a.table_stride + blk];
        const int64_t row = static_cast<int64_t>(id) * a.bs;
        if (id < 0 || row + a.bs > a.pool_tokens) {
            atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
            return 0;
        }
        return static_cast<int>((row + within) >> 3);
    };
    // the next slot, once it is empty, for `bytes`
    auto acquire = [&](uint32_t bytes) -> bool {
        ok = __all_sync(kAll, c.wait(L::empty + 8 * slot, turn ^ 1));
        if (ok && lane == 0) mbar_arrive_expect_tx(c.base + L::full + 8 * slot, bytes);
        __syncwarp();
        return ok;
    };
    auto advance = [&]() {
        if (++slot == L::kSlots) {
            slot = 0;
            turn ^= 1;
        }
    };
    auto put_k = [&](const Segment& s, int group) {
        const uint32_t bytes = __popc(__ballot_sync(kAll, group >= 0)) * (static_cast<uint32_t>(hk) * L::kSlotChunks * 128u);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (!acquire(bytes)) return;
            if (group >= 0)
                tma_load_5d(k_dst + slot * L::kSlot, mk, c.base + L::full + 8 * slot, 0, 0, p * L::kSlotChunks, group, s.g);
            advance();
        }
    };
    auto put_v = [&](const Segment& s, int tile, int group) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            // the rows of a V box lie in the block of a K box of the tile
            const int key = p * kPer + key_v, at = tile * kKeys + key;
            const int first = __shfl_sync(kAll, group, key >> a.hk_shift & 31);
            const bool there = lane < sub && first >= 0 && at < s.it.khi && at + hv > s.it.klo;
            const uint32_t bytes = __popc(__ballot_sync(kAll, there)) * (static_cast<uint32_t>(hv) * L::kChunks * 128u);
            if (!acquire(bytes)) return;
            if (there)
                tma_load_5d(v_dst + slot * L::kSlot, mv, c.base + L::full + 8 * slot, 0, 0, 0, first + ((key & (hk - 1)) >> 3), s.g);
            advance();
        }
    };

    Walk w(c.range, items);
    Segment s;
    while (ok && w.next(a, s)) {
        if (s.n == 0) continue;
        const bool two = two_tiles(a, s, D);
        int group = lookup(s, s.first), next = -1;
        if (s.n > 1) next = lookup(s, s.first + 1);
        if (!two) put_k(s, group);
        for (int j = 0; j < s.n && ok; ++j) {
            const int after = j + 2 < s.n ? lookup(s, s.first + j + 2) : -1;
            if (two) put_k(s, group);
            else if (j + 1 < s.n) put_k(s, next);
            if (ok) put_v(s, s.first + j, group);
            group = next;
            next = after;
        }
    }
    // every copy this warp issued lands before it leaves: slots before `slot`
    // were last used in this turn of the ring, the others in the one before
    // (a wait on a first turn's parity 1 returns at once)
    if (lane == 0)
        for (int i = 0; i < L::kSlots; ++i)
            mbar_wait_spin(c.base + L::full + 8 * i, i < slot ? turn : turn ^ 1, kDrainSpin);
}

template <int D>
__device__ __forceinline__ void load_queries(const Ctx& c, const AttnArgs& a, const CUtensorMap* mq, int items) {
    using L = Smem<D>;
    Walk w(c.range, items);
    Segment s;
    uint32_t n = 0;
    while (w.next(a, s)) {
        if (s.n == 0) continue;
        const int tiles = two_tiles(a, s, D) ? 2 : 1;
        if (!c.wait(L::qempty, (n & 1) ^ 1)) break;
        mbar_arrive_expect_tx(c.base + L::qfull, a.q_bytes * L::kChunks * tiles);
        for (int t = 0; t < tiles; ++t)
            for (int ch = 0; ch < L::kChunks; ++ch)
                tma_load_3d(c.base + L::q + (t * L::kChunks + ch) * kChunk, mq, c.base + L::qfull, ch * 64, s.g * a.G,
                            s.it.tok0 + t * a.tq);
        ++n;
    }
    if (n) mbar_wait_spin(c.base + L::qfull, (n - 1) & 1, kDrainSpin);
}

// ------------------------------------------------------------ values

// The values of keys that some rows of an item see and others are masked from
// are looked at: a zero weight times infinity or NaN is NaN, and a tile's
// product takes all its rows through all its keys. (Keys that no row sees are
// never loaded, or zeroed.)
__device__ __forceinline__ bool looked_at(const AttnArgs& a, const Segment& s) {
    return a.causal && s.n > 0 && s.it.ntok > 1;
}

// Adds 0 * x of the eight values of x to acc: not zero once one is infinite or NaN.
template <bool kBf16>
__device__ __forceinline__ void add_zero_times(uint32_t& acc, uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kBf16)
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w[i]), "r"(0u));
        else
            asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w[i]), "r"(0u));
    }
}

// Whether one of those values is infinite or NaN, by one warp from global
// memory (some 100 rows per item).
template <int D, bool kBf16>
__device__ __forceinline__ bool odd_values(const AttnArgs& a, const Segment& s, int lane) {
    constexpr int kLanes = D / 8, kStep = 32 / kLanes;   // lanes of a row, rows at a time
    const int k0 = s.first * kKeys, k1 = (s.first + s.n) * kKeys;
    const int last = s.it.pos0 + s.it.ntok - 1;
    uint32_t acc = 0;
    // keys behind the first row's position, keys before the last row's window
#pragma unroll 1
    for (int part = 0; part < (a.window > 0 ? 2 : 1); ++part) {
        const int lo = max(part ? s.it.klo : max(s.it.klo, s.it.pos0 + 1), k0);
        const int hi = min(part ? min(s.it.khi, last - a.window + 1) : s.it.khi, k1);
        // block by block, a lane for each 16 bytes of a row
        const int per = a.bs;
        int blk = lo / per, in = lo - blk * per;
        const int32_t* tab = a.table + static_cast<int64_t>(s.it.b) * a.table_stride;
        for (int j = lo; j < hi; ++blk, in = 0) {
            const int id = tab[blk];
            int64_t row = static_cast<int64_t>(id) * per;
            if (id < 0 || row + per > a.pool_tokens) row = 0;
            const int n = min(per - in, hi - j);
            const uint16_t* p = a.v + (row + in + lane / kLanes) * a.v_st + s.g * a.v_sh + lane % kLanes * 8;
            const int64_t step = kStep * a.v_st;
#pragma unroll 4
            for (int i = lane / kLanes; i < n; i += kStep, p += step) add_zero_times<kBf16>(acc, *reinterpret_cast<const uint4*>(p));
            j += n;
        }
    }
    return __any_sync(0xffffffffu, (acc & 0x7fff7fffu) != 0);
}

// By a warp of its own: one flag per segment. The softmax warps write no rows of
// a flagged segment; they take them one by one when their range is done. It
// costs a prefill at d = 256 4 % of its time; by the softmax warps, from the
// ring, it was 20 %.
template <int D, bool kBf16V>
__device__ __forceinline__ void check_values(const Ctx& c, const AttnArgs& a, int items, int lane) {
    using L = Smem<D>;
    constexpr unsigned kAll = 0xffffffffu;
    uint32_t n = 0;
    Walk w(c.range, items);
    Segment s;
    while (w.next(a, s)) {
        if (!looked_at(a, s)) continue;
        if (!__all_sync(kAll, c.wait(L::seen + 8 * (n & 1), (n >> 1 & 1) ^ 1))) return;
        const bool odd = odd_values<D, kBf16V>(a, s, lane);
        if (lane == 0) {
            reinterpret_cast<volatile uint32_t*>(c.smem + L::odd)[n & 1] = odd;
            if (odd) reinterpret_cast<volatile uint32_t*>(c.smem + L::odd)[2] = 1;
            mbar_arrive(c.base + L::checked + 8 * (n & 1));
        }
        __syncwarp();
        ++n;
    }
}

// ------------------------------------------------------------ MMA

// Run by the whole warp: control flow and descriptors are the same in every
// lane (broadcasts tell the compiler so: operands then stay in uniform
// registers; issued by one diverged lane, eight MMAs took some 1,300 cycles),
// and one elected lane issues. A step of a stream is the product of its weights
// with V_j and the product of the next keys with its queries. Its barriers are
// polled together, one per lane: a wait costs some 200 cycles even when it is
// over, and the MMA queue holds only a few instructions.
template <int D, bool kBf16, bool kBf16V>
__device__ __forceinline__ void issue_mma(const Ctx& c, const AttnArgs& a, uint32_t tmem_base, int items) {
    using L = Smem<D>;
    constexpr unsigned kAll = 0xffffffffu;
    constexpr uint32_t kIdQk = idesc_f16_f32(kRows, kKeys, kBf16, false);
    constexpr uint32_t kIdPv = idesc_f16_f32(kRows, D, kBf16V, true);
    constexpr int P = L::kParts, kPer = L::kSlotKeys;
    // lane 0: weights; 1 .. P: V slots; P + 1 .. 2 P: K slots; then the accumulator
    constexpr unsigned kNeedV = ((1u << P) - 1) << 1, kNeedK = kNeedV << P, kNeedO = 1u << (2 * P + 1);
    const int lane = threadIdx.x & 31;
    const uint32_t tmem = __shfl_sync(kAll, tmem_base, 0);
    const uint32_t base = __shfl_sync(kAll, c.base, 0);
    uint32_t nq = 0;                 // segments with keys so far
    uint32_t np0 = 0, np1 = 0;       // weight tiles consumed of each stream
    uint32_t no0 = 0, no1 = 0;       // segments that used each accumulator
    bool ok = true, any = false;

    // Polls this lane's barrier until all lanes of `need` have theirs; the
    // lanes that do, then.
    auto poll = [&](uint32_t bar, uint32_t parity, unsigned need) -> unsigned {
        for (int64_t it = 0; ok; ++it) {
            const unsigned got = __ballot_sync(kAll, mbar_test_wait(base + bar, parity & 1));
            if ((got & need) == need) return got;
            if (__any_sync(kAll, *c.abort_flag != 0) || it > 16 * c.spin) ok = false;   // (16 polls to a suspended wait)
        }
        if (lane == 0) {
            *c.abort_flag = 1;
            atomicCAS(c.status, 0, static_cast<int32_t>(SP_ERR_TIMEOUT));
        }
        return 0;
    };
    // a place in the ring: slot and turn
    struct Place {
        int slot;
        uint32_t turn;
    };
    auto ahead = [&](Place p, int n) -> Place {
        p.slot += n;
        if (p.slot >= L::kSlots) {
            p.slot -= L::kSlots;
            p.turn ^= 1;
        }
        return p;
    };
    // logits of query tile t and the K tile at p into stream buffer sb
    auto qk = [&](Place p, int t, int sb, bool release) {
        any = true;
#pragma unroll(P == 1 ? 2 : 1)
        for (int part = 0; part < P; ++part) {
            const int slot = __shfl_sync(kAll, ahead(p, part).slot, 0);
            const uint64_t qd = smem_desc_sw128(base + L::q + t * L::kChunks * kChunk + part * L::kSlot);
            const uint64_t kd = smem_desc_sw128_k(base + L::ring + slot * L::kSlot, 1024 * L::kSlotChunks);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4 * L::kSlotChunks; ++k)
                    tc_mma_bf16(tmem + sb * kKeys, qd + (k / 4) * (kChunk / 16) + 2 * (k % 4),
                                kd + (k / 4) * 64 + 2 * (k % 4), kIdQk, (part | k) != 0);
                if (release) tc_commit(base + L::empty + 8 * slot);
                if (part == P - 1) tc_commit(base + L::sfull + 8 * sb);
            }
        }
    };
    // accumulator o (+)= weights of stream sb times the V tile at p
    auto pv = [&](Place p, int sb, int o, bool first, bool release) {
#pragma unroll(P == 1 ? 2 : 1)
        for (int part = 0; part < P; ++part) {
            const int slot = __shfl_sync(kAll, ahead(p, part).slot, 0);
            const uint64_t vd = smem_desc_sw128_mn(base + L::ring + slot * L::kSlot, 1024, 1024 * L::kChunks);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kPer / 16; ++k)
                    tc_mma_f16_ts(tmem + 2 * kKeys + o * D, tmem + sb * kKeys + (part * (kPer / 16) + k) * 8,
                                  vd + 128 * L::kChunks * k, kIdPv, !first || (part | k) != 0);
                if (release) tc_commit(base + L::empty + 8 * slot);
                if (part == P - 1) tc_commit(base + L::odone + 8 * sb);
            }
        }
    };
    // The next step of stream sb on query tile t: V at v, and K behind it when
    // `more`. `fresh`: nobody has waited for their slots yet.
    auto step = [&](Place v, int t, int sb, int o, bool first, bool more, bool fresh, bool release) {
        const Place k = ahead(v, P);
        const Place mine = lane <= P ? ahead(v, lane - 1 < 0 ? 0 : lane - 1) : ahead(k, (lane - 1) % P);
        uint32_t bar = L::pfull + 8 * sb, parity = sb ? np1 : np0;
        if (lane >= 1 && lane <= 2 * P) {
            bar = L::full + 8 * mine.slot;
            parity = mine.turn;
        } else if (lane == 2 * P + 1) {
            bar = L::oempty + 8 * o;
            parity = (o ? no1 : no0) ^ 1;
        }
        const unsigned got = poll(bar, parity, 1u | (fresh ? kNeedV : 0u) | (first ? kNeedO : 0u));
        if (!ok) return;
        if (sb) ++np1; else ++np0;
        if (first) { if (o) ++no1; else ++no0; }
        tc_fence_after();
        pv(v, sb, o, first, release);
        if (more) {
            if (fresh && (got & kNeedK) != kNeedK) {
                poll(bar, parity, kNeedK);
                if (!ok) return;
            }
            qk(k, t, sb, release);
        }
    };
    auto keys_at = [&](Place p) {   // the K tile at p is there
        const Place mine = ahead(p, lane % P);
        poll(L::full + 8 * mine.slot, mine.turn, (1u << P) - 1);
        tc_fence_after();
        return ok;
    };
    auto queries_read = [&]() {
        if (elect_one()) tc_commit(base + L::qempty);
    };

    Walk w(c.range, items);
    Segment s;
    Place at{0, 0};
    while (ok && w.next(a, s)) {
        const int n = __shfl_sync(kAll, s.n, 0);
        if (n == 0) continue;
        const bool two = __shfl_sync(kAll, static_cast<int>(two_tiles(a, s, D)), 0) != 0;
        poll(L::qfull, nq, 1);
        if (!ok) break;
        ++nq;
        // first logits: both query tiles with K0, or K0 and K1
        for (int i = 0; i < (two || n > 1 ? 2 : 1); ++i) {
            if ((i == 0 || !two) && !keys_at(at)) break;
            qk(at, two ? i : 0, i, !two || i == 1);
            if (!two || i == 1) at = ahead(at, P);
        }
        if (n <= (two ? 1 : 2)) queries_read();
        if (two) {
            // ring: V0 K1 V1 K2 ..., each tile for both streams in turn
            for (int j = 0; j < n && ok; ++j) {
                step(at, 0, 0, 0, j == 0, j + 1 < n, true, false);
                if (!ok) break;
                step(at, 1, 1, 1, j == 0, j + 1 < n, false, true);
                if (j + 2 == n) queries_read();
                at = ahead(ahead(at, P), j + 1 < n ? P : 0);
            }
        } else {
            // ring: V0 K2 V1 K3 ..., for one stream each
            for (int j = 0; j < n && ok; ++j) {
                const int sb = j & 1;
                step(at, 0, sb, D <= 128 ? sb : 0, D <= 128 ? j < 2 : j == 0, j + 2 < n, true, true);
                if (j + 3 == n) queries_read();
                at = ahead(ahead(at, P), j + 2 < n ? P : 0);
            }
        }
    }
    if (any) {
        if (elect_one()) tc_commit(base + L::drain);
        __syncwarp();
        mbar_wait_spin(base + L::drain, 0, kDrainSpin);
    }
}

// ------------------------------------------------------------ softmax

template <bool kBf16>
__device__ __forceinline__ uint32_t pack_pair(float x, float y) {
    if constexpr (kBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// One 32-byte sector from one thread.
__device__ __forceinline__ void store_32b(void* p, const uint32_t* x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}

__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

// How a warp's rows of an item end: this lane's row (its place, factors of the
// accumulators, reference and sum), and what all lanes share.
struct RowEnd {
    int64_t t;
    int h, part;       // part < 0: the whole item is here
    uint32_t ot;       // accumulator of the warp's rows
    int rows, col0;    // rows in use from the warp's first, first column
    float f0, f1, m, l;
    bool join;
};

// Writes the rows of a warp, one per lane: results, or (kSplit) a part for the join
// kernel. Not inlined: the softmax loop keeps its registers. (Whole lines after
// an exchange between quads took 1.4 times as long: the shuffles cost more
// than the 32 lines of a store. One code for both, with the choice at run time: one token
// over 512 9.2 us in place of 9.0.)
template <int D, bool kBf16, bool kOver, bool kSplit>
__device__ __noinline__ void write_rows(const AttnArgs& a, RowEnd e) {
    constexpr int kCols = D > 128 ? D / 2 : D;    // columns of a warpgroup
    const bool mine = static_cast<int>(threadIdx.x & 31) < e.rows;
    const bool none = e.l == 0.0f && !kSplit;
    // (the approximate reciprocal and, for lse, logarithm are off by 2^-22: with
    // the exact ones out is the same to four digits of its error, lse is 0.5e-6 in
    // place of 0.7e-6 off at 8.5, where a step of 32 bits is 1e-6, and a prompt at
    // d = 256 and the mixed batch take 1 % longer)
    const float inv = kSplit ? 1.0f : none ? 0.0f : kOver ? __fdividef(1.0f, e.l) * a.out_scale : __fdividef(1.0f, e.l);
    const float e0 = e.f0 * inv, e1 = e.f1 * inv;
    char* dst = kSplit ? reinterpret_cast<char*>(a.part_o + static_cast<int64_t>(e.part) * D + e.col0)
                      : reinterpret_cast<char*>(a.out + e.t * a.o_st + e.h * a.o_sh + e.col0);
    if (mine && e.col0 == 0) {
        if constexpr (kSplit) a.part_ml[e.part] = make_float2(e.m, e.l);
        else if (a.lse) a.lse[e.t * a.G * a.hk + e.h] = none ? -INFINITY : (e.m - weight_bias(bf16_values(kBf16, kOver)) + __log2f(e.l)) * kLn2;
    }
#pragma unroll 1
    for (int q = 0; q < kCols / 32; ++q) {
        float x[32];
        tmem_ld_32x32b_x32(e.ot + 32 * q, x);
        if (e.join) {
            float y[32];
            tmem_ld_32x32b_x32(e.ot + D + 32 * q, y);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = x[i] * e0 + y[i] * e1;
        } else {
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] *= e0;
        }
        if (!mine) continue;
        if constexpr (kSplit) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                store_32b(dst + q * 128 + i * 32, reinterpret_cast<const uint32_t*>(x + 8 * i));
        } else {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = none ? 0u : pack_pair<kBf16>(x[2 * i], x[2 * i + 1]);
            if (a.wide_out) {
                store_32b(dst + q * 64, w);
                store_32b(dst + q * 64 + 32, w + 8);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<uint4*>(dst + q * 64)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
        }
    }
}

// Rows [row0, min(row0 + 32, rows)) of query tile `tok0` tokens into the item,
// over the segment's keys.
struct RowsAgain {
    Item it;
    int g, first, n, tok0, row0, rows, part;   // part < 0: the whole item is here
};

template <bool kBf16, int E>
__device__ __forceinline__ void load_elements(const uint16_t* p, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if constexpr (kBf16) x[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
        else x[i] = __half2float(__ushort_as_half(p[i]));
    }
}

// The same rows without the tensor cores, by one warp, a row at a time with
// the head dimension over its lanes: for segments in which a row is masked from
// a value that is infinite or NaN (its zero weight would make the product NaN).
// Slow, and right for any input.
template <int D, bool kBf16, bool kOver>
__device__ __noinline__ void rows_again(const AttnArgs& a, const RowsAgain e) {
    constexpr int E = D / 32;
    constexpr float kBias = weight_bias(bf16_values(kBf16, kOver));
    const int lane = threadIdx.x & 31;
    for (int r = e.row0; r < min(e.rows, e.row0 + 32); ++r) {
        const int tok = r / a.G, h = e.g * a.G + r - tok * a.G;
        const int64_t t = e.it.tok0 + e.tok0 + tok;
        const int pos = e.it.pos0 + e.tok0 + tok;
        int hi = min(a.causal ? min(e.it.khi, pos + 1) : e.it.khi, (e.first + e.n) * kKeys);
        int lo = max(a.window > 0 ? max(pos - a.window + 1, 0) : 0, e.first * kKeys);
        float q[E], acc[E];
        load_elements<kBf16>(a.q + t * a.q_st + h * a.q_sh + lane * E, q);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0.0f;
        float m = -INFINITY, l = 0.0f;
        for (int j = lo; j < hi; ++j) {
            const int blk = j / a.bs;
            const int id = a.table[static_cast<int64_t>(e.it.b) * a.table_stride + blk];
            int64_t row = static_cast<int64_t>(id) * a.bs;
            row = id < 0 || row + a.bs > a.pool_tokens ? 0 : row + j - blk * a.bs;
            float x[E], y = 0.0f;
            load_elements<kBf16>(a.k + row * a.k_st + e.g * a.k_sh + lane * E, x);
#pragma unroll
            for (int i = 0; i < E; ++i) y += q[i] * x[i];
#pragma unroll
            for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
            y *= a.scale2;
            const float mn = fmaxf(m, y), base = mn == -INFINITY ? 0.0f : mn;
            const float f = mn == m ? 1.0f : exp2_ftz(m - mn), p = exp2_ftz(y - base + kBias);
            l = l * f + p;
            load_elements<bf16_values(kBf16, kOver)>(a.v + row * a.v_st + e.g * a.v_sh + lane * E, x);
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = acc[i] * f + p * x[i];
            m = mn;
        }
        if (e.part >= 0) {
            float* o = a.part_o + static_cast<int64_t>(e.part + r) * D + lane * E;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = acc[i];
            if (lane == 0) a.part_ml[e.part + r] = make_float2(m, l);
        } else {
            const bool none = l == 0.0f;
            uint16_t* o = a.out + t * a.o_st + h * a.o_sh + lane * E;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const uint32_t w = none ? 0u : pack_pair<kBf16>(kOver ? acc[i] / l * a.out_scale : acc[i] / l, 0.0f);
                o[i] = static_cast<uint16_t>(w & 0xffffu);
            }
            if (a.lse && lane == 0) a.lse[t * a.G * a.hk + h] = none ? -INFINITY : (m - kBias + __log2f(l)) * kLn2;
        }
    }
}

// The rows of the flagged segments, when nothing of the CTA waits any more: their
// time grows with the context (0.1 s and more at 40,000 keys), beyond what a
// bounded wait may last. The segments are found by looking at their values once
// more (as many flags as a range has segments have no place to stay).
template <int D, bool kBf16, bool kOver>
__device__ __noinline__ void flagged_rows(const AttnArgs& a, const Range* range, int items, int wg) {
    const int warp = threadIdx.x >> 5 & 3, lane = threadIdx.x & 31;
    Walk w(range, items);
    Segment s;
    while (w.next(a, s)) {
        const bool two = two_tiles(a, s, D);
        const int tile = two ? wg : 0;
        const int rows = min(max(s.it.ntok - tile * a.tq, 0), a.tq) * a.G;
        if (wg == 1 && !two) continue;   // (the first warpgroup's rows)
        if (warp * 32 >= rows || !looked_at(a, s) || !odd_values<D, bf16_values(kBf16, kOver)>(a, s, lane)) continue;
        RowsAgain e;
        e.it = s.it;
        e.g = s.g;
        e.first = s.first;
        e.n = s.n;
        e.tok0 = tile * a.tq;
        e.row0 = warp * 32;
        e.rows = rows;
        e.part = s.split ? ((static_cast<int>(blockIdx.x) * 2 + (s.head ? 0 : 1)) * Smem<D>::kTiles + tile) * kRows : -1;
        rows_again<D, kBf16, kOver>(a, e);
    }
}

// One warpgroup (index wg) of softmax threads over the CTA's segments.
template <int D, bool kBf16, bool kOver>
__device__ __forceinline__ void softmax_rows(const Ctx& c, const AttnArgs& a, uint32_t tmem, int items, int wg) {
    using L = Smem<D>;
    constexpr unsigned kAll = 0xffffffffu;
    constexpr float kBias = weight_bias(bf16_values(kBf16, kOver));
    const int warp = threadIdx.x >> 5 & 3, lane = threadIdx.x & 31;
    const int row = warp * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const int tid = threadIdx.x & 127;
    uint32_t cnt0 = 0, cnt1 = 0; // tiles of each stream buffer before this segment
    uint32_t alt = 0;            // segments joined from two accumulators so far
    int ring = 0;                // slot of the segment's first K tile
    uint32_t turn = 0;           // and its turn
    bool ok = true;
    uint32_t checks = 0;         // segments whose values are looked at so far
    Walk w(c.range, items);
    Segment s;
    while (w.next(a, s)) {
        const bool two = two_tiles(a, s, D);
        const int tile = two ? wg : 0;                 // query tile of this warpgroup
        const int ntok = min(max(s.it.ntok - tile * a.tq, 0), a.tq);
        const int rows = ntok * a.G;
        const bool live = warp * 32 < rows;            // (warp-uniform)
        const int tok = row / a.G;                     // token of the tile
        const bool valid = row < rows;
        const int pos = s.it.pos0 + tile * a.tq + tok;
        // (unused rows of the tile compute on: masked, they would send every
        // tile of their warp through the masking)
        const int hi = a.causal && valid ? min(s.it.khi, pos + 1) : s.it.khi;
        const int lo = a.window > 0 && valid ? max(pos - a.window + 1, 0) : 0;
        // tiles of this warpgroup: all with two query tiles or d = 256 (first
        // warpgroup only), every second one otherwise
        const bool whole = two || D > 128;
        const int j0 = two ? 0 : wg, dj = whole ? 1 : 2;
        const bool works = s.n > 0 && !(D > 128 && wg == 1);
        float m = -INFINITY, l = 0.0f;
        // waits until the weights of tile j are in the accumulator. (Every
        // stream buffer has a barrier of its own, also where both feed one
        // accumulator: once the logits of a tile are there, all updates but
        // the last of each buffer have ended, so one parity tells.)
        auto updated = [&](int j) {
            const int b = two ? wg : j & 1;
            return __all_sync(kAll, c.wait(L::odone + 8 * b, ((b ? cnt1 : cnt0) + (two ? j : j >> 1)) & 1)) != 0;
        };
        if (works) {
            for (int j = j0; j < s.n; j += dj) {
                const int sb = two ? wg : j & 1;
                const uint32_t k = two ? j : j >> 1;
                const uint32_t seen = (sb ? cnt1 : cnt0) + k;     // tiles of this buffer before this one
                if (ok) ok = __all_sync(kAll, c.wait(L::sfull + 8 * sb, seen & 1));
                if (!ok) break;
                tc_fence_after();
                const int key0 = (s.first + j) * kKeys;
                if (live) {
                    float v[4][32];
                    const uint32_t st = tmem + lanes + sb * kKeys;
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(st + 32 * q, v[q]);
                    tmem_ld_wait();
                    const int h = hi - key0, b = lo - key0;
                    if (__any_sync(kAll, h < kKeys || b > 0)) {
                        // 32 columns at a time: most are seen by all rows of the
                        // warp or by none
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int hq = min(max(h - q * 32, 0), 32), bq = min(max(b - q * 32, 0), 32);
                            if (!__any_sync(kAll, hq < 32 || bq > 0)) continue;
                            const uint32_t seen_cols = static_cast<uint32_t>((1ull << hq) - (1ull << min(bq, hq)));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(seen_cols & (1u << i))) v[q][i] = -INFINITY;
                        }
                    }
                    float mx[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        mx[q] = fmaxf(v[q][0], v[q][1]);
#pragma unroll
                        for (int i = 2; i < 32; i += 2) mx[q] = max3(mx[q], v[q][i], v[q][i + 1]);
                    }
                    const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * a.scale2;
                    const bool move = mt > m + kSlack;
                    if (__any_sync(kAll, move)) {
                        const float mn = move ? mt : m;
                        const float f = mn == m ? 1.0f : exp2_ftz(m - mn);
                        l *= f;
                        m = mn;
                        // the accumulator holds earlier tiles of this segment
                        if (j > j0) {
                            const int o = D > 128 ? 0 : sb;
                            ok = updated(j - dj);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t ot = tmem + lanes + 2 * kKeys + o * D;
#pragma unroll 1
                            for (int q = 0; q < D / 32; ++q) {
                                float x[32];
                                tmem_ld_32x32b_x32(ot + 32 * q, x);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 32; ++i) x[i] *= f;
                                tmem_st_32x32b_x32(ot + 32 * q, x);
                            }
                        }
                    }
                    // The weights are rounded to 16 bits, the type of the tensor
                    // cores' operands (half a step each, not their sum, which stays
                    // as it is): beside the rounding of the result, which any form
                    // has, that takes the relative error over long contexts from
                    // 0.0017 to 0.0023 (bf16). Their exponentials are off by 2^-22
                    // at most, results below 2^-126 are 0.
                    const float shift = (m == -INFINITY ? 0.0f : -m) + kBias;
                    const float2 scale = make_float2(a.scale2, a.scale2), move2 = make_float2(shift, shift);
                    float2 sum[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 x = fma2(make_float2(v[q][2 * i], v[q][2 * i + 1]), scale, move2);
                            x.x = exp2_ftz(x.x);
                            x.y = exp2_ftz(x.y);
                            sum[i & 3] = (q == 0 && i < 4) ? x : add2(sum[i & 3], x);
                            pk[i] = pack_pair<bf16_values(kBf16, kOver)>(x.x, x.y);
                        }
                        tmem_st_32x32b_x16(st + 16 * q, pk);
                    }
                    sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                    l += sum[0].x + sum[0].y;
                    tmem_st_wait();
                }
                // V rows outside the item's keys are not loaded: zeros, so that
                // their zero weights meet no NaN (with two query tiles the first
                // warpgroup's zeros are in place before either product)
                const int z0 = max(s.it.klo - key0, 0), z1 = min(s.it.khi - key0, kKeys);
                if ((z0 > 0 || z1 < kKeys) && !(two && wg == 1)) {
                    const int place = ring + v_position(two, j, s.n) * L::kParts;
                    int p = place % L::kSlots;
                    uint32_t ph = turn ^ (place / L::kSlots & 1);
                    constexpr int kPer = L::kSlotKeys;
                    // d = 256: the slots of V_j are those of V_{j-1} and K_j, five
                    // slots back; V_{j-1} is consumed before they are looked at
                    if (D > 128 && j > 0) ok = updated(j - 1);
#pragma unroll 1
                    for (int part = 0; part < L::kParts && ok; ++part) {
                        ok = __all_sync(kAll, c.wait(L::full + 8 * p, ph));
                        if (!ok) break;
                        // vectors of this slot: [8 keys][chunk][key][8]
                        uint4* v = reinterpret_cast<uint4*>(c.smem + L::ring + p * L::kSlot);
                        for (int e = tid; e < static_cast<int>(L::kSlot / 16); e += 128) {
                            const int key = part * kPer + e / (64 * L::kChunks) * 8 + (e >> 3) % 8;
                            if (key < z0 || key >= z1) v[e] = make_uint4(0, 0, 0, 0);
                        }
                        if (++p == L::kSlots) {
                            p = 0;
                            ph ^= 1;
                        }
                    }
                    if (!ok) break;
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(c.base + L::pfull + 8 * sb);
            }
        }
        // ---- the item's end. With alternating key tiles of d <= 128 the first
        // warpgroup joins both accumulators; with d = 256 the second one writes
        // the upper half of the columns.
        const bool join = D <= 128 && !two && s.n > 1;
        const bool halves = D > 128 && s.n > 0;
        const uint32_t buf0 = two ? s.n : (s.n + 1) / 2, buf1 = two ? s.n : s.n / 2;
        float2* stat = reinterpret_cast<float2*>(c.smem + L::stat) + (alt & 1) * kRows;
        if ((join && wg == 1) || (halves && wg == 0)) {
            stat[row] = make_float2(m, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(c.base + L::statfull + 8 * (alt & 1));
        }
        cnt0 += buf0;
        cnt1 += buf1;
        bool again = false;
        if (looked_at(a, s)) {
            if (ok) ok = __all_sync(kAll, c.wait(L::checked + 8 * (checks & 1), checks >> 1 & 1));
            again = reinterpret_cast<volatile uint32_t*>(c.smem + L::odd)[checks & 1] != 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(c.base + L::seen + 8 * (checks & 1));
            ++checks;
        }
        if (two || wg == 0 || D > 128) {   // this warpgroup writes rows
            const int o = two ? wg : 0;
            float f0 = 1.0f, f1 = 0.0f;
            if ((join && wg == 0) || (halves && wg == 1)) {
                if (ok) ok = __all_sync(kAll, c.wait(L::statfull + 8 * (alt & 1), alt >> 1 & 1));
                if (ok) {
                    const float2 other = stat[row];
                    if (join) {
                        const float mn = fmaxf(m, other.x);
                        f0 = m == mn ? 1.0f : exp2_ftz(m - mn);
                        f1 = other.x == mn ? 1.0f : exp2_ftz(other.x - mn);
                        l = l * f0 + other.y * f1;
                        m = mn;
                    } else {
                        m = other.x;
                        l = other.y;
                    }
                }
            }
            if (s.n > 0) {
                const int b = D > 128 ? (s.n - 1) & 1 : o;   // buffer of the last update
                if (ok) ok = __all_sync(kAll, c.wait(L::odone + 8 * b, ((b ? cnt1 : cnt0) - 1) & 1));
                if (join && ok) ok = __all_sync(kAll, c.wait(L::odone + 8, (cnt1 - 1) & 1));
                tc_fence_after();
            }
            constexpr int kCols = D > 128 ? D / 2 : D;    // columns of this warpgroup
            const int col0 = D > 128 ? wg * kCols : 0;
            if (ok && live && !again) {
                RowEnd e;
                e.ot = tmem + lanes + 2 * kKeys + o * D + col0;
                e.rows = rows - warp * 32;
                e.t = s.it.tok0 + tile * a.tq + tok;
                e.h = s.g * a.G + row - tok * a.G;
                e.part = s.split ? ((static_cast<int>(blockIdx.x) * 2 + (s.head ? 0 : 1)) * L::kTiles + tile) * kRows + row : -1;
                e.col0 = col0;
                e.f0 = s.n > 0 ? f0 : 0.0f;
                e.f1 = f1;
                e.m = m;
                e.l = s.n > 0 ? l : 0.0f;
                e.join = join;
                if (s.split) write_rows<D, kBf16, kOver, true>(a, e);
                else write_rows<D, kBf16, kOver, false>(a, e);
            }
            if (s.n > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(c.base + L::oempty + 8 * o);
                    if (join) mbar_arrive(c.base + L::oempty + 8);
                }
            }
        }
        if (join || halves) ++alt;
        // the ring moves on by the segment's 2 n tiles
        ring += 2 * s.n * L::kParts % (2 * L::kSlots);
        while (ring >= L::kSlots) {
            ring -= L::kSlots;
            turn ^= 1;
        }
    }
    // (this warp has seen the flag of every segment that is looked at)
    if (ok && reinterpret_cast<volatile uint32_t*>(c.smem + L::odd)[2]) flagged_rows<D, kBf16, kOver>(a, c.range, items, wg);
}

// ------------------------------------------------------------ kernel

template <int D, bool kBf16, bool kOver>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnArgs a) {
    using L = Smem<D>;
    extern __shared__ __align__(1024) uint8_t attn_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Ctx c;
    c.smem = attn_smem;
    c.base = smem_u32(attn_smem);
    c.abort_flag = reinterpret_cast<volatile int*>(attn_smem + L::abort);
    c.status = a.status;
    c.spin = a.spin;
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kSlots; ++i) {
            mbar_init(c.base + L::full + 8 * i, 1);
            mbar_init(c.base + L::empty + 8 * i, 1);
        }
        mbar_init(c.base + L::qfull, 1);
        mbar_init(c.base + L::qempty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(c.base + L::sfull + 8 * i, 1);
            mbar_init(c.base + L::pfull + 8 * i, 4);
            mbar_init(c.base + L::odone + 8 * i, 1);
            mbar_init(c.base + L::oempty + 8 * i, D > 128 ? 8 : 4);
            mbar_init(c.base + L::statfull + 8 * i, 4);
            mbar_init(c.base + L::checked + 8 * i, 1);
            mbar_init(c.base + L::seen + 8 * i, 8);
        }
        mbar_init(c.base + L::drain, 1);
        *c.abort_flag = 0;
        reinterpret_cast<volatile uint32_t*>(attn_smem + L::odd)[2] = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(c.base + L::tmem, 512);
        tmem_relinquish();
    }
    if (warp == kQWarp && lane == 0) {
        prefetch_tmap(&mq);
        prefetch_tmap(&mk);
        prefetch_tmap(&mv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(attn_smem + L::tmem);
    grid_dep_wait();
    const bool aligned = (c.base & 1023u) == 0;   // the swizzle pattern starts at the slots
    if (!aligned && threadIdx.x == 0) {
        atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
        if (blockIdx.x == 0) a.head->tasks = 0;
    }
    int items = 0;
    Range* range = reinterpret_cast<Range*>(attn_smem + L::range);
    c.range = range;
    if (aligned) {
        if (a.local_plan) {
            // the ring is scratch until the first copy into it
            items = local_plan<kOver>(a, L::kTiles, *reinterpret_cast<LocalPlan*>(attn_smem + L::ring), range);
            fence_proxy_async_smem();
        } else {
            items = a.head->items;
            if (threadIdx.x == 0 && items > 0) {
                range->begin = a.starts[blockIdx.x];
                range->end = a.starts[blockIdx.x + 1];
            }
        }
        __syncthreads();
    }
    const bool work = items > 0;
    // 384 threads x 168 registers at launch = 64,512; 128 x 80 + 256 x 208 = 63,488
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (work) {
            if (warp == kLoadWarp) load_keys<D>(c, a, &mk, &mv, items, lane);
            else if (warp == kMmaWarp) issue_mma<D, kBf16, bf16_values(kBf16, kOver)>(c, a, tmem, items);
            else if (warp == kQWarp && lane == 0) load_queries<D>(c, a, &mq, items);
        }
        if (warp == kListWarp) {
            if (work) check_values<D, bf16_values(kBf16, kOver)>(c, a, items, lane);
            if (blockIdx.x == 0 && aligned) list_cuts(a, L::kChunks, lane);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        if (work) softmax_rows<D, kBf16, kOver>(c, a, tmem, items, warp >> 2);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------ join

// out = sum_p w_p O_p / sum_p w_p l_p, w_p = exp2(m_p - max m), for the rows of
// the cut items: 2 to 5 us for decode steps, two chained reads of L2 and the
// launch; some 10 us for a prompt at d = 256, whose 300 parts are 40 MB. A task is
// 64 columns of a row with many parts, which the 16 groups of a block share (the
// L2 latency of 76 parts in turn would be the kernel's time), or of 32 rows with
// few, two for each group.
template <int D, bool kBf16, bool kOver>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks) attn_join_kernel(const AttnArgs a) {
    using L = Smem<D>;
    constexpr float kBias = weight_bias(bf16_values(kBf16, kOver));
    __shared__ Job job_s[kMaxCtas];
    __shared__ float2 ml_s[kMaxCtas];
    __shared__ float4 acc_s[kJoinGroups][16];
    __shared__ float sum_s[kJoinGroups];
    grid_dep_wait();
    const PlanHead head = *a.head;
    const int group = threadIdx.x / 16, vec = threadIdx.x % 16, lane = threadIdx.x & 31;
    // (requested along with the head: the list holds at most one job per CTA)
    for (int i = threadIdx.x; i < a.grid; i += kJoinThreads) job_s[i] = a.jobs[i];
    if (static_cast<int>(blockIdx.x) >= head.tasks) return;
    __syncthreads();
    for (int task = blockIdx.x; task < head.tasks; task += gridDim.x) {
        int lo = 0, hi = head.jobs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (job_s[mid].task0 <= task) lo = mid; else hi = mid;
        }
        const Job job = job_s[lo];
        const int parts = job.parts;
        const int rows0 = min(job.ntok, a.tq) * a.G, rows = job.ntok * a.G;   // of the first tile, of both
        const bool share = join_shares(parts, rows * L::kChunks);
        // 64 columns of a row, this thread's four of them
        struct Place {
            int tile, row, col;
        };
        auto place = [&](int unit) {
            const int r = unit / L::kChunks, tile = r >= rows0 ? 1 : 0;
            return Place{tile, r - tile * rows0, unit % L::kChunks * 64 + vec * 4};
        };
        auto at = [&](Place x, int p) {
            const int part = (job.c0 + p) * 2 + (p == 0 && !job.c0_head ? 1 : 0);
            return (static_cast<int64_t>(part) * L::kTiles + x.tile) * kRows + x.row;
        };
        auto load = [&](Place x, int p) { return __ldcg(reinterpret_cast<const float4*>(a.part_o + at(x, p) * D + x.col)); };
        struct Row {
            float top, sum;
            float4 acc;
            __device__ __forceinline__ void add(float2 ml, float4 x) {
                const float f = ml.x == top ? 1.0f : exp2_ftz(ml.x - top);
                sum += ml.y * f;
                acc.x += x.x * f;
                acc.y += x.y * f;
                acc.z += x.z * f;
                acc.w += x.w * f;
            }
        };
        const Row zero{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
        auto write = [&](Place x, const Row& y) {
            const bool none = y.sum == 0.0f;
            const float inv = none ? 0.0f : kOver ? 1.0f / y.sum * a.out_scale : 1.0f / y.sum;
            const int tok = x.row / a.G;
            const int64_t t = job.tok0 + x.tile * a.tq + tok;
            const int h = job.g * a.G + x.row - tok * a.G;
            uint2 w;
            w.x = none ? 0u : pack_pair<kBf16>(y.acc.x * inv, y.acc.y * inv);
            w.y = none ? 0u : pack_pair<kBf16>(y.acc.z * inv, y.acc.w * inv);
            *reinterpret_cast<uint2*>(a.out + t * a.o_st + h * a.o_sh + x.col) = w;
            if (a.lse && x.col == 0) a.lse[t * a.G * a.hk + h] = none ? -INFINITY : (y.top - kBias + __log2f(y.sum)) * kLn2;
        };
        if (share) {
            const Place x = place(task - job.task0);
            Row y = zero;
            for (int p = threadIdx.x; p < parts; p += kJoinThreads) ml_s[p] = __ldcg(a.part_ml + at(x, p));
            __syncthreads();
            for (int p = lane; p < parts; p += 32) y.top = fmaxf(y.top, ml_s[p].x);
#pragma unroll
            for (int o = 16; o; o >>= 1) y.top = fmaxf(y.top, __shfl_xor_sync(0xffffffffu, y.top, o));
#pragma unroll 4
            for (int p = group; p < parts; p += kJoinGroups) y.add(ml_s[p], load(x, p));
            acc_s[group][vec] = y.acc;
            if (vec == 0) sum_s[group] = y.sum;
            __syncthreads();
            if (group == 0) {
#pragma unroll
                for (int k = 1; k < kJoinGroups; ++k) {
                    const float4 o = acc_s[k][vec];
                    y.acc.x += o.x;
                    y.acc.y += o.y;
                    y.acc.z += o.z;
                    y.acc.w += o.w;
                    y.sum += sum_s[k];
                }
                write(x, y);
            }
            __syncthreads();   // (the shared arrays are free for the next task)
            continue;
        }
        const int first = (task - job.task0) * (kJoinGroups * kJoinRows) + group, units = rows * L::kChunks;
        if (parts == 2) {
            Place x[kJoinRows];
            float2 ml[kJoinRows][2];
            float4 o[kJoinRows][2];
#pragma unroll
            for (int k = 0; k < kJoinRows; ++k) {
                x[k] = place(min(first + k * kJoinGroups, units - 1));
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    ml[k][p] = __ldcg(a.part_ml + at(x[k], p));
                    o[k][p] = load(x[k], p);
                }
            }
#pragma unroll
            for (int k = 0; k < kJoinRows; ++k) {
                Row y = zero;
                y.top = fmaxf(ml[k][0].x, ml[k][1].x);
                y.add(ml[k][0], o[k][0]);
                y.add(ml[k][1], o[k][1]);
                if (first + k * kJoinGroups < units) write(x[k], y);
            }
            continue;
        }
#pragma unroll 1
        for (int unit = first; unit < min(units, first + kJoinGroups * kJoinRows); unit += kJoinGroups) {
            const Place x = place(unit);
            Row y = zero;
            if (parts <= kJoinFew) {
                float2 ml[kJoinFew];
                float4 o[kJoinFew];
#pragma unroll
                for (int p = 0; p < kJoinFew; ++p)
                    if (p < parts) {
                        ml[p] = __ldcg(a.part_ml + at(x, p));
                        o[p] = load(x, p);
                    }
#pragma unroll
                for (int p = 0; p < kJoinFew; ++p)
                    if (p < parts) y.top = fmaxf(y.top, ml[p].x);
#pragma unroll
                for (int p = 0; p < kJoinFew; ++p)
                    if (p < parts) y.add(ml[p], o[p]);
            } else {
#pragma unroll 8
                for (int p = 0; p < parts; ++p) y.top = fmaxf(y.top, __ldcg(a.part_ml + at(x, p)).x);
#pragma unroll 8
                for (int p = 0; p < parts; ++p) y.add(__ldcg(a.part_ml + at(x, p)), load(x, p));
            }
            write(x, y);
        }
    }
}

// ------------------------------------------------------------ host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &qr) !=
                cudaSuccess ||
            qr != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// Map of rows of 64-element chunks, swizzled: dims (d, n1, n2) with element
// strides s1 and s2, box (64, b1, b2). The stride of an axis of one entry
// counts for nothing and is replaced.
bool make_map(CUtensorMap* m, bool bf16, const void* p, int d, int64_t n1, int64_t s1, int64_t n2, int64_t s2,
              int b1, int b2) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(n1 > 1 ? s1 : d) * 2, static_cast<cuuint64_t>(n2 > 1 ? s2 : d) * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p),
               dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of a pool for boxes of `rows` rows x `chunks` 64-element chunks of one
// head: dims (64, 8 rows, chunk, group of 8 rows, head). A box lands as
// [8-row group][chunk][8][64], the swizzle atoms of both products' operands at
// fixed strides whatever the box's rows, so one copy brings a whole block.
bool make_pool_map(CUtensorMap* m, bool bf16, const void* p, int d, int64_t pool_rows, int64_t row_stride, int heads,
                   int64_t head_stride, int rows, int chunks) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(d / 64), static_cast<cuuint64_t>(pool_rows / 8),
                          static_cast<cuuint64_t>(heads)};
    cuuint64_t strides[4] = {static_cast<cuuint64_t>(row_stride) * 2, 128, static_cast<cuuint64_t>(row_stride) * 16,
                             static_cast<cuuint64_t>(heads > 1 ? head_stride : d) * 2};
    cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(chunks), static_cast<cuuint32_t>(rows / 8), 1};
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<void*>(p),
               dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout {
    int64_t items_max;
    size_t head, items, pre, req, starts, jobs, ml, o, total;
};

Layout layout(const sp_paged_shape* s, int grid) {
    Layout l;
    const int tiles = tiles_per_item(s->head_dim), tq = kRows / (s->n_q_heads / s->n_kv_heads);
    l.items_max = s->n_tokens / (tq * tiles) + s->n_seqs;
    size_t off = sizeof(WsHeader);
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = (off + bytes + 255) & ~size_t(255);
        return o;
    };
    l.head = take(sizeof(PlanHead));
    l.items = take(sizeof(Item) * l.items_max);
    l.pre = take(8 * (l.items_max + 1));
    l.req = take(4 * (static_cast<size_t>(s->n_seqs) + 1));
    l.starts = take(sizeof(Start) * (static_cast<size_t>(grid) + 1));
    l.jobs = take(sizeof(Job) * grid);
    l.ml = take(8 * static_cast<size_t>(grid) * 2 * tiles * kRows);
    l.o = take(4 * static_cast<size_t>(grid) * 2 * tiles * kRows * s->head_dim);
    l.total = off;
    return l;
}

template <int D, bool kOver>
cudaError_t launch_d(const AttnArgs& a, bool bf16, const CUtensorMap& mq, const CUtensorMap& mk,
                     const CUtensorMap& mv, cudaStream_t st) {
    auto kern = bf16 ? attn_kernel<D, true, kOver> : attn_kernel<D, false, kOver>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(Smem<D>::total));
    if (e != cudaSuccess) return e;
    const cudaError_t r = launch_k(kern, static_cast<unsigned>(a.grid), kAttnThreads, Smem<D>::total, st, mq, mk, mv, a);
    if (r != cudaSuccess) return r;
    return launch_k(bf16 ? attn_join_kernel<D, true, kOver> : attn_join_kernel<D, false, kOver>,
                    static_cast<unsigned>(kJoinBlocks * a.grid), kJoinThreads, 0, st, a);
}

template <bool kOver>
cudaError_t launch_all(const AttnArgs& a, int d, bool bf16, const CUtensorMap& mq, const CUtensorMap& mk,
                       const CUtensorMap& mv, cudaStream_t st) {
    if (!a.local_plan) {
        const cudaError_t e = launch_k(attn_plan_kernel<kOver>, 1, kPlanThreads, 0, st, a, tiles_per_item(d));
        if (e != cudaSuccess) return e;
    }
    return d == 64    ? launch_d<64, kOver>(a, bf16, mq, mk, mv, st)
           : d == 128 ? launch_d<128, kOver>(a, bf16, mq, mk, mv, st)
                      : launch_d<256, kOver>(a, bf16, mq, mk, mv, st);
}

}  // namespace

// One CTA per SM (its shared memory fills one).
int attn_grid() {
    const int sms = device_sms();
    return sms < kMaxCtas ? sms : kMaxCtas;
}

size_t attn_workspace(const sp_paged_shape* s) { return layout(s, attn_grid()).total; }

cudaError_t launch_paged_attention(const sp_paged_shape* s, const sp_attn_params* p, const int32_t* q_off,
                                   const int32_t* kv_len, const int32_t* table, const uint16_t* q,
                                   const uint16_t* k_pool, const uint16_t* v_pool, uint16_t* out, float* lse,
                                   void* ws, cudaStream_t st, const AttnMore* more) {
    const int d = s->head_dim, bs = s->block_size;
    const bool bf16 = s->dtype == SP_DTYPE_BF16;
    AttnArgs a;
    a.grid = attn_grid();
    const Layout l = layout(s, a.grid);
    a.q_off = q_off;
    a.kv_len = kv_len;
    a.table = table;
    a.q = q;
    a.k = k_pool;
    a.v = v_pool;
    a.out = out;
    a.lse = lse;
    a.status = more ? more->status : &ws_ptr<WsHeader>(ws, 0)->status;
    a.only = more ? more->only : nullptr;
    a.out_scale = more ? more->out_scale : 1.0f;
    a.head = ws_ptr<PlanHead>(ws, l.head);
    a.items = ws_ptr<Item>(ws, l.items);
    a.pre = ws_ptr<int64_t>(ws, l.pre);
    a.req_item = ws_ptr<int32_t>(ws, l.req);
    a.starts = ws_ptr<Start>(ws, l.starts);
    a.jobs = ws_ptr<Job>(ws, l.jobs);
    a.part_o = ws_ptr<float>(ws, l.o);
    a.part_ml = ws_ptr<float2>(ws, l.ml);
    a.q_st = s->q_stride_token, a.q_sh = s->q_stride_head;
    a.k_st = s->k_stride_token, a.k_sh = s->k_stride_head;
    a.v_st = s->v_stride_token, a.v_sh = s->v_stride_head;
    a.o_st = s->o_stride_token, a.o_sh = s->o_stride_head;
    a.pool_tokens = s->pool_tokens;
    a.spin = p->spin_limit > 0 ? p->spin_limit : kDefaultSpin;
    a.B = s->n_seqs;
    a.hk = s->n_kv_heads;
    a.G = s->n_q_heads / s->n_kv_heads;
    a.tq = kRows / a.G;
    a.bs = bs;
    a.table_stride = s->table_stride;
    a.cap = s->n_tokens;
    a.item_cost = item_cost(d);
    a.causal = p->causal;
    a.window = p->window <= kMaxCached ? p->window : 0;   // (a longer one hides nothing)
    const int per = kKeys / slots_per_tile(d);
    const int hk = bs < kKeys ? bs : kKeys, hv = bs < per ? bs : per;
    a.hk_shift = __builtin_ctz(hk);
    a.hv_shift = __builtin_ctz(hv);
    a.q_bytes = static_cast<uint32_t>(a.G * a.tq) * 128u;
    const double scale = p->scale > 0.0f ? static_cast<double>(p->scale) : 1.0 / std::sqrt(static_cast<double>(d));
    a.scale2 = static_cast<float>(scale * 1.4426950408889634);
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, bf16, q, d, s->n_q_heads, s->q_stride_head, s->n_tokens, s->q_stride_token, a.G, a.tq) ||
        !make_pool_map(&mk, bf16, k_pool, d, s->pool_tokens, s->k_stride_token, a.hk, s->k_stride_head, hk,
                       d / 64 / slots_per_tile(d)) ||
        !make_pool_map(&mv, bf16_values(bf16, more != nullptr), v_pool, d, s->pool_tokens, s->v_stride_token, a.hk, s->v_stride_head, hv,
                       d / 64))
        return cudaErrorInvalidValue;
    // (a prompt of 4,916 tokens at d = 256: 102 us with 32-byte stores, 114 with 16)
    a.wide_out = (reinterpret_cast<uintptr_t>(out) & 31) == 0 && (s->n_tokens == 1 || a.o_st % 16 == 0) &&
                 (s->n_q_heads == 1 || a.o_sh % 16 == 0);
    // costs (times CTAs) of a plan in 32 bits
    const int64_t tiles = (static_cast<int64_t>(a.table_stride) * bs + kKeys - 1) / kKeys + a.item_cost;
    a.local_plan = l.items_max <= kLocalItems && a.B <= kLocalItems &&
                   tiles < INT32_MAX / kLocalItems / kMaxCtas / a.hk;
    return more ? launch_all<true>(a, d, bf16, mq, mk, mv, st) : launch_all<false>(a, d, bf16, mq, mk, mv, st);
}

}  // namespace sp
