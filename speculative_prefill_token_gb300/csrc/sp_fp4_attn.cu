// Attention of new tokens over a block-paged cache in 4 bits ("SpecPrefill —
// Implementation Guide", §How It Works / Sparse Prefill: the target's decode
// steps and short chunks over the kept tokens' cache).
//
// For a query row (token i of request b, head h) with visible cache indices
// [lo, hi), and KV head g = h / G,
//   out = v_scale sum_j exp2(y_j - m) v_j / sum_j exp2(y_j - m),
//   y_j = scale k_scale log2(e) <q, k_j>,
// where k_j and v_j are numbers times their group's scale, exact in fp16.
//
// The codes never exist as 16-bit values outside registers. A warp takes a tile
// of 64 keys alone: it converts the key codes into the left operand of an
// m16n8k16 product (16 keys x 16 elements; the right operand are 8 query rows),
// keeps the logits in registers, and converts the value codes into the left
// operand of the second product (16 elements x 16 keys), whose right operand
// are the transposed weights. The elements of a row are dealt to the lanes so
// that every lane's codes are consecutive bytes of one load: the sum over the
// elements, and the order of the result's elements, may be permuted freely.
// (Operands of tcgen05.mma lie in shared or tensor memory: 16-bit values written there
// and read again are 7 bytes for each byte of codes, 167 a cycle and SM where HBM delivers
// 23.5 of codes and shared memory moves 128. From registers, mma.sync needs 0.3 of its rate.)
//
// Work. The new tokens x the G heads of a KV head are rows; an item is up to
// 8 or 16 rows of a request and KV head, its unit a tile of 64 keys (32 at d = 256). All units
// of all items are cut into equal contiguous ranges, one for each CTA (one CTA an
// SM); tile i of the CTA goes to warp i mod W, which copies it into its own part
// of shared memory, keys and values in turn, while it works on what came before: no warp
// waits for another one inside an item. (One warp that loaded for all by bulk copies: some
// 120 cycles a copy, two to sixteen of them a tile: 174 us in place of 155 with blocks of 64
// tokens, 455 in place of 207 with blocks of 8.) At an item's end each warp leaves its share in shared memory and
// goes on; it takes its part of the join when all shares are there. Results of CTAs that share
// an item are joined by another kernel, in their order: results do not depend on timing.
//
// Requests with many rows are bound by the products, not by the cache: their keys
// and values are written once as 16-bit values into the workspace (exactly), and
// computed by the attention over a 16-bit cache (sp_attn.cu), on
// fifth-generation tensor cores, 128 rows at a time.
//
// Measured (bf16): 64 requests of 2K to 32K tokens, a token of each, 16/4 heads of 128, 728 MB: 125 to
// 127 us, 5.8 TB/s, 85 % of a copy's rate; its loads alone 116. Issue slots 56 % busy at 12 warps, ALU and fp16 pipes
// 47 and 38 %, tensor pipe 27 %, DRAM 69 %: no pipe is full, the rest is the chain convert - multiply
// - softmax of a warp, of which registers and shared memory hold no more than 12. The same bytes at
// d = 256 135 us, at d = 64, half of them, 96. A token of 16 requests of 4K to 16K, 8/2 heads of 256, 86 MB:
// 33 us, of which 5 are the start (lengths, ranges, table, first tile: reads that follow one
// another) and 3 the join. One token over 512: 8 us, all of it latency. 8 tokens over 32K, d =
// 256: 30.5 us, four items of 8 rows that convert the same codes (16 rows would take 128
// accumulators a lane, beside 64 registers of queries). 4,096 tokens over 39,322 in all: 0.83 to 0.86
// ms, of which the copy is 0.03.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sp_device.cuh"
#include "sp_fp4.cuh"
#include "sp_fp4.h"
#include "sp_internal.h"
#include "sp_paged.h"
#include "sp_ptx.cuh"

namespace sp {
namespace {

// Keys of a tile, the unit of work of a warp. (d = 128: 32 keys 167 us in place of 137; d = 256:
// 64 do not fit into a warp's registers.)
__host__ __device__ constexpr int tile_keys(int d) { return d <= 128 ? 64 : 32; }
constexpr int kItemCost = 16;                // of an item besides its tiles, in tiles (64 long decodes 127.8 us; 4: 134.2, 8: 129.7, 24: 128.7)
constexpr int kLocalSeqs = 1024;             // requests of a plan made by every CTA
constexpr int kPlanThreads = 1024;
constexpr int kMaxGrid = 256;
constexpr float kSlack = 8.0f;               // log2 units the reference may lag behind the maximum
constexpr float kBias = 6.0f;                // fp16 weights are scaled by 2^6: normal down to 2^-20 of the reference
constexpr float kLn2 = 0.6931471805599453f;
// Where a CTA's range starts: key tile `off` of item `gj` (KV head, row tile) of
// request b, an item that CTAs c0 .. c0 + parts - 1 work on. b = n_seqs: the end of
// everything.
struct alignas(16) Start {
    int32_t b, gj, off, c0, parts, pad[3];
};

struct Args {
    const int32_t* q_off;
    const int32_t* kv_len;
    const int32_t* table;
    const int32_t* dense;      // [B] or null: requests computed elsewhere (>= 0)
    const uint16_t* q;
    const uint8_t* k;
    const uint8_t* v;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int64_t* pre;              // units before each request [B + 1]; pre[B] < 0: nothing to do
    Start* starts;             // [grid + 1]
    float* part_o;             // [2 grid][rows][d]
    float2* part_ml;           // [2 grid][rows] (reference, sum)
    int64_t q_st, q_sh, o_st, o_sh, spin;
    uint32_t k_sb, k_sh, v_sb, v_sh, pool_blocks;   // (bytes)
    int B, hk, G, bs, table_stride, cap, max_new, causal, window, grid;
    int tile_shift;            // log2 of a tile's keys
    int piece_shift;           // log2 of a copy's tokens: a block's, at most a tile's
    int bs_shift;              // log2(bs), or -1
    int whole;                 // tiles of an item up to which it is not cut
    int cuts;                  // whether the table's rows hold longer ones (if not, there is no second join: one token
                               // over 512 by a row of 544 tokens 10.0 to 7.8 us, 64 over 900 by rows of 928, 2 heads of 64, 14.9 to 9.3)
    int local_plan, bf16;
    float scale2, v_scale;
};

template <typename T, typename U>
__device__ __forceinline__ int last_at_most(const T* v, int n, U x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// Exclusive sum over the block's NT threads, and the total.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    const int64_t mine = lane < NT / 32 ? sums[lane] : 0;
    int64_t all = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += x;
    }
    *total = __shfl_sync(0xffffffffu, all, 31);
    return __shfl_sync(0xffffffffu, all - mine, warp) + incl - v;
}

// Tiles that the keys below cache index n touch (n <= 2^30).
__device__ __forceinline__ int tiles_below(const Args& a, int n) {
    return (n + (1 << a.tile_shift) - 1) >> a.tile_shift;
}

// Key tiles that some row of a request sees, and its tiles of rows.
struct Span {
    int tile0, tiles, row_tiles;
};

__device__ __forceinline__ Span span_of(const Args& a, int nq, int kv, int rows) {
    Span s;
    const int lo = a.window > 0 ? max(0, kv - nq - a.window + 1) : 0;
    s.tile0 = lo >> a.tile_shift;
    s.tiles = kv > lo ? tiles_below(a, kv) - s.tile0 : 0;
    s.row_tiles = static_cast<int>((static_cast<int64_t>(nq) * a.G + rows - 1) / rows);
    return s;
}

// (of Args or DenseArgs, with its rows of q)
template <typename A>
__device__ __forceinline__ bool bad_request(const A& a, int tokens, int64_t lo, int64_t hi, int64_t kv) {
    return hi < lo || hi > tokens || hi - lo > a.max_new || kv < 0 || kv > kMaxCached ||
           kv > static_cast<int64_t>(a.table_stride) * a.bs;
}

// Units before each request, by the block's NT threads; the total, or -1 when a
// length is out of range.
template <int NT>
__device__ __forceinline__ int64_t plan_requests(const Args& a, int rows, int64_t* pre, int64_t* sums) {
    const int tid = threadIdx.x;
    int bad = tid == 0 ? a.q_off[0] != 0 : 0;
    int64_t units = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int b = b0 + tid;
        int64_t n = 0;
        if (b < a.B) {
            const int64_t lo = a.q_off[b], hi = a.q_off[b + 1], kv = a.kv_len[b];
            if (bad_request(a, a.cap, lo, hi, kv)) bad = 1;
            else if (!a.dense || a.dense[b] < 0) {
                const Span s = span_of(a, static_cast<int>(hi - lo), static_cast<int>(kv), rows);
                n = static_cast<int64_t>(a.hk) * s.row_tiles * (s.tiles + kItemCost);
            }
        }
        int64_t total;
        const int64_t at = units + block_scan<NT>(n, sums, &total);
        if (b < a.B) pre[b] = at;
        units += total;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
        units = -1;
    }
    return units;
}

// Lays out a batch of more than kLocalSeqs requests, by one block of its own.
__global__ void __launch_bounds__(kPlanThreads) fp4_plan_kernel(const Args a, int rows) {
    __shared__ int64_t sums[32];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t units = plan_requests<kPlanThreads>(a, rows, a.pre, sums);
    if (threadIdx.x == 0) a.pre[a.B] = units;
}

// CTAs that share `units`: few of them get less than a tile for every other warp. (4 tokens
// over 8K in 4 requests, d = 64: 14.3 us; 16 15.3, 32 17.9. One token over 512: 10.2 us; 2 and 4, where
// more CTAs shared it, 11.0 and 10.9.)
constexpr int kLeastUnits = 8;

__device__ __forceinline__ int64_t ctas_for(const Args& a, int64_t units) {
    return min(static_cast<int64_t>(a.grid), (units + kLeastUnits - 1) / kLeastUnits);
}

// The CTA whose range holds unit u of `units`. (T: int64_t, or uint32_t where units
// are below 2^24.)
template <typename T>
__device__ __forceinline__ int range_owner(T units, T ctas, T u) {
    return static_cast<int>(((u + 1) * ctas - 1) / units);
}

// Unit u of `units`, of request b whose units begin at `at`, as a start; a cut inside
// an item's fixed cost, or an item that has a tile for each warp at most, falls on the
// item's start: a warp's time there is that of one tile, and pieces of items cost their ends and
// the second join. (Cut as the others: a token of 16 requests of 900, 2 heads of 64, 14.9 us in
// place of 10.9; a prompt of 70, 4 heads of 128, 19.5 in place of 13.9.) Items of two tiles a warp are not cut
// either where there are 64 or more of them and no CTA gets two while most get one: a token of
// 16, 32 and 64 requests of 900, 4 heads of 128, 17.3, 19.9 and 26.0 us cut, 14.0, 14.1 and 21.5 whole; of 8 16.4
// and 13.9, but of 4 12.0 and 13.7; of 40 requests of 1,400 19.7 and 24.0.
template <typename T>
__device__ __forceinline__ Start make_start(const Args& a, int b, int nq, int kv, T at, T units, T ctas, T u, int rows) {
    Start s{b, 0, 0, 0, 1, {0, 0, 0}};
    const Span sp = span_of(a, nq, kv, rows);
    const T per = sp.tiles + kItemCost;
    s.gj = static_cast<int32_t>((u - at) / per);
    const T item = at + s.gj * per;
    s.off = sp.tiles > a.whole ? max(static_cast<int32_t>(u - item) - kItemCost, 0) : 0;
    s.c0 = range_owner(units, ctas, item + kItemCost);
    s.parts = range_owner(units, ctas, item + per - 1) - s.c0 + 1;
    return s;
}

// The starts of this CTA's range and of the next one's, to `range`. Every thread
// looks whether one of them falls into a request of its own.
__device__ __forceinline__ void find_range(const Args& a, const int64_t* pre, int64_t units, int rows, Start* range) {
    const int64_t ctas = units > 0 ? ctas_for(a, units) : 0;
    const int c = blockIdx.x, t = threadIdx.x;
    auto tell = [&](int i, const Start& s) {
        range[i] = s;
        if (i == 0 || c == a.grid - 1) a.starts[c + i] = s;
    };
    if (t < 2 && c + t >= ctas) tell(t, Start{a.B, 0, 0, 0, 1, {0, 0, 0}});
    if (c >= ctas) return;
    const int64_t u[2] = {units * c / ctas, units * (c + 1) / ctas};
    if (a.local_plan) {
        for (int b = t; b < a.B; b += blockDim.x) {
            const int64_t at = pre[b], end = b + 1 < a.B ? pre[b + 1] : units;
#pragma unroll 1
            for (int i = 0; i < 2; ++i)
                if (u[i] >= at && u[i] < end) tell(i, make_start(a, b, a.q_off[b + 1] - a.q_off[b], a.kv_len[b], at, units, ctas, u[i], rows));
        }
    } else if (t < 2 && c + t < ctas) {
        const int b = last_at_most(pre, a.B, u[t]);
        tell(t, make_start(a, b, a.q_off[b + 1] - a.q_off[b], a.kv_len[b], pre[b], units, ctas, u[t], rows));
    }
}

// The same for a batch of at most 64 requests, by one warp, two requests a lane: one
// read of the lengths and one rendezvous, all in 32 bits. A batch of 2^24 units or more
// is left to the block: the first start is then of request -1. (16 decode steps 36.4 to 35.5
// us against 64-bit quotients, with the first segment worked out by that warp alone.)
constexpr int kWarpSeqs = 64;

__device__ __forceinline__ void warp_plan(const Args& a, int rows, Start* range, int lane) {
    constexpr unsigned kAll = 0xffffffffu;
    const bool two = a.B > 32;
    int q0[2], nq[2] = {0, 0}, kv[2] = {0, 0};
    uint32_t n[2] = {0, 0};
    bool bad = false, large = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int b = lane + 32 * i;
        if (b < a.B) {
            q0[i] = a.q_off[b];
            nq[i] = a.q_off[b + 1];
            kv[i] = a.kv_len[b];
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int b = lane + 32 * i;
        if (b >= a.B) continue;
        bad |= bad_request(a, a.cap, q0[i], nq[i], kv[i]) || (b == 0 && q0[i] != 0);
        nq[i] -= q0[i];
        if (bad || (a.dense && a.dense[b] >= 0)) continue;
        const Span s = span_of(a, nq[i], kv[i], rows);
        // (the first product is below 2^32: max_new Hq is)
        const int64_t cost = static_cast<int64_t>(static_cast<uint32_t>(a.hk) * static_cast<uint32_t>(s.row_tiles)) * (s.tiles + kItemCost);
        large |= cost >> 24 != 0;
        n[i] = static_cast<uint32_t>(cost);
    }
    const bool none = __any_sync(kAll, bad);
    if (none && lane == 0) atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
    large = __any_sync(kAll, large);
    uint32_t pre[2] = {0, 0}, run = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (i && !two) break;
        uint32_t incl = n[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += x;
        }
        pre[i] = run + incl - n[i];
        run += __shfl_sync(kAll, incl, 31);
    }
    if (!none && (large || run >> 24 != 0)) {
        if (lane == 0) range->b = -1;
        return;
    }
    const uint32_t units = none ? 0 : run, ctas = static_cast<uint32_t>(ctas_for(a, units));
    // lanes 0 to 15: this CTA's start; the others: the next one's
    const uint32_t c = blockIdx.x + (lane >> 4);
    Start s{a.B, 0, 0, 0, 1, {0, 0, 0}};
    const uint32_t u = c < ctas ? units * c / ctas : 0;
    int b = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // the last request with a cost that begins at or before the unit
        const uint32_t v = __shfl_sync(kAll, u, 16 * h);
        const unsigned lo = __ballot_sync(kAll, n[0] > 0 && pre[0] <= v);
        const unsigned hi = two ? __ballot_sync(kAll, n[1] > 0 && pre[1] <= v) : 0u;
        if (lane >> 4 == h) b = hi ? 63 - __clz(hi) : lo ? 31 - __clz(lo) : 0;
    }
    uint32_t at = __shfl_sync(kAll, pre[0], b & 31);
    int my_nq = __shfl_sync(kAll, nq[0], b & 31), my_kv = __shfl_sync(kAll, kv[0], b & 31);
    if (two) {
        const uint32_t at1 = __shfl_sync(kAll, pre[1], b & 31);
        const int nq1 = __shfl_sync(kAll, nq[1], b & 31), kv1 = __shfl_sync(kAll, kv[1], b & 31);
        if (b >= 32) at = at1, my_nq = nq1, my_kv = kv1;
    }
    if (c < ctas) s = make_start<uint32_t>(a, b, my_nq, my_kv, at, units, ctas, u, rows);
    if ((lane & 15) == 0) {
        range[lane >> 4] = s;
        if (lane == 0 || static_cast<int>(blockIdx.x) == a.grid - 1) a.starts[c] = s;
    }
}

// ------------------------------------------------------------ segments

// A CTA's part of one item: rows [row0, row0 + rows) of request b and KV head g
// over key tiles [first, first + n).
struct alignas(16) Segment {
    int b, g, q0, pos0, kv, row0, rows, first, n;
    int lo, hi;             // cache indices that some row sees
    int all_lo, all_hi;     // and that all rows see
    int c0, parts;          // the CTAs that share the item; parts = 0: the whole item is here
};

// Walks a CTA's range; every warp takes the same steps.
struct Walk {
    const Start* range;     // in shared memory
    int at_b, at_gj, at_off;
    __device__ __forceinline__ Walk(const Start* r, int b, int gj, int off) : range(r), at_b(b), at_gj(gj), at_off(off) {}
    __device__ __forceinline__ bool next(const Args& a, int tile_rows, Segment& s) {
        const Start &begin = range[0], &end = range[1];
        for (;;) {
            if (at_b > end.b || at_b >= a.B ||
                (at_b == end.b && (at_gj > end.gj || (at_gj == end.gj && at_off >= end.off))))
                return false;
            const int q0 = a.q_off[at_b], nq = a.q_off[at_b + 1] - q0, kv = a.kv_len[at_b];
            const Span sp = span_of(a, nq, kv, tile_rows);
            if (sp.row_tiles == 0 || (a.dense && a.dense[at_b] >= 0) || at_gj >= a.hk * sp.row_tiles) {
                ++at_b;
                at_gj = at_off = 0;
                continue;
            }
            s.b = at_b;
            s.g = sp.row_tiles == 1 ? at_gj : at_gj / sp.row_tiles;
            s.q0 = q0;
            s.kv = kv;
            s.pos0 = kv - nq;
            s.row0 = (at_gj - s.g * sp.row_tiles) * tile_rows;
            s.rows = min(tile_rows, nq * a.G - s.row0);
            const int i0 = nq == 1 ? 0 : s.row0 / a.G, i1 = nq == 1 ? 0 : (s.row0 + s.rows - 1) / a.G;
            s.hi = a.causal ? max(0, min(kv, s.pos0 + i1 + 1)) : kv;
            s.lo = a.window > 0 ? max(0, s.pos0 + i0 - a.window + 1) : 0;
            s.all_hi = a.causal ? min(kv, s.pos0 + i0 + 1) : kv;
            s.all_lo = a.window > 0 ? max(0, s.pos0 + i1 - a.window + 1) : 0;
            const int last = at_b == end.b && at_gj == end.gj ? end.off : sp.tiles;
            s.parts = 0;
            if (at_off > 0 || last < sp.tiles) {   // (cut: the CTA's first item, or its last)
                const Start& x = at_off > 0 ? begin : end;
                s.c0 = x.c0;
                s.parts = x.parts;
            }
            // (the first row tiles of a chunk see less than its last)
            s.first = max(sp.tile0 + at_off, s.lo >> a.tile_shift);
            s.n = s.hi > s.lo ? max(0, min(sp.tile0 + last, tiles_below(a, s.hi)) - s.first) : 0;
            at_off = 0;
            ++at_gj;
            return true;
        }
    }
};

// A CTA's first segment, and where the walk goes on; at_b < 0: there is none.
struct alignas(16) First {
    Segment s;
    int at_b, at_gj;
};

// ------------------------------------------------------------ shared memory

// Warps of a CTA: as many as their registers and shares of shared memory allow (d = 128: 12 of 168
// registers 145 us for 64 long decodes when 16 of 128, which spill, took 151).
constexpr int warps_of(int d, int nt) { return d * nt == 64 ? 16 : d * nt == 128 || d == 256 ? 12 : 8; }

template <int D, int NT>
struct Smem {
    static constexpr int kWarps = warps_of(D, NT);
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRows = 8 * NT;
    static constexpr uint32_t kRec = fp4_record(D);
    static constexpr int kKeys = tile_keys(D);
    static constexpr int kMt = kKeys / 16;                       // products over a tile's keys
    static constexpr uint32_t kHalf = kKeys / kFp4Rows * kRec;   // K or V of a tile
    // Halves of a warp in shared memory: one in work and two on their way, or, at d = 256, the
    // other one on its way, which leaves room for 12 warps (three halves and 8 warps: 64 long
    // decodes 151 us in place of 135; at d = 128, where registers hold 12 at most, two halves
    // 129.1 in place of 127.8, with blocks of 8 tokens 200 in place of 197).
    static constexpr int kHalves = D == 256 ? 2 : 3;
    static constexpr int kAcc = D / 16 * NT * 4;          // accumulator registers of a lane
    static constexpr int kVals = kAcc + NT * 4;           // and references and sums
    static constexpr uint32_t kShare = kVals * 32 * 4;    // a warp's share for the join at an item's end
    static constexpr uint32_t ring = 0;                   // [kWarps][kHalves]
    static constexpr uint32_t shares = kWarps * kHalves * kHalf;   // [kWarps]
    static constexpr uint32_t range = shares + kWarps * kShare;    // [2] Start
    static constexpr uint32_t first = range + 2 * sizeof(Start);   // First
    static constexpr uint32_t bars = first + sizeof(First);        // shares written, shares read
    static constexpr uint32_t seg = bars + 16;                     // [kWarps][3] Segment in work, on its way, to be joined
    static constexpr uint32_t total = seg + 3 * kWarps * sizeof(Segment);
    // the plan, before the first tile
    static constexpr uint32_t sums = 0;
    static constexpr uint32_t pre = 32 * 8;
    static_assert(pre + 8 * (kLocalSeqs + 1) <= range && bars % 16 == 0 && total <= 232448, "shared memory of one CTA");
};

// ------------------------------------------------------------ loads

// (the stream is the first to leave L2: what it pushes out otherwise are the lengths,
// the tables and the code of the next launches)
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)),
                 "l"(policy)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits until all but the last N groups of this lane have landed.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The tiles of one warp, every kWarps-th of the CTA's, on their way into its
// halves. A tile is cut into pieces (runs of tokens of one block); lane p looks
// piece p up. Pieces outside the item's keys are not loaded (their blocks may be
// gone).
template <int D, int NT>
struct Feed {
    using L = Smem<D, NT>;
    Walk w;
    Segment* s;              // in shared memory
    const int32_t* table;    // of the segment's request
    const uint8_t *k_head, *v_head;   // the segment's KV head, this lane's 16 bytes
    int k, n;                // the warp's next tile in the segment; its tiles
    int64_t k_at, v_at;      // this lane's piece (-1: not loaded)
    bool live;
    uint64_t policy;

    // (the walk has taken its first step, to `t`)
    __device__ __forceinline__ Feed(const Args& a, const Walk& walk, const Segment& t, bool some, Segment* seg, int warp, int lane)
        : w(walk), s(seg), k(warp), n(0), k_at(-1), v_at(-1), live(some), policy(policy_evict_first()) {
        if (live) take(a, t, lane);
        settle(a, lane);
    }
    __device__ __forceinline__ void take(const Args& a, const Segment& t, int lane) {
        __syncwarp();
        if (lane == 0) *s = t;
        __syncwarp();
        n = t.n;
        table = a.table + static_cast<int64_t>(t.b) * a.table_stride;
        k_head = a.k + static_cast<uint64_t>(t.g) * a.k_sh + 16 * lane;
        v_head = a.v + static_cast<uint64_t>(t.g) * a.v_sh + 16 * lane;
    }
    __device__ __forceinline__ void settle(const Args& a, int lane) {
        while (live && k >= n) {
            k -= n;
            Segment t;
            live = w.next(a, L::kRows, t);
            if (live) take(a, t, lane);
        }
        if (live) look_up(a, lane);
    }
    __device__ __forceinline__ void next(const Args& a, int lane) {
        k += L::kWarps;
        settle(a, lane);
    }
    __device__ __forceinline__ void look_up(const Args& a, int lane) {
        const int pieces = L::kKeys >> a.piece_shift, p = lane & (pieces - 1);   // (one piece: every lane's)
        const int key = (s->first + k) * L::kKeys + (p << a.piece_shift);
        k_at = -1;
        if (key < s->hi && key + (1 << a.piece_shift) > s->lo) {
            const uint32_t blk = a.bs_shift >= 0 ? key >> a.bs_shift : key / a.bs;
            const uint32_t row = key - blk * a.bs;
            uint32_t id = __ldg(table + blk);
            if (id >= a.pool_blocks) {
                atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
                id = 0;
            }
            // (a pool of one block and head may be one run of more than 2^32 bytes)
            const uint64_t in = static_cast<uint64_t>(row) * (L::kRec / kFp4Rows);
            k_at = static_cast<uint64_t>(id) * a.k_sb + in;
            v_at = static_cast<uint64_t>(id) * a.v_sb + in;
        }
    }
    // Keys or values of the tile to `dst`, as a group of copies.
    template <bool kValues>
    __device__ __forceinline__ void issue(const Args& a, uint32_t dst, int lane) const {
        if (live) {
            const int pieces = L::kKeys >> a.piece_shift;
            const uint8_t* head = kValues ? v_head : k_head;
            dst += 16 * lane;
            if (pieces == 1) {   // (one run of tokens)
                if (k_at >= 0) {
                    const uint8_t* src = head + (kValues ? v_at : k_at);
#pragma unroll
                    for (uint32_t o = 0; o < L::kHalf; o += 512)
                        if (o + 512 <= L::kHalf || o + 16 * lane < L::kHalf) copy16(dst + o, src + o, policy);
                }
            } else {
                const uint32_t bytes = (L::kRec / kFp4Rows) << a.piece_shift;
                for (int p = 0; p < pieces; ++p, dst += bytes) {
                    const int64_t at = __shfl_sync(0xffffffffu, kValues && k_at >= 0 ? v_at : k_at, p);
                    if (at < 0) continue;
                    const uint8_t* src = head + at;
#pragma unroll
                    for (uint32_t o = 0; o < L::kHalf; o += 512) {
                        if (o + 16 * lane >= bytes) break;
                        copy16(dst + o, src + o, policy);
                    }
                }
            }
        }
        cp_async_commit();
    }
};

// ------------------------------------------------------------ products

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Transpose of an 8 x 8 matrix of 16-bit values held two in each lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Two fp32 values at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// (low half x, high half y; rounded to nearest)
__device__ __forceinline__ uint32_t half2_of(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Loads from shared memory: a byte, two bytes, N words.
__device__ __forceinline__ uint32_t lds_u8(uint32_t at) {
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(at));
    return r;
}

__device__ __forceinline__ uint32_t lds_u16(uint32_t at) {
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(at));
    return r;
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[N]) {
    static_assert(N == 1 || N == 2 || N % 4 == 0, "words of a lane");
    if constexpr (N == 1) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(at + 4 * i));
    }
}

// The place of CTA c's part of an item that is cut first in CTA c0's range: c0's
// second one (its first may be the end of an earlier item), the others' first.
__device__ __forceinline__ int64_t part_of(int c0, int c) { return 2 * static_cast<int64_t>(c) + (c == c0); }

// ------------------------------------------------------------ one warp's share

// Lane (gid, tig) = (lane / 4, lane % 4). It holds
//   of a key row       elements [tig D/4, (tig + 1) D/4): four of them a product
//   of a value row     elements [gid D/8, (gid + 1) D/8): two a product
//   of the logits      keys gid and gid + 8 of 16, query rows 2 tig and 2 tig + 1 of 8
//   of the result      its elements of a value row, query rows 2 tig and 2 tig + 1
template <int D, int NT>
struct Worker {
    using L = Smem<D, NT>;
    static constexpr int kM = D / 16;
    uint32_t q[D / 16][NT][2];
    uint32_t w[L::kMt][NT][2];     // the tile's weights
    float acc[kM][NT][4];
    float m[NT][2], l[NT][2];      // reference (a logit before its scale), sum of this lane's keys
    float sc[NT][2];               // scale of a row's logits, log2 units
    int gid, tig;

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) m[n][c] = -INFINITY, l[n][c] = 0.0f;
#pragma unroll
            for (int i = 0; i < kM; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][n][c] = 0.0f;
        }
    }

    // Query rows, and then their scaling, as the products' right operand. bf16 rows are scaled by a power of
    // two that takes their largest element to [2^14, 2^15): exact in fp16 down to
    // 2^-31 of it (8 significant bits above the last subnormal).
    __device__ __forceinline__ void fetch_q(const Args& a, const Segment& s) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = s.row0 + 8 * n + gid, tok = a.G == 1 ? r : r / a.G;
            const bool live = 8 * n + gid < s.rows;
            const uint16_t* p = a.q + (s.q0 + static_cast<int64_t>(tok)) * a.q_st +
                                (static_cast<int64_t>(s.g) * a.G + r - tok * a.G) * a.q_sh + tig * (D / 4);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
                q[2 * i][n][0] = x.x, q[2 * i][n][1] = x.y;
                q[2 * i + 1][n][0] = x.z, q[2 * i + 1][n][1] = x.w;
            }
        }
    }
    __device__ __forceinline__ void scale_q(const Args& a) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float back = 1.0f;
            if (a.bf16) {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        top = max(top, max(q[i][n][u] & 0x7fff0000u, (q[i][n][u] << 16) & 0x7fff0000u));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // exponent field of the factor and of its inverse, both kept normal
                const int e = min(max(268 - static_cast<int>(top >> 23), 1), 253);
                const float f = __uint_as_float(static_cast<uint32_t>(e) << 23);
                back = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        q[i][n][u] = half2_of(__uint_as_float(q[i][n][u] << 16) * f, __uint_as_float(q[i][n][u] & 0xffff0000u) * f);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)   // (not zero, which times a masked logit is no number)
                sc[n][c] = fmaxf(a.scale2 * __shfl_sync(0xffffffffu, back, (2 * tig + c) * 4), 1.1754944e-38f);
        }
    }

    // Cache indices [lo, hi) that query row n, c sees.
    __device__ __forceinline__ void sees(const Args& a, const Segment& s, int n, int c, int* lo, int* hi) const {
        const int r = min(8 * n + 2 * tig + c, s.rows - 1);   // (rows behind the last are like it)
        const int pos = s.pos0 + (s.row0 + r) / a.G;
        *hi = a.causal ? min(s.kv, pos + 1) : s.kv;
        *lo = a.window > 0 ? pos - a.window + 1 : 0;
    }

    // Minus infinity where a row does not see a key. (A branch of its own: as selects in
    // the loops above and below it took a tenth of the tile's instructions.)
    __device__ __forceinline__ void mask(const Args& a, const Segment& s, float (&y)[L::kMt][NT][4], int key0) const {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                int lo, hi;
                sees(a, s, n, c, &lo, &hi);
                lo -= key0 + gid;
                hi -= key0 + gid;
#pragma unroll
                for (int i = 0; i < 2 * L::kMt; ++i)
                    if (8 * i < lo || 8 * i >= hi) y[i / 2][n][i % 2 * 2 + c] = -INFINITY;
            }
    }

    // A tile's keys, the first at cache index key0, to the weights of its values;
    // `edge`: not every row sees every key.
    __device__ __forceinline__ void keys(const Args& a, const Segment& s, uint32_t kt, int key0, bool edge) {
        const uint32_t k_at = kt + gid * (D / 2) + tig * (D / 8);
        const uint32_t kf_at = kt + fp4_codes(D) + gid * (D / 16) + tig * (D / 64);
        float y[L::kMt][NT][4];
#pragma unroll
        for (int mt = 0; mt < L::kMt; ++mt) {
            uint32_t w0[D / 32], w1[D / 32];
            lds_words(k_at + 2 * mt * L::kRec, w0);
            lds_words(k_at + (2 * mt + 1) * L::kRec, w1);
            uint32_t f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t at = kf_at + (2 * mt + h) * L::kRec;
                if constexpr (D == 64) f[h] = lds_u8(at);
                else if constexpr (D == 128) f[h] = lds_u16(at);
                else lds_words(at, *reinterpret_cast<uint32_t(*)[1]>(f + h));
            }
            // scales of neighbouring groups, two in a register
            uint32_t g0[(D + 127) / 128], g1[(D + 127) / 128];
#pragma unroll
            for (int j = 0; j < (D + 127) / 128; ++j) {
                g0[j] = fp8_unpack(f[0] >> (16 * j));
                g1[j] = fp8_unpack(f[1] >> (16 * j));
            }
            uint32_t s0 = 0, s1 = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                if (i % 2 == 0) {   // the scale of the next 16 elements, in both halves
                    const uint32_t pick = i / 2 % 2 ? 0x3232u : 0x1010u;
                    s0 = __byte_perm(g0[i / 4], 0, pick);
                    s1 = __byte_perm(g1[i / 4], 0, pick);
                }
                uint32_t x0[4], x1[4];
                fp4_unpack(w0[i], x0);
                fp4_unpack(w1[i], x1);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t op[4] = {mul_f16x2(x0[2 * u], s0), mul_f16x2(x1[2 * u], s1),
                                            mul_f16x2(x0[2 * u + 1], s0), mul_f16x2(x1[2 * u + 1], s1)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (i == 0 && u == 0) mma_f16_first(y[mt][n], op, q[0][n][0], q[0][n][1]);
                        else mma_f16(y[mt][n], op, q[2 * i + u][n][0], q[2 * i + u][n][1]);
                    }
                }
            }
        }
        // masked at the edges of what the rows see; the largest
        if (edge) mask(a, s, y, key0);
        float top[NT][2];
        bool above = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float t = y[0][n][c];
#pragma unroll
                for (int i = 1; i < 2 * L::kMt; ++i) t = fmaxf(t, y[i / 2][n][i % 2 * 2 + c]);
                top[n][c] = t;
                // (a first value is above a reference of minus infinity)
                above |= (t - m[n][c]) * sc[n][c] > kSlack;
            }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float t = top[n][c];
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                    if ((t - m[n][c]) * sc[n][c] > kSlack) {
                        const float f = ex2((m[n][c] - t) * sc[n][c]);   // (0 for a first value)
                        m[n][c] = t;
                        l[n][c] *= f;
#pragma unroll
                        for (int i = 0; i < kM; ++i) acc[i][n][c] *= f, acc[i][n][2 + c] *= f;
                    }
                }
        }
        // weights, transposed to the right operand of the second product
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 f = make_float2(sc[n][0], sc[n][1]);
            // (the difference before the scale: the largest logit gives 2^kBias whatever its size)
            const float2 less = make_float2(m[n][0] == -INFINITY ? 0.0f : -m[n][0], m[n][1] == -INFINITY ? 0.0f : -m[n][1]);
            float2 sum = make_float2(l[n][0], l[n][1]);
#pragma unroll
            for (int mt = 0; mt < L::kMt; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 x = fma2(add2(make_float2(y[mt][n][2 * h], y[mt][n][2 * h + 1]), less), f, make_float2(kBias, kBias));
                    const float2 p = make_float2(ex2(x.x), ex2(x.y));
                    sum = add2(sum, p);
                    w[mt][n][h] = transpose8(half2_of(p.x, p.y));
                }
            l[n][0] = sum.x;
            l[n][1] = sum.y;
        }
    }

    // The tile's values, times its weights.
    __device__ __forceinline__ void values(const Args& a, const Segment& s, uint32_t vt, int key0, bool edge) {
        const uint32_t v_at = vt + 2 * tig * (D / 2) + gid * (D / 16);
        const uint32_t vf_at = vt + fp4_codes(D) + 2 * tig * (D / 16) + gid * (D / 8) / kFp4Group;
        if (edge) take_nan(a, s, vt, key0);
#pragma unroll
        for (int mt = 0; mt < L::kMt; ++mt) {
            constexpr int N = D / 64;
            const uint32_t r0 = v_at + 2 * mt * L::kRec, r1 = r0 + L::kRec;
            uint32_t w00[N], w01[N], w10[N], w11[N];   // record, row 2 tig and 2 tig + 1
            lds_words(r0, w00);
            lds_words(r0 + D / 2, w01);
            lds_words(r1, w10);
            lds_words(r1 + D / 2, w11);
            // scales of both rows' groups: low byte row 2 tig, high byte row 2 tig + 1
            constexpr int kGroups = D == 256 ? 2 : 1;
            uint32_t f0[kGroups], f1[kGroups];
            const uint32_t g0 = vf_at + 2 * mt * L::kRec, g1 = g0 + L::kRec;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                f0[k] = fp8_unpack(lds_u8(g0 + k) | lds_u8(g0 + k + D / 16) << 8);
                f1[k] = fp8_unpack(lds_u8(g1 + k) | lds_u8(g1 + k + D / 16) << 8);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                // the same element of two neighbouring rows in one byte
                constexpr uint32_t kLow = 0x0f0f0f0fu;
                uint32_t e0[4], o0[4], e1[4], o1[4];
                fp4_unpack((w00[i] & kLow) | (w01[i] << 4 & ~kLow), e0);
                fp4_unpack((w00[i] >> 4 & kLow) | (w01[i] & ~kLow), o0);
                fp4_unpack((w10[i] & kLow) | (w11[i] << 4 & ~kLow), e1);
                fp4_unpack((w10[i] >> 4 & kLow) | (w11[i] & ~kLow), o1);
                const uint32_t s0 = f0[kGroups == 2 ? i / 2 : 0], s1 = f1[kGroups == 2 ? i / 2 : 0];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t op[4] = {mul_f16x2(e0[u], s0), mul_f16x2(o0[u], s0), mul_f16x2(e1[u], s1),
                                            mul_f16x2(o1[u], s1)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(acc[4 * i + u][n], op, w[mt][n][0], w[mt][n][1]);
                }
            }
        }
    }

    // Value scales that are no number, at the edge of what the rows see: a weight of
    // zero does not take such a value away. The elements of its group become NaN in
    // the rows that see it, whatever their weight, and the scale zero.
    __device__ __forceinline__ void take_nan(const Args& a, const Segment& s, uint32_t vt, int key0) {
        const int lane = 4 * gid + tig;
        constexpr int kWords = L::kKeys * (D / 16) / 4, kPerRec = D / 8;   // words of scales of a tile, of a record
        bool odd = false;
        for (int i = lane; i < kWords; i += 32) {
            uint32_t w[1];
            lds_words(vt + i / kPerRec * L::kRec + fp4_codes(D) + i % kPerRec * 4, w);
            odd |= scale_is_nan(w[0]) || scale_is_nan(w[0] >> 8) || scale_is_nan(w[0] >> 16) || scale_is_nan(w[0] >> 24);
        }
        if (!__any_sync(0xffffffffu, odd)) return;
        spread_nan(a, s, vt, key0);
        __syncwarp();
        for (int i = lane; i < 4 * kWords; i += 32) {
            const uint32_t at = vt + i / (4 * kPerRec) * L::kRec + fp4_codes(D) + i % (4 * kPerRec);
            if (scale_is_nan(lds_u8(at))) asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(0) : "memory");
        }
        __syncwarp();
    }

    __device__ __forceinline__ void spread_nan(const Args& a, const Segment& s, uint32_t vt, int key0) {
        constexpr int kGroups = D == 256 ? 2 : 1;
#pragma unroll 1
        for (int k = 0; k < L::kKeys; ++k) {
            const int j = key0 + k;
            if (j < s.lo || j >= s.hi) continue;
            const uint32_t f = vt + k / kFp4Rows * L::kRec + fp4_codes(D) + k % kFp4Rows * (D / 16) + gid * (D / 8) / kFp4Group;
#pragma unroll
            for (int x = 0; x < kGroups; ++x) {
                if (!scale_is_nan(lds_u8(f + x))) continue;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        int lo, hi;
                        sees(a, s, n, c, &lo, &hi);
                        if (j < lo || j >= hi) continue;
#pragma unroll
                        for (int i = 0; i < kM; ++i)
                            if (i / 8 == x || kGroups == 1) acc[i][n][c] = acc[i][n][2 + c] = NAN;
                    }
            }
        }
    }

    // This lane's share of the item's result to `p` (32 lanes interleaved): references
    // and sums (over the lanes' keys), then the accumulators.
    __device__ __forceinline__ void put(float* p) const {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float t = l[n][c];
                t += __shfl_xor_sync(0xffffffffu, t, 4);
                t += __shfl_xor_sync(0xffffffffu, t, 8);
                t += __shfl_xor_sync(0xffffffffu, t, 16);
                p[(n * 4 + c) * 32] = m[n][c] * sc[n][c];   // (in log2 units from here on)
                p[(n * 4 + 2 + c) * 32] = t;
            }
#pragma unroll
        for (int i = 0; i < kM; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) p[(NT * 4 + (i * NT + n) * 4 + c) * 32] = acc[i][n][c];
    }
};

// This warp's part of joining the warps' shares of an item, in their order: units of
// two neighbouring elements of four rows.
template <int D, int NT>
__device__ __forceinline__ void join_shares(const Args& a, const Segment& s, const float* shares, int warp, int lane) {
    using L = Smem<D, NT>;
    constexpr int kUnits = D / 16 * NT * 2, kStep = L::kShare / 4;
    const int gid = lane >> 2, tig = lane & 3;
    shares += lane;
    for (int u = warp; u < kUnits; u += L::kWarps) {
        const int c = u & 1, n = (u >> 1) % NT, i = (u >> 1) / NT;
        const int row = 8 * n + 2 * tig + c;
        float m[L::kWarps], top = -INFINITY;
#pragma unroll
        for (int w = 0; w < L::kWarps; ++w) {
            m[w] = shares[w * kStep + (n * 4 + c) * 32];
            top = fmaxf(top, m[w]);
        }
        float sum = 0.0f, lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int w = 0; w < L::kWarps; ++w) {
            const float f = m[w] == top ? 1.0f : ex2(m[w] - top);
            const float* p = shares + w * kStep;
            sum += p[(n * 4 + 2 + c) * 32] * f;
            lo += p[(NT * 4 + (i * NT + n) * 4 + c) * 32] * f;
            hi += p[(NT * 4 + (i * NT + n) * 4 + 2 + c) * 32] * f;
        }
        if (row >= s.rows) continue;
        const int col = gid * (D / 8) + 2 * i;
        if (s.parts) {
            const int64_t part = part_of(s.c0, blockIdx.x) * L::kRows + row;
            *reinterpret_cast<float2*>(a.part_o + part * D + col) = make_float2(lo, hi);
            if (col == 0) a.part_ml[part] = make_float2(top, sum);
            continue;
        }
        const int r = s.row0 + row, tok = r / a.G;
        const int64_t h = static_cast<int64_t>(s.g) * a.G + r - tok * a.G, at = s.q0 + static_cast<int64_t>(tok);
        const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
        uint32_t x;
        if (a.bf16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(lo * inv, hi * inv);
            x = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            x = half2_of(lo * inv, hi * inv);
        }
        *reinterpret_cast<uint32_t*>(a.out + at * a.o_st + h * a.o_sh + col) = x;
        if (a.lse && col == 0) a.lse[at * a.G * a.hk + h] = sum == 0.0f ? -INFINITY : (top - kBias + __log2f(sum)) * kLn2;
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(Smem<D, NT>::kThreads, 1) fp4_attn_kernel(const __grid_constant__ Args a) {
    using L = Smem<D, NT>;
    constexpr int kWarps = L::kWarps;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    if (threadIdx.x == 0) {
        mbar_init(base + L::bars, kWarps);
        mbar_init(base + L::bars + 8, kWarps);
        fence_mbar_init();
    }
    grid_dep_wait();
    grid_dep_launch();
    Start* range = reinterpret_cast<Start*>(smem + L::range);
    First* start = reinterpret_cast<First*>(smem + L::first);
    bool planned = a.B <= kWarpSeqs;
    if (planned && warp == 0) {
        warp_plan(a, L::kRows, range, lane);
        __syncwarp();
    }
    for (;;) {
        if (planned && warp == 0 && range->b >= 0) {
            Walk w(range, range->b, range->gj, range->off);
            Segment t;
            const bool some = w.next(a, L::kRows, t);
            if (lane == 0) {
                if (some) start->s = t;
                start->at_b = some ? w.at_b : -1;
                start->at_gj = w.at_gj;
            }
        }
        __syncthreads();
        if (planned && range->b >= 0) break;
        int64_t* pre = reinterpret_cast<int64_t*>(smem + L::pre);
        int64_t units;
        if (a.local_plan) {
            units = plan_requests<L::kThreads>(a, L::kRows, pre, reinterpret_cast<int64_t*>(smem + L::sums));
        } else {
            pre = a.pre;
            units = __ldcg(a.pre + a.B);
        }
        __syncthreads();   // (the first start is read)
        find_range(a, pre, units, L::kRows, range);
        __syncthreads();
        planned = true;
    }
    // (what only the edges and ends of an item need stays out of the registers)
    Segment* seg = reinterpret_cast<Segment*>(smem + L::seg) + 3 * warp;
    float* shares = reinterpret_cast<float*>(smem + L::shares);
    const uint32_t mine = base + L::ring + warp * (L::kHalves * L::kHalf);
    const uint32_t written = base + L::bars, read = written + 8;
    Worker<D, NT> me;
    me.gid = lane >> 2;
    me.tig = lane & 3;
    const bool some = start->at_b >= 0;
    Walk walk(range, start->at_b, start->at_gj, 0);
    Segment& s = *seg;
    int n, first, all_lo, all_hi;
    // a segment in work, its queries on their way
    auto begin = [&](const Segment& t) {
        __syncwarp();
        if (lane == 0) s = t;
        __syncwarp();
        n = t.n, first = t.first, all_lo = t.all_lo, all_hi = t.all_hi;
        me.fetch_q(a, s);
    };
    auto advance = [&]() -> bool {
        Segment t;
        if (!walk.next(a, L::kRows, t)) return false;
        begin(t);
        return true;
    };
    const Segment one = start->s;
    Feed<D, NT> feed(a, walk, one, some, seg + 1, warp, lane);
    feed.template issue<false>(a, mine, lane);
    feed.template issue<true>(a, mine + L::kHalf, lane);
    if (some) begin(one);   // (while they are on their way)
    if (feed.live) feed.next(a, lane);
    int k = warp;       // the warp's next tile in the segment
    uint32_t half = 0;  // and the half that it begins in
    // The warps do not wait for one another at an item's end: each leaves its share and
    // goes on, and takes its part of the join once all shares are there. Every warp
    // sees every phase of both barriers, one after the other.
    uint32_t ends = 0;  // items whose share this warp has left
    bool owed = false;  // its part of the last one's join is still to do
    auto wait = [&](uint32_t bar, uint32_t parity) {
        int never = 0;
        if (!mbar_wait_bounded(bar, parity & 1, a.spin, &never)) atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_TIMEOUT));
    };
    auto join = [&]() {
        join_shares<D, NT>(a, seg[2], shares, warp, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(read);
        owed = false;
    };
    for (bool more = some; more; more = advance()) {
        me.scale_q(a);
        me.reset();
        for (; k < n; k += kWarps) {
            if (owed && __all_sync(0xffffffffu, mbar_test_wait(written, (ends - 1) & 1))) join();
            const int key0 = (first + k) * L::kKeys;
            const bool edge = key0 < all_lo || key0 + L::kKeys > all_hi;
            if constexpr (L::kHalves == 2) {
                cp_async_wait<1>();
                __syncwarp();
                me.keys(a, s, mine, key0, edge);
                __syncwarp();
                feed.template issue<false>(a, mine, lane);
                cp_async_wait<1>();
                __syncwarp();
                me.values(a, s, mine + L::kHalf, key0, edge);
                __syncwarp();
                feed.template issue<true>(a, mine + L::kHalf, lane);
                if (feed.live) feed.next(a, lane);
                continue;
            }
            // halves in turn: this tile's keys, its values, the next tile's keys (copied
            // over the values of the tile before)
            const uint32_t k_at = mine + half * L::kHalf;
            half = half == 2 ? 0 : half + 1;
            const uint32_t v_at = mine + half * L::kHalf;
            half = half == 2 ? 0 : half + 1;
            __syncwarp();   // (every lane has read the tile before)
            feed.template issue<false>(a, mine + half * L::kHalf, lane);
            cp_async_wait<2>();
            __syncwarp();
            me.keys(a, s, k_at, key0, edge);
            __syncwarp();
            feed.template issue<true>(a, k_at, lane);
            if (feed.live) feed.next(a, lane);
            cp_async_wait<2>();
            __syncwarp();
            me.values(a, s, v_at, key0, edge);
        }
        k -= n;
        if (owed) {
            wait(written, ends - 1);
            join();
        }
        if (ends) wait(read, ends - 1);   // (the shares' places are free)
        me.put(shares + warp * (L::kShare / 4) + lane);
        if (lane == 0) seg[2] = s;
        __syncwarp();
        if (lane == 0) mbar_arrive(written);
        ++ends;
        owed = true;
    }
    if (owed) {
        wait(written, ends - 1);
        join();
    }
    cp_async_wait<0>();
}

// ------------------------------------------------------------ join

constexpr int kJoinThreads = 128;

// Parts of the items that were cut between CTAs, in the order of the CTAs. Block
// (c, r) joins row r of the item that is cut first at the end of CTA c's range, if
// one is.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) fp4_join_kernel(const __grid_constant__ Args a) {
    constexpr int kRows = 8 * NT, kCols = D / 32, kJoinWarps = kJoinThreads / 32;
    __shared__ float acc_s[kJoinWarps][D], sum_s[kJoinWarps];
    grid_dep_wait();
    grid_dep_launch();
    const int c = blockIdx.x, row = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Start* next = a.starts + c + 1;
    if (__ldcg(&next->off) == 0 || __ldcg(&next->c0) != c) return;
    const int b = __ldcg(&next->b), gj = __ldcg(&next->gj), parts = __ldcg(&next->parts);
    const int q0 = a.q_off[b], nq = a.q_off[b + 1] - q0;
    const int row_tiles = static_cast<int>((static_cast<int64_t>(nq) * a.G + kRows - 1) / kRows);
    const int g = gj / row_tiles, r = (gj - g * row_tiles) * kRows + row;
    if (r >= nq * a.G) return;
    auto at = [&](int p) { return part_of(c, c + p) * kRows + row; };
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, __ldcg(a.part_ml + at(p)).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float acc[kCols] = {}, sum = 0.0f;
#pragma unroll 4
    for (int p = warp; p < parts; p += kJoinWarps) {
        const float2 ml = __ldcg(a.part_ml + at(p));
        const float f = ml.x == top ? 1.0f : ex2(ml.x - top);
        sum += ml.y * f;
        const float* o = a.part_o + at(p) * D + lane * kCols;
#pragma unroll
        for (int i = 0; i < kCols; i += 2) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(o + i));
            acc[i] += v.x * f;
            acc[i + 1] += v.y * f;
        }
    }
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc_s[warp][lane * kCols + i] = acc[i];
    if (lane == 0) sum_s[warp] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int k = 0; k < kJoinWarps; ++k) sum += sum_s[k];
    const int tok = r / a.G;
    const int64_t h = static_cast<int64_t>(g) * a.G + r - tok * a.G, t = q0 + static_cast<int64_t>(tok);
    const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
    for (int i = 2 * threadIdx.x; i < D; i += 2 * kJoinThreads) {
        float lo = 0.0f, hi = 0.0f;
        for (int k = 0; k < kJoinWarps; ++k) lo += acc_s[k][i], hi += acc_s[k][i + 1];
        lo *= inv, hi *= inv;
        uint32_t w;
        if (a.bf16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
            w = *reinterpret_cast<const uint32_t*>(&x);
        } else {
            w = half2_of(lo, hi);
        }
        *reinterpret_cast<uint32_t*>(a.out + t * a.o_st + h * a.o_sh + i) = w;
    }
    if (a.lse && threadIdx.x == 0) a.lse[t * a.G * a.hk + h] = sum == 0.0f ? -INFINITY : (top - kBias + __log2f(sum)) * kLn2;
}

// ------------------------------------------------------------ requests with many rows

// Rows from which a request is read through 16 bits. (4 requests of 8K tokens, groups of
// 4, 16 bits and 4: 96 rows 36 and 22 us at d = 64, 63 and 45 at 128, 67 and 60 at
// 256; 192 rows 44 and 31, 69 and 76, 66 and 104; 512 rows 48 and 61, 92 and 175, 85
// and 249.)
__host__ __device__ constexpr int dense_rows(int d) { return d == 64 ? 256 : 128; }

// Units (tiles of keys and items' starts, as the ranges count them) of a call up to which every
// request is computed from the 4-bit rows, by a bound of them from the call's shape: the copy and the kernels
// over it take 22 us at the least. (The 4-bit rows, and the copy, at units: d = 64, 8 heads: 5.8K 16 and 23 us, 11.5K 29
// and 35, 12.6K 39 and 25; 2 heads: 10K 31 to 39 and 33, 17K 47 and 28. d = 128, 4 heads: 2.9K 14 and 25, 6.3K 28 and
// 27, 10.4K 41 and 31. d = 256, 2 heads: 3.2K 20 and 29, 7.8K 28 and 29, 10.8K 32 and 35, 14K 42 and 32.)
constexpr int dense_units(int d) { return d == 128 ? 6000 : 9000; }
constexpr int kDenseBlock = 128;      // tokens of a block of the copy
constexpr int kDenseThreads = 256;

struct DenseArgs {
    const int32_t* q_off;
    const int32_t* kv_len;
    const int32_t* table;
    const uint8_t* k;
    const uint8_t* v;
    uint16_t* k_out;       // [hk][cap * kDenseBlock][d]
    uint16_t* v_out;
    int32_t* status;
    int32_t* base;         // [B] first block of a request's copy, or -1
    int32_t* dense_table;  // [B][width]
    int2* owner;           // [cap] request and table column of a block
    int32_t* used;         // blocks in use
    int64_t k_sb, k_sh, v_sb, v_sh, pool_blocks;
    int B, hk, G, d, bs, bs_shift, table_stride, width, tokens, max_new, window, cap;
};

// First cached token that a request's rows see: those before it are not read (their blocks
// may be gone), and their places in the copy hold anything.
__device__ __forceinline__ int dense_low(const DenseArgs& a, int nq, int kv) {
    return a.window > 0 ? max(0, kv - nq - a.window + 1) : 0;
}

// And the block of 128 that it lies in.
__device__ __forceinline__ int dense_first(const DenseArgs& a, int nq, int kv) { return dense_low(a, nq, kv) / kDenseBlock; }

// Blocks of request b's copy, from `first` on; 0: it is read from the 4-bit rows.
// Lengths that are out of range are noted, and told by the kernels that follow.
__device__ __forceinline__ int dense_blocks(const DenseArgs& a, int b, int* first, int* bad) {
    const int64_t lo = a.q_off[b], hi = a.q_off[b + 1], nq = hi - lo, kv = a.kv_len[b];
    if (bad_request(a, a.tokens, lo, hi, kv) || (b == 0 && lo != 0)) *bad = 1;
    else if (nq * a.G >= dense_rows(a.d) && kv > 0 && kv <= static_cast<int64_t>(a.width) * kDenseBlock) {
        *first = dense_first(a, static_cast<int>(nq), static_cast<int>(kv));
        return static_cast<int>((kv + kDenseBlock - 1) / kDenseBlock) - *first;
    }
    return 0;
}

// Which requests are read through 16 bits, and where their copies lie: those of
// dense_rows() rows and more, in order, as long as their blocks fit. By one block, for
// more requests than a warp of each of the copying blocks lays out for itself.
__global__ void __launch_bounds__(kPlanThreads) fp4_dense_plan_kernel(const DenseArgs a) {
    __shared__ int64_t sums[32];
    __shared__ int most;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) most = 0;
    int64_t blocks = 0;
    int bad = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int first;
        const int64_t n = b < a.B ? dense_blocks(a, b, &first, &bad) : 0;
        int64_t total;
        const int64_t at = blocks + block_scan<kPlanThreads>(n, sums, &total);
        if (b < a.B) a.base[b] = n > 0 && at + n <= a.cap ? static_cast<int32_t>(at) : -1;
        if (n > 0 && at + n <= a.cap) atomicMax(&most, static_cast<int>(at + n));
        blocks += total;
    }
    if (__syncthreads_or(bad)) {   // nothing is computed
        for (int b = tid; b < a.B; b += kPlanThreads) a.base[b] = -1;
        if (tid == 0) *a.used = 0;
        return;
    }
    for (int b0 = 32 * warp; b0 < a.B; b0 += kPlanThreads) {
        const int mine = b0 + lane < a.B ? a.base[b0 + lane] : -1;
        for (unsigned who = __ballot_sync(0xffffffffu, mine >= 0); who; who &= who - 1) {
            const int b = b0 + __ffs(who) - 1, base = __shfl_sync(0xffffffffu, mine, __ffs(who) - 1);
            const int kv = a.kv_len[b], first = dense_first(a, a.q_off[b + 1] - a.q_off[b], kv);
            for (int i = first + lane; i < (kv + kDenseBlock - 1) / kDenseBlock; i += 32) {
                a.dense_table[static_cast<int64_t>(b) * a.width + i] = base + i - first;
                a.owner[base + i - first] = make_int2(b, i);
            }
        }
    }
    if (tid == 0) *a.used = most;
}

// The same for at most 64 requests, by one warp, two a lane: each request's blocks of the
// copy, [base, last), and the blocks in use.
__device__ __forceinline__ void plan_copy(const DenseArgs& a, int* base, int* last, int* first, int* used, int lane) {
    constexpr unsigned kAll = 0xffffffffu;
    int n[2] = {0, 0}, from[2] = {0, 0}, bad = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < a.B) n[i] = dense_blocks(a, lane + 32 * i, from + i, &bad);
    const bool none = __any_sync(kAll, bad != 0);
    int64_t run = 0;
    int most = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int64_t incl = n[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += x;
        }
        const int64_t end = run + incl;
        const bool fits = !none && n[i] > 0 && end <= a.cap;
        base[32 * i + lane] = fits ? static_cast<int>(end - n[i]) : -1;
        last[32 * i + lane] = fits ? static_cast<int>(end) : -1;
        first[32 * i + lane] = from[i];
        if (fits) most = max(most, static_cast<int>(end));
        run += __shfl_sync(kAll, incl, 31);
    }
    most = __reduce_max_sync(kAll, most);
    if (lane == 0) *used = most;
}

// The copies: a block of tokens of one head by a CTA, 16 elements a thread. (The layout with them, in
// place of a launch before: a chunk of 60 tokens 27.6 to 25.6 us, the mixed batch 78.4 to 74.7.)
template <bool kBf16>
__global__ void __launch_bounds__(kDenseThreads) fp4_dense_kernel(const DenseArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    __shared__ int base_s[kWarpSeqs], last_s[kWarpSeqs], first_s[kWarpSeqs], used_s;
    const int lane = threadIdx.x & 31;
    const bool local = a.B <= kWarpSeqs;
    if (local) {
        if (threadIdx.x < 32) plan_copy(a, base_s, last_s, first_s, &used_s, lane);
        __syncthreads();
        if (blockIdx.x == 0 && threadIdx.x < a.B) a.base[threadIdx.x] = base_s[threadIdx.x];
    }
    const int shift = 31 - __clz(a.d / kFp4Group), groups = 1 << shift, units = (local ? used_s : *a.used) * a.hk;
    const int64_t head = static_cast<int64_t>(a.cap) * kDenseBlock * a.d;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int blk = u / a.hk, h = u - blk * a.hk;
        int2 own;
        if (local) {
            const unsigned in0 = __ballot_sync(0xffffffffu, base_s[lane] >= 0 && base_s[lane] <= blk && blk < last_s[lane]);
            const unsigned in1 = __ballot_sync(0xffffffffu, base_s[32 + lane] >= 0 && base_s[32 + lane] <= blk && blk < last_s[32 + lane]);
            own.x = in0 ? __ffs(in0) - 1 : 31 + __ffs(in1);
            own.y = first_s[own.x] + blk - base_s[own.x];
            if (h == 0 && threadIdx.x == 0) a.dense_table[static_cast<int64_t>(own.x) * a.width + own.y] = blk;
        } else {
            own = a.owner[blk];
        }
        const int kv = a.kv_len[own.x], lo = dense_low(a, a.q_off[own.x + 1] - a.q_off[own.x], kv);
        for (int x = threadIdx.x; x < kDenseBlock * groups; x += kDenseThreads) {
            const int r = x >> shift, g = x & (groups - 1), j = own.y * kDenseBlock + r;
            if (j < lo || j >= kv) continue;
            const int col = a.bs_shift >= 0 ? j >> a.bs_shift : j / a.bs, within = j - col * a.bs;
            int id = a.table[static_cast<int64_t>(own.x) * a.table_stride + col];
            if (id < 0 || id >= a.pool_blocks) {
                atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
                id = 0;
            }
            const int64_t rec = static_cast<int64_t>(within / kFp4Rows) * fp4_record(a.d);
            const int code = within % kFp4Rows * (a.d / 2) + 8 * g, scale = fp4_codes(a.d) + within % kFp4Rows * groups + g;
            const int64_t to = h * head + (static_cast<int64_t>(blk) * kDenseBlock + r) * a.d + 16 * g;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const uint8_t* src = (v ? a.v + id * a.v_sb + h * a.v_sh : a.k + id * a.k_sb + h * a.k_sh) + rec;
                const uint2 c = *reinterpret_cast<const uint2*>(src + code);
                const uint32_t s = fp8_unpack(src[scale] * 0x101u);
                uint32_t n[8], o[8];
                fp4_unpack(c.x, *reinterpret_cast<uint32_t(*)[4]>(n));
                fp4_unpack(c.y, *reinterpret_cast<uint32_t(*)[4]>(n + 4));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[i] = mul_f16x2(n[i], s);
                    if (kBf16 && !v) {   // (exact: 6 significant bits; values stay fp16, as their weights are)
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
                        const __nv_bfloat162 w = __floats2bfloat162_rn(f.x, f.y);
                        o[i] = *reinterpret_cast<const uint32_t*>(&w);
                    }
                }
                uint4* dst = reinterpret_cast<uint4*>((v ? a.v_out : a.k_out) + to);
                dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
                dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}

// ------------------------------------------------------------ host

constexpr int kMostRows = 16;

struct Layout {
    size_t pre, starts, ml, o;
    int dense_cap, dense_width;   // blocks of the copy (0: none), entries of a row of its table
    size_t base, table, owner, used, k, v, inner, total;
};

int most_new(const sp_fp4_shape* s) { return s->max_new > 0 ? s->max_new : s->n_tokens; }

// Entries of a row of the copy's table: as many as the pool's tokens fill (the
// workspace is made before a table is there; a longer request, which has blocks
// twice, is read from the 4-bit rows). More of them than kMaxDenseTable in all:
// there is no copy.
constexpr int64_t kMaxDenseTable = int64_t(1) << 28;

int dense_width(const sp_fp4_shape* s) {
    return static_cast<int>((s->pool_blocks * s->block_size + kDenseBlock - 1) / kDenseBlock);
}

// The call over the copy.
sp_paged_shape dense_shape(const sp_fp4_shape* s, int cap, int width) {
    sp_paged_shape p = {};
    p.n_seqs = s->n_seqs;
    p.n_q_heads = s->n_q_heads;
    p.n_kv_heads = s->n_kv_heads;
    p.head_dim = s->head_dim;
    p.dtype = s->dtype;
    p.block_size = kDenseBlock;
    p.table_stride = width;
    p.n_tokens = s->n_tokens;
    p.pool_tokens = static_cast<int64_t>(cap) * kDenseBlock;
    p.q_stride_token = s->q_stride_token, p.q_stride_head = s->q_stride_head;
    p.o_stride_token = s->o_stride_token, p.o_stride_head = s->o_stride_head;
    p.k_stride_token = p.v_stride_token = s->head_dim;
    p.k_stride_head = p.v_stride_head = p.pool_tokens * s->head_dim;
    return p;
}

int grid_of() {
    const int sms = device_sms();
    return sms < kMaxGrid ? sms : kMaxGrid;
}

Layout layout(const sp_fp4_shape* s, int grid) {
    Layout l;
    size_t off = sizeof(WsHeader);
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = (off + bytes + 255) & ~size_t(255);
        return o;
    };
    l.pre = take(8 * (static_cast<size_t>(s->n_seqs) + 1));
    l.starts = take(sizeof(Start) * (static_cast<size_t>(grid) + 1));
    l.ml = take(8 * static_cast<size_t>(grid) * 2 * kMostRows);
    l.o = take(4 * static_cast<size_t>(grid) * 2 * kMostRows * s->head_dim);
    const int64_t rows = static_cast<int64_t>(s->n_tokens) * (s->n_q_heads / s->n_kv_heads);
    const int64_t most = static_cast<int64_t>(most_new(s)) * (s->n_q_heads / s->n_kv_heads);
    l.dense_cap = 0;
    if (s->dense_tokens > 0 && most >= dense_rows(s->head_dim) && static_cast<int64_t>(dense_width(s)) * s->n_seqs <= kMaxDenseTable) {
        // (a request's last block may be begun)
        const int64_t begun = rows / dense_rows(s->head_dim) < s->n_seqs ? rows / dense_rows(s->head_dim) : s->n_seqs;
        l.dense_cap = static_cast<int>(s->dense_tokens / kDenseBlock + begun);
        l.dense_width = dense_width(s);
        const size_t copy = static_cast<size_t>(l.dense_cap) * kDenseBlock * s->n_kv_heads * s->head_dim * 2;
        l.base = take(4 * static_cast<size_t>(s->n_seqs));
        l.table = take(4 * static_cast<size_t>(s->n_seqs) * l.dense_width);
        l.owner = take(8 * static_cast<size_t>(l.dense_cap));
        l.used = take(4);
        l.k = take(copy);
        l.v = take(copy);
        const sp_paged_shape p = dense_shape(s, l.dense_cap, l.dense_width);
        l.inner = take(attn_workspace(&p));
    }
    l.total = off;
    return l;
}

// Rows of an item.
int rows_of(int d, int max_new, int G) { return d == 256 || static_cast<int64_t>(max_new) * G <= 8 ? 8 : 16; }

// A stride of a pool (below 2^32 where it counts).
uint32_t stride32(int64_t extent, int64_t stride) { return extent > 1 ? static_cast<uint32_t>(stride) : 0u; }

template <int D, int NT>
cudaError_t launch_rows(const Args& a, cudaStream_t st) {
    using L = Smem<D, NT>;
    if (!a.local_plan) {
        const cudaError_t e = launch_k(fp4_plan_kernel, 1, kPlanThreads, 0, st, a, L::kRows);
        if (e != cudaSuccess) return e;
    }
    auto kern = fp4_attn_kernel<D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(L::total));
    if (e != cudaSuccess) return e;
    e = launch_k(kern, static_cast<unsigned>(a.grid), L::kThreads, L::total, st, a);
    if (e != cudaSuccess || a.grid < 2 || !a.cuts) return e;
    return launch_k(fp4_join_kernel<D, NT>, dim3(a.grid - 1, L::kRows), kJoinThreads, 0, st, a);
}

}  // namespace

size_t attn_fp4_workspace(const sp_fp4_shape* s) { return layout(s, grid_of()).total; }

cudaError_t launch_paged_attention_fp4(const sp_fp4_shape* s, const sp_fp4_params* p, const int32_t* q_off,
                                       const int32_t* kv_len, const int32_t* table, const uint16_t* q,
                                       const uint8_t* k_pool, const uint8_t* v_pool, uint16_t* out, float* lse,
                                       void* ws, cudaStream_t st) {
    const int d = s->head_dim;
    Args a;
    a.grid = grid_of();
    const Layout l = layout(s, a.grid);
    a.q_off = q_off;
    a.kv_len = kv_len;
    a.table = table;
    a.dense = nullptr;
    a.q = q;
    a.k = k_pool;
    a.v = v_pool;
    a.out = out;
    a.lse = lse;
    a.status = &ws_ptr<WsHeader>(ws, 0)->status;
    a.pre = ws_ptr<int64_t>(ws, l.pre);
    a.starts = ws_ptr<Start>(ws, l.starts);
    a.part_o = ws_ptr<float>(ws, l.o);
    a.part_ml = ws_ptr<float2>(ws, l.ml);
    a.q_st = s->q_stride_token, a.q_sh = s->q_stride_head;
    a.o_st = s->o_stride_token, a.o_sh = s->o_stride_head;
    a.k_sb = stride32(s->pool_blocks, s->k_stride_block), a.k_sh = stride32(s->n_kv_heads, s->k_stride_head);
    a.v_sb = stride32(s->pool_blocks, s->v_stride_block), a.v_sh = stride32(s->n_kv_heads, s->v_stride_head);
    a.pool_blocks = static_cast<uint32_t>(s->pool_blocks);
    a.spin = p->spin_limit > 0 ? p->spin_limit : kDefaultSpin;
    a.B = s->n_seqs;
    a.hk = s->n_kv_heads;
    a.G = s->n_q_heads / s->n_kv_heads;
    a.bs = s->block_size;
    a.table_stride = s->table_stride;
    a.cap = s->n_tokens;
    a.max_new = s->max_new > 0 ? s->max_new : s->n_tokens;
    a.causal = p->causal;
    a.window = p->window <= kMaxCached ? p->window : 0;   // (a longer one hides nothing)
    a.bs_shift = (a.bs & (a.bs - 1)) == 0 ? __builtin_ctz(a.bs) : -1;
    a.tile_shift = __builtin_ctz(tile_keys(d));
    a.piece_shift = a.bs < tile_keys(d) ? __builtin_ctz(a.bs) : a.tile_shift;
    a.local_plan = a.B <= kLocalSeqs;
    a.bf16 = s->dtype == SP_DTYPE_BF16;
    const double scale = p->scale > 0.0f ? static_cast<double>(p->scale) : 1.0 / std::sqrt(static_cast<double>(d));
    a.scale2 = static_cast<float>(scale * p->k_scale * 1.4426950408889634);
    a.v_scale = p->v_scale;
    const int rows = rows_of(d, a.max_new, a.G);
    // (as many as there may be, without those that a padded batch does not have)
    const int64_t items = a.hk * (static_cast<int64_t>(a.max_new) * a.G <= rows ? a.B : static_cast<int64_t>(a.cap) * a.G / rows + a.B);
    a.whole = warps_of(d, rows / 8) * (items >= 64 && (items <= a.grid || 2 * items >= 3 * a.grid) ? 2 : 1);
    const int64_t room = static_cast<int64_t>(a.table_stride) * a.bs, keys = ((room < kMaxCached ? room : kMaxCached) + tile_keys(d) - 1) >> a.tile_shift;
    a.cuts = keys > a.whole;
    if (l.dense_cap > 0 && items * (keys + kItemCost) > dense_units(d)) {
        DenseArgs e;
        e.q_off = q_off;
        e.kv_len = kv_len;
        e.table = table;
        e.k = k_pool;
        e.v = v_pool;
        e.k_out = ws_ptr<uint16_t>(ws, l.k);
        e.v_out = ws_ptr<uint16_t>(ws, l.v);
        e.status = a.status;
        e.base = ws_ptr<int32_t>(ws, l.base);
        e.dense_table = ws_ptr<int32_t>(ws, l.table);
        e.owner = ws_ptr<int2>(ws, l.owner);
        e.used = ws_ptr<int32_t>(ws, l.used);
        e.k_sb = a.k_sb, e.k_sh = a.k_sh, e.v_sb = a.v_sb, e.v_sh = a.v_sh;
        e.pool_blocks = a.pool_blocks;
        e.B = a.B;
        e.hk = a.hk;
        e.G = a.G;
        e.d = d;
        e.bs = a.bs;
        e.bs_shift = a.bs_shift;
        e.table_stride = a.table_stride;
        e.width = l.dense_width;
        e.tokens = a.cap;
        e.max_new = a.max_new;
        e.window = a.window;
        e.cap = l.dense_cap;
        cudaError_t rc = cudaSuccess;
        if (a.B > kWarpSeqs) rc = launch_k(fp4_dense_plan_kernel, 1, kPlanThreads, 0, st, e);
        if (rc != cudaSuccess) return rc;
        const int64_t units = static_cast<int64_t>(l.dense_cap) * a.hk, most = int64_t(8) * a.grid;
        rc = launch_k(a.bf16 ? fp4_dense_kernel<true> : fp4_dense_kernel<false>,
                      static_cast<unsigned>(units < most ? units : most), kDenseThreads, 0, st, e);
        if (rc != cudaSuccess) return rc;
        const sp_paged_shape shape = dense_shape(s, l.dense_cap, l.dense_width);
        sp_attn_params params;
        params.causal = p->causal;
        params.window = p->window;
        params.scale = static_cast<float>(scale * p->k_scale);
        params.spin_limit = p->spin_limit;
        const AttnMore more{e.base, a.status, a.v_scale};
        rc = launch_paged_attention(&shape, &params, q_off, kv_len, e.dense_table, q, e.k_out, e.v_out, out, lse,
                                    ws_ptr<char>(ws, l.inner), st, &more);
        if (rc != cudaSuccess) return rc;
        a.dense = e.base;
    }
    if (d == 64) return rows == 8 ? launch_rows<64, 1>(a, st) : launch_rows<64, 2>(a, st);
    if (d == 128) return rows == 8 ? launch_rows<128, 1>(a, st) : launch_rows<128, 2>(a, st);
    return launch_rows<256, 1>(a, st);
}

}  // namespace sp
