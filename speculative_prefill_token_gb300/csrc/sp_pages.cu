// Pages of the block-paged cache ("SpecPrefill — Implementation Guide", §How It
// Works / Sparse Prefill: what the target holds of a prompt; several
// continuations of one prompt share its blocks, kept tokens of a cached prompt
// move to blocks of their own, ended requests give theirs back).
//
// copy_kv_kernel. A warp takes up to 32 tasks of one pool: a task is a row of all heads
// (or, for whole blocks of a 4-bit pool, one head's records). Its lanes look the tasks'
// places up side by side, and the warp copies 2 KB of them at a time, every load issued
// before the first store. 39,322 rows of 1 KB in two pools, a third of a prompt's, 161 MB:
// 32.9 us, 4.9 TB/s; whole blocks by the same kernel 5.1 to 5.4. Their tokens in 4 bits, 288 bytes in
// four pools, 91 MB: 33.1 us, 2.7 TB/s. What bounds it is not shown: the kernels spill 56 to 136
// bytes a thread, and each 16 bytes cost a division by the run's length.
//
// fork_blocks_kernel. With len_i the cached tokens of src_i, full_i = len_i / bs and
// pre_i the begun blocks of the forks before i,
//   table[dst_i][k] = table[src_i][k],  shared[table[src_i][k]] += 1,  k < full_i
//   table[dst_i][full_i] = free[n_free - 1 - pre_i]          if len_i % bs != 0.
// Every CTA checks and scans all forks itself (no communication between CTAs),
// and then takes its share of runs of 256 table entries. Counts go up by atomic
// additions, whose order changes nothing. (3,200 forks of 400 prompts: 21 us under ncu; each fork adds
// to every count of its parent's blocks, and every CTA scans all forks.)
//
// free_blocks. One kernel takes a holder off every block that a request lets go
// (shared[id] -= 1, so that a block that nobody holds any more is at -1), leaving
// requests with lengths out of range alone; a second, one cluster of 8 CTAs, checks all
// lengths, walks the counts in the order of the ids, each CTA a slice, and puts the
// blocks at -1 behind the free ones. The order of the list is that of the ids, so it
// does not depend on timing. After a length out of range, a count below -1 (a block
// let go too often) or, on request, a cut inside a block that keeps other holders,
// everything is put back.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sp_device.cuh"
#include "sp_fp4.cuh"
#include "sp_fp4.h"
#include "sp_internal.h"
#include "sp_paged.h"

namespace sp {
namespace {

__device__ __forceinline__ void raise_status(int32_t* status, int code) {
    if (status) atomicMax(status, code);
}

// ------------------------------------------------------------ copies

constexpr int kCopyThreads = 256;
constexpr int kCopyWarps = kCopyThreads / 32;
// Resident, of an SM. (Rows of 1 KB 32.9 us by five, 33.7 by four, 33.9 by six; tokens in 4 bits,
// 288 bytes in four pools, 33.2 us by four, 36.4 by five, 32.0 by three.)
constexpr int copy_ctas(int tokens) { return tokens ? 4 : 5; }
// Of a warp's step: what the GPU copies at a time lies close together. (Rows of 1 KB: 12 a
// step 37.5 us, 8 or 4 32.6, 2 33.8, 1 49.8; of 256 bytes: 32 22.1, 16 18.8, 8 20.3; records of
// 4.6 KB: 12 63, 4 57, 1 54.)
constexpr int kStepBytes = 4096;

struct CopyArgs {
    void* pools[SP_MAX_COPY_POOLS];
    const int32_t* src;
    const int32_t* dst;
    const int32_t* table;
    const int32_t* src_off;
    const int32_t* n_used;
    int32_t* status;
    int64_t sb, st, sh;
    int pool_blocks, n_pools, entries, rows, bs, hk, d, fp4, B, table_stride;
    int per_warp;   // tasks of a warp's step
};

// The last b of B with off[b] <= i (off[0] = 0).
__device__ __forceinline__ int request_of(const int32_t* off, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// A slot: its block and its row there.
struct Place {
    int block, row;
};

// Where entry i's first row comes from and goes to; false where it copies nothing.
// (slots stay below 2^31)
__device__ __forceinline__ bool places_of(const CopyArgs& a, int i, Place* from, Place* to) {
    const int s = a.src[i], t = a.dst[i];
    if (s < 0 || t < 0) return false;
    bool ok = true;
    if (a.rows > 1) {
        *from = Place{s, 0};
        *to = Place{t, 0};
    } else {
        const int k = s / a.bs;
        *from = Place{k, s - k * a.bs};
        to->block = t / a.bs;
        to->row = t - to->block * a.bs;
        if (a.table) {
            const int b = request_of(a.src_off, a.B, i);
            from->block = k < a.table_stride ? a.table[static_cast<int64_t>(b) * a.table_stride + k] : -1;
            ok = from->block >= 0;
        }
    }
    ok = ok && from->block < a.pool_blocks && to->block < a.pool_blocks;
    if (!ok) raise_status(a.status, SP_ERR_DEVICE);
    return ok;
}

// Copies `count` runs of n vectors of 16 bytes, by a warp; lane r holds where run r
// comes from and goes to, in bytes into the pool (from -1: nothing), and `at` gives a
// vector's offset in its run. Four vectors of a lane are in flight.
template <typename F>
__device__ __forceinline__ void copy_runs(uint8_t* pool, int64_t in, int64_t out, int count, int n, int lane, F at) {
    constexpr int kAhead = 4;
    // (vector v of run r is number r * n + v: short runs share a step)
    const int all = count * n;
    for (int v0 = 0; v0 < all; v0 += 32 * kAhead) {
        uint4 x[kAhead];
        int64_t to[kAhead];
        bool live[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int v = min(v0 + 32 * u + lane, all - 1), r = v / n;
            const int64_t o = at(v - r * n), from = __shfl_sync(0xffffffffu, in, r);
            to[u] = __shfl_sync(0xffffffffu, out, r) + o;
            live[u] = v0 + 32 * u + lane < all && from >= 0;
            x[u] = make_uint4(0, 0, 0, 0);
            if (live[u]) x[u] = __ldcs(reinterpret_cast<const uint4*>(pool + from + o));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (live[u]) *reinterpret_cast<uint4*>(pool + to[u]) = x[u];
    }
}

// The same for tokens of a 4-bit pool of head size D: of each head D / 2 bytes of codes, 16
// a lane, and D / 16 of scales, a lane's. Lane r holds the records of token r and, in
// `rows`, its rows there.
template <int D>
__device__ __forceinline__ void copy_tokens_fp4(uint8_t* pool, int64_t in, int64_t out, int rows, int count, int hk,
                                                int64_t sh, int lane) {
    constexpr int kAhead = 4, kCodes = D / 32, kUnits = kCodes + 1, kScales = D / 16;
    const int n = hk * kUnits, all = count * n;
    for (int v0 = 0; v0 < all; v0 += 32 * kAhead) {
        uint4 x[kAhead];
        int64_t to[kAhead];
        bool live[kAhead], codes[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int v = min(v0 + 32 * u + lane, all - 1), r = v / n, o = v - r * n, h = o / kUnits, w = o - h * kUnits;
            const int64_t from = __shfl_sync(0xffffffffu, in, r);
            const int both = __shfl_sync(0xffffffffu, rows, r);
            codes[u] = w < kCodes;
            const int64_t at = h * sh + (codes[u] ? 16 * w : fp4_codes(D));
            const int row = codes[u] ? D / 2 : D / 16;
            to[u] = __shfl_sync(0xffffffffu, out, r) + at + (both >> 8) * row;
            live[u] = v0 + 32 * u + lane < all && from >= 0;
            x[u] = make_uint4(0, 0, 0, 0);
            if (!live[u]) continue;
            const uint8_t* src = pool + from + at + (both & 255) * row;
            if (codes[u] || kScales == 16) x[u] = __ldcs(reinterpret_cast<const uint4*>(src));
            else if constexpr (kScales == 8) *reinterpret_cast<uint2*>(&x[u]) = __ldcs(reinterpret_cast<const uint2*>(src));
            else x[u].x = __ldcs(reinterpret_cast<const uint32_t*>(src));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (!live[u]) continue;
            uint8_t* dst = pool + to[u];
            if (codes[u] || kScales == 16) *reinterpret_cast<uint4*>(dst) = x[u];
            else if constexpr (kScales == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(x[u].x, x[u].y);
            else *reinterpret_cast<uint32_t*>(dst) = x[u].x;
        }
    }
}

// kTokens: the head size where tokens of 4-bit pools are copied, 0 where runs of bytes.
template <int kTokens>
__global__ void __launch_bounds__(kCopyThreads, copy_ctas(kTokens)) copy_kv_kernel(const __grid_constant__ CopyArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    int64_t n = a.entries;
    if (a.table) n = min(n, static_cast<int64_t>(max(a.src_off[a.B], 0)));
    if (a.n_used) n = min(n, static_cast<int64_t>(max(*a.n_used, 0)));
    // tasks of an entry: its rows, or the heads of a 4-bit block
    const bool records = !kTokens && a.fp4;
    const int parts = records ? a.hk : a.rows;
    const int64_t tasks = n * parts, steps = (tasks + a.per_warp - 1) / a.per_warp;   // of a pool
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5); w < steps * a.n_pools;
         w += static_cast<int64_t>(gridDim.x) * kCopyWarps) {
        const int p = static_cast<int>(w / steps);
        const int64_t task = (w - p * steps) * a.per_warp + lane;
        const bool mine = lane < a.per_warp && task < tasks;
        const int i = mine ? static_cast<int>(task / parts) : 0, part = static_cast<int>(task - static_cast<int64_t>(i) * parts);
        Place from = {0, 0}, to = {0, 0};
        const bool live = mine && places_of(a, i, &from, &to);
        uint8_t* pool = static_cast<uint8_t*>(a.pools[p]);
        int64_t in, out;
        if (!kTokens && !a.fp4) {
            in = from.block * a.sb + (from.row + part) * a.st;
            out = to.block * a.sb + (to.row + part) * a.st;
        } else if (records) {
            in = from.block * a.sb + part * a.sh;
            out = to.block * a.sb + part * a.sh;
        } else {
            // (a block may be more than 2^31 bytes)
            in = from.block * a.sb + static_cast<int64_t>(from.row / kFp4Rows) * fp4_record(a.d);
            out = to.block * a.sb + static_cast<int64_t>(to.row / kFp4Rows) * fp4_record(a.d);
        }
        if (!live) in = -1;
        const int count = static_cast<int>(min(static_cast<int64_t>(a.per_warp), tasks - (w - p * steps) * a.per_warp));
        [[maybe_unused]] auto plain = [](int v) { return static_cast<int64_t>(v) * 16; };
        if constexpr (kTokens != 0) {
            copy_tokens_fp4<kTokens>(pool, in, out, from.row % kFp4Rows | to.row % kFp4Rows << 8, count, a.hk, a.sh, lane);
        } else if (records) {
            copy_runs(pool, in, out, count, a.bs / kFp4Rows * (fp4_record(a.d) / 16), lane, plain);
        } else {
            const int per_head = a.d / 8;
            if (a.sh == 2 * a.d || a.hk == 1) copy_runs(pool, in, out, count, a.hk * per_head, lane, plain);
            else copy_runs(pool, in, out, count, a.hk * per_head, lane, [&](int v) { return v / per_head * a.sh + v % per_head * 16; });
        }
    }
}

// ------------------------------------------------------------ forks

constexpr int kForkThreads = 512;
constexpr int kRun = 256;         // table entries of a unit of work: 8 a lane

struct PageArgs {
    const int32_t* src;
    const int32_t* dst;
    const int32_t* ctx_len;
    const int32_t* new_len;
    int32_t* table;
    int32_t* shared;
    const int32_t* free_in;
    int32_t* free_out;
    const int32_t* n_free;
    int32_t* kv_len;
    int32_t* copy_src;
    int32_t* copy_dst;
    int32_t* n_left;
    int32_t* status;
    int B, F, bs, table_stride, pool_blocks, free_cap, alone;
};

__device__ __forceinline__ int blocks_for(int tokens, int bs) { return tokens / bs + (tokens % bs != 0); }

__global__ void __launch_bounds__(kForkThreads) fork_blocks_kernel(const PageArgs a) {
    extern __shared__ int32_t fork_smem[];
    int32_t* len = fork_smem;            // [F] tokens of the fork, -1: none
    int32_t* pre = len + a.F;            // [F] begun blocks before it
    uint32_t* taken = reinterpret_cast<uint32_t*>(pre + a.F);   // a bit for each row that becomes a fork
    __shared__ int warp_sum[kForkThreads / 32];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int words = (a.B + 31) / 32;
    for (int i = tid; i < words; i += kForkThreads) taken[i] = 0;
    const int n_free = *a.n_free;
    __syncthreads();
    bool ok = n_free >= 0 && n_free <= a.free_cap;
    constexpr int kAhead = 4;   // entries of a thread whose reads are under way together
    for (int i0 = tid; i0 < a.F; i0 += kAhead * kForkThreads) {
        int s[kAhead], t[kAhead], n[kAhead], held[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kForkThreads;
            s[u] = i < a.F ? a.src[i] : -1;
            t[u] = i < a.F ? a.dst[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            n[u] = -1, held[u] = 0;
            if (s[u] < 0) continue;
            if (s[u] >= a.B || t[u] < 0 || t[u] >= a.B) {
                ok = false;
            } else {
                n[u] = a.ctx_len[s[u]];
                held[u] = a.ctx_len[t[u]];
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * kForkThreads;
            if (i < a.F) len[i] = n[u];
            if (s[u] < 0 || s[u] >= a.B || t[u] < 0 || t[u] >= a.B) continue;
            if (n[u] < 0 || blocks_for(n[u], a.bs) > a.table_stride || held[u] != 0) ok = false;
            if (atomicOr(taken + t[u] / 32, 1u << (t[u] % 32)) >> (t[u] % 32) & 1) ok = false;   // a row forked into twice
        }
    }
    ok = __syncthreads_and(ok);
    // (a row that is forked from and into)
    if (ok)
        for (int i = tid; i < a.F; i += kForkThreads)
            if (len[i] >= 0 && taken[a.src[i] / 32] >> (a.src[i] % 32) & 1) ok = false;
    // each thread takes a run of forks, of odd length (no bank conflicts)
    const int per = (a.F + kForkThreads - 1) / kForkThreads | 1;
    const int i0 = min(tid * per, a.F), i1 = min(i0 + per, a.F);
    int mine = 0;
    for (int i = i0; i < i1; ++i) mine += len[i] > 0 && len[i] % a.bs != 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    ok = __syncthreads_and(ok);
    int before = 0, total = 0;
    for (int k = 0; k < kForkThreads / 32; ++k) {
        if (k < warp) before += warp_sum[k];
        total += warp_sum[k];
    }
    before += incl - mine;
    for (int i = i0; i < i1; ++i) {
        pre[i] = before;
        before += len[i] > 0 && len[i] % a.bs != 0;
    }
    const bool go = ok && total <= n_free;   // (the same on every thread)
    if (blockIdx.x == 0 && tid == 0) {
        *a.n_left = go ? n_free - total : n_free;
        if (!ok) raise_status(a.status, SP_ERR_DEVICE);
        else if (!go) raise_status(a.status, SP_ERR_CAPACITY);
    }
    __syncthreads();
    for (int b = blockIdx.x * kForkThreads + tid; b < a.B; b += gridDim.x * kForkThreads)
        if (!go || !(taken[b / 32] >> (b % 32) & 1)) a.kv_len[b] = a.ctx_len[b];
    // units: runs of kRun table entries of a fork, its begun block with the run that holds it
    const int runs = (a.table_stride + kRun - 1) / kRun;
    const int64_t units = static_cast<int64_t>(a.F) * runs;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kForkThreads / 32) + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * (kForkThreads / 32)) {
        const int i = static_cast<int>(u / runs), k0 = static_cast<int>(u - static_cast<int64_t>(i) * runs) * kRun;
        const int n = go ? len[i] : -1;
        const int full = n > 0 ? n / a.bs : 0;
        const bool begun = n > 0 && n % a.bs != 0;
        if (k0 == 0 && lane == 0) {
            if (!begun) a.copy_src[i] = a.copy_dst[i] = -1;
            if (n >= 0) a.kv_len[a.dst[i]] = n;
        }
        if (n <= 0 || k0 > full) continue;
        const int32_t* from = a.table + static_cast<int64_t>(a.src[i]) * a.table_stride;
        int32_t* to = a.table + static_cast<int64_t>(a.dst[i]) * a.table_stride;
        int id[kRun / 32];
#pragma unroll
        for (int x = 0; x < kRun / 32; ++x) {
            const int k = k0 + 32 * x + lane;
            id[x] = k < full ? from[k] : 0;
        }
#pragma unroll
        for (int x = 0; x < kRun / 32; ++x) {
            const int k = k0 + 32 * x + lane;
            if (k >= full) continue;
            to[k] = id[x];
            if (id[x] < 0 || id[x] >= a.pool_blocks) raise_status(a.status, SP_ERR_DEVICE);
            else atomicAdd(a.shared + id[x], 1);
        }
        if (begun && full - k0 < kRun && lane == 0) {
            const int fresh = a.free_in[n_free - 1 - pre[i]];
            to[full] = fresh;
            a.copy_src[i] = from[full];
            a.copy_dst[i] = fresh;
            if (fresh < 0 || fresh >= a.pool_blocks) raise_status(a.status, SP_ERR_DEVICE);
        }
    }
}

// ------------------------------------------------------------ frees

constexpr int kDropThreads = 256;
constexpr int kSweepThreads = 1024;
constexpr int kSweepCtas = 8;     // one cluster
constexpr int kSweepPer = 4 * kSweepThreads;   // counts of a step: 4 a thread

// Whether a request may be cut like this.
__device__ __forceinline__ bool cut_fits(const PageArgs& a, int ctx, int left) {
    return left >= 0 && left <= ctx && blocks_for(ctx, a.bs) <= a.table_stride;
}

// Adds `by` to the count of every block that a request lets go: runs of kRun
// entries of a row, from warp w of `warps`.
__device__ __forceinline__ void count_drops(const PageArgs& a, int by, int64_t w, int64_t warps, int32_t* status) {
    const int lane = threadIdx.x & 31, runs = (a.table_stride + kRun - 1) / kRun;
    const int64_t units = static_cast<int64_t>(a.B) * runs;
    for (int64_t u = w; u < units; u += warps) {
        const int b = static_cast<int>(u / runs), k0 = static_cast<int>(u - static_cast<int64_t>(b) * runs) * kRun;
        const int ctx = a.ctx_len[b], left = a.new_len[b];
        if (!cut_fits(a, ctx, left)) continue;
        const int keep = blocks_for(left, a.bs), held = blocks_for(ctx, a.bs);
        if (k0 >= held || k0 + kRun <= keep) continue;
        const int32_t* row = a.table + static_cast<int64_t>(b) * a.table_stride;
        int id[kRun / 32];
#pragma unroll
        for (int x = 0; x < kRun / 32; ++x) {
            const int k = k0 + 32 * x + lane;
            id[x] = k >= keep && k < held ? row[k] : -1;
        }
#pragma unroll
        for (int x = 0; x < kRun / 32; ++x) {
            const int k = k0 + 32 * x + lane;
            if (k < keep || k >= held) continue;
            if (id[x] < 0 || id[x] >= a.pool_blocks) raise_status(status, SP_ERR_DEVICE);
            else atomicAdd(a.shared + id[x], by);
        }
    }
}

__global__ void __launch_bounds__(kDropThreads) drop_blocks_kernel(const PageArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    count_drops(a, -1, static_cast<int64_t>(blockIdx.x) * (kDropThreads / 32) + (threadIdx.x >> 5),
                static_cast<int64_t>(gridDim.x) * (kDropThreads / 32), a.status);
}

// Counts [4 i, 4 i + 4) of the pool's (0 behind its end).
__device__ __forceinline__ int4 counts_at(const PageArgs& a, int64_t i) {
    int4 v = make_int4(0, 0, 0, 0);
    if (i < a.pool_blocks) v.x = a.shared[i];
    if (i + 1 < a.pool_blocks) v.y = a.shared[i + 1];
    if (i + 2 < a.pool_blocks) v.z = a.shared[i + 2];
    if (i + 3 < a.pool_blocks) v.w = a.shared[i + 3];
    return v;
}

__global__ void __cluster_dims__(kSweepCtas, 1, 1) __launch_bounds__(kSweepThreads) sweep_blocks_kernel(const PageArgs a) {
    namespace cg = cooperative_groups;
    __shared__ int sums[32];
    __shared__ int told[2];     // blocks freed in the CTA's slice; something is wrong there
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_free = *a.n_free;
    bool low = n_free < 0 || n_free > a.free_cap;   // something is wrong
    for (int b = rank * kSweepThreads + tid; b < a.B; b += kSweepCtas * kSweepThreads) {
        const int ctx = a.ctx_len[b], left = a.new_len[b];
        if (!cut_fits(a, ctx, left)) {
            low = true;
        } else if (a.alone && left < ctx && left % a.bs != 0) {   // (the block that the cut leaves begun)
            const int id = a.table[static_cast<int64_t>(b) * a.table_stride + left / a.bs];
            low |= id >= 0 && id < a.pool_blocks && a.shared[id] > 0;
        }
    }
    // a slice of whole steps for each CTA
    const int64_t steps = (static_cast<int64_t>(a.pool_blocks) + kSweepPer - 1) / kSweepPer;
    const int64_t first = steps * rank / kSweepCtas, last = steps * (rank + 1) / kSweepCtas;
    int freed = 0;
    for (int64_t s = first; s < last; ++s) {
        const int4 v = counts_at(a, s * kSweepPer + 4 * tid);
        freed += (v.x == -1) + (v.y == -1) + (v.z == -1) + (v.w == -1);
        low |= min(min(v.x, v.y), min(v.z, v.w)) < -1;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) freed += __shfl_xor_sync(0xffffffffu, freed, o);
    if (lane == 0) sums[warp] = freed;
    low = __syncthreads_or(low);
    if (tid == 0) {
        int all = 0;
        for (int k = 0; k < 32; ++k) all += sums[k];
        told[0] = all;
        told[1] = low;
    }
    cluster.sync();
    int64_t base = n_free, total = 0;
    bool bad = false;
    for (int k = 0; k < kSweepCtas; ++k) {
        const int* o = cluster.map_shared_rank(told, k);
        if (k < rank) base += o[0];
        total += o[0];
        bad |= o[1] != 0;
    }
    const bool room = n_free + total <= a.free_cap;
    const bool go = !bad && room;
    cluster.sync();   // (every count is read before a block changes its own again)
    for (int b = rank * kSweepThreads + tid; b < a.B; b += kSweepCtas * kSweepThreads)
        a.kv_len[b] = go ? a.new_len[b] : a.ctx_len[b];
    if (rank == 0 && tid == 0) {
        *a.n_left = static_cast<int32_t>(go ? n_free + total : n_free);
        if (bad) raise_status(a.status, SP_ERR_DEVICE);
        else if (!room) raise_status(a.status, SP_ERR_CAPACITY);
    }
    if (!go) {   // every holder back
        count_drops(a, 1, static_cast<int64_t>(rank) * 32 + warp, int64_t(32) * kSweepCtas, nullptr);
        return;
    }
    if (told[0] == 0) return;
    for (int64_t s = first; s < last; ++s) {
        const int64_t i = s * kSweepPer + 4 * tid;
        const int4 v = counts_at(a, i);
        const int mine = (v.x == -1) + (v.y == -1) + (v.z == -1) + (v.w == -1);
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        __syncthreads();   // (the sums of the step before are read)
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int own = sums[lane], run = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += x;
        }
        const int all = __shfl_sync(0xffffffffu, run, 31);
        int64_t at = base + __shfl_sync(0xffffffffu, run - own, warp) + incl - mine;
        const int c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c[k] == -1) {
                a.free_out[at++] = static_cast<int32_t>(i + k);
                a.shared[i + k] = 0;
            }
        base += all;
    }
}

}  // namespace

cudaError_t launch_copy_kv(const sp_copy_shape* s, void* const* pools, const int32_t* src, const int32_t* dst,
                           const int32_t* block_table, const int32_t* src_off, const int32_t* n_used,
                           int32_t* status, cudaStream_t st) {
    CopyArgs a = {};
    for (int i = 0; i < s->n_pools; ++i) a.pools[i] = pools[i];
    a.src = src;
    a.dst = dst;
    a.table = block_table;
    a.src_off = src_off;
    a.n_used = n_used;
    a.status = status;
    a.sb = s->stride_block, a.st = s->stride_token, a.sh = s->stride_head;
    a.pool_blocks = static_cast<int>(s->pool_blocks);
    a.n_pools = s->n_pools;
    a.entries = s->n_entries;
    a.rows = s->rows;
    a.bs = s->block_size;
    a.hk = s->n_kv_heads;
    a.d = s->head_dim;
    a.fp4 = s->fp4;
    a.B = s->n_seqs;
    a.table_stride = s->table_stride;
    // as many tasks a step as leave every warp of the GPU one, and kStepBytes
    const int64_t tasks = static_cast<int64_t>(a.entries) * (a.fp4 && a.rows > 1 ? a.hk : a.rows);
    const int tokens = a.fp4 && a.rows == 1 ? a.d : 0;
    const int64_t most = int64_t(copy_ctas(tokens)) * device_sms(), all = tasks * a.n_pools / (most * kCopyWarps);
    const int64_t bytes = !a.fp4 ? 2 * int64_t(a.hk) * a.d : a.rows > 1 ? a.bs / kFp4Rows * int64_t(fp4_record(a.d)) : a.hk * (9 * int64_t(a.d) / 16);
    const int64_t few = kStepBytes / bytes, per = all < few ? all : few;
    a.per_warp = static_cast<int>(per < 1 ? 1 : per > 32 ? 32 : per);
    const int64_t steps = (tasks + a.per_warp - 1) / a.per_warp * a.n_pools;
    int64_t grid = (steps + kCopyWarps - 1) / kCopyWarps;
    if (grid > most) grid = most;
    auto kern = tokens == 0 ? copy_kv_kernel<0> : tokens == 64 ? copy_kv_kernel<64> : tokens == 128 ? copy_kv_kernel<128> : copy_kv_kernel<256>;
    return launch_k(kern, static_cast<unsigned>(grid), kCopyThreads, 0, st, a);
}

cudaError_t launch_fork_blocks(const sp_pages_shape* s, const int32_t* src, const int32_t* dst,
                               const int32_t* ctx_len, int32_t* table, int32_t* shared, const int32_t* free_blocks,
                               const int32_t* n_free, int32_t* kv_len, int32_t* copy_src, int32_t* copy_dst,
                               int32_t* n_left, int32_t* status, cudaStream_t st) {
    PageArgs a = {};
    a.src = src;
    a.dst = dst;
    a.ctx_len = ctx_len;
    a.table = table;
    a.shared = shared;
    a.free_in = free_blocks;
    a.n_free = n_free;
    a.kv_len = kv_len;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.n_left = n_left;
    a.status = status;
    a.B = s->n_seqs;
    a.F = s->n_forks;
    a.bs = s->block_size;
    a.table_stride = s->table_stride;
    a.pool_blocks = s->pool_blocks;
    a.free_cap = s->free_capacity;
    const size_t smem = 8 * static_cast<size_t>(a.F) + 4 * ((static_cast<size_t>(a.B) + 31) / 32);
    // (the limit of the largest call, whatever this one takes: a smaller one set by another
    // thread between these two calls would have the launch refused)
    if (smem > 48 * 1024) {
        constexpr int kMost = 8 * kMaxForks + 4 * ((kMaxTableSeqs + 31) / 32);
        const cudaError_t e = cudaFuncSetAttribute(fork_blocks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
    }
    const int64_t units = static_cast<int64_t>(a.F) * ((a.table_stride + kRun - 1) / kRun);
    const int64_t work = units * 32 > a.B ? units * 32 : a.B;
    int64_t grid = (work + kForkThreads - 1) / kForkThreads;
    const int sms = device_sms();
    if (grid > sms) grid = sms;
    return launch_k(fork_blocks_kernel, static_cast<unsigned>(grid), kForkThreads, smem, st, a);
}

cudaError_t launch_free_blocks(const sp_pages_shape* s, const int32_t* ctx_len, const int32_t* new_len,
                               const int32_t* table, int32_t* shared, int32_t* free_blocks, const int32_t* n_free,
                               int32_t* kv_len, int32_t* n_left, int32_t* status, cudaStream_t st) {
    PageArgs a = {};
    a.ctx_len = ctx_len;
    a.new_len = new_len;
    a.table = const_cast<int32_t*>(table);
    a.shared = shared;
    a.free_out = free_blocks;
    a.n_free = n_free;
    a.kv_len = kv_len;
    a.n_left = n_left;
    a.status = status;
    a.B = s->n_seqs;
    a.bs = s->block_size;
    a.table_stride = s->table_stride;
    a.pool_blocks = s->pool_blocks;
    a.free_cap = s->free_capacity;
    a.alone = s->alone;
    const int64_t units = static_cast<int64_t>(a.B) * ((a.table_stride + kRun - 1) / kRun);
    int64_t grid = (units + kDropThreads / 32 - 1) / (kDropThreads / 32);
    const int64_t most = int64_t(2) * device_sms();
    if (grid > most) grid = most;
    const cudaError_t e = launch_k(drop_blocks_kernel, static_cast<unsigned>(grid), kDropThreads, 0, st, a);
    if (e != cudaSuccess) return e;
    return launch_k(sweep_blocks_kernel, kSweepCtas, kSweepThreads, 0, st, a);
}

}  // namespace sp
