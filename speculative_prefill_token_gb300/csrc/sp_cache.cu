// Block-paged cache of the sparse prefill ("SpecPrefill — Implementation
// Guide", §How It Works / Sparse Prefill: the target prefills the kept
// tokens, each at its original position): the block tables and slots of a
// step's new tokens, and the store of their rotated keys and values.
//
// block_tables_kernel. With held_b = ceil(ctx_b / bs) blocks held and
// need_b = ceil((ctx_b + new_b) / bs) needed by request b, and pre_b the
// blocks taken by the requests before it,
//   table[b][k] = free[n_free - 1 - (pre_b + k - held_b)],  held_b <= k < need_b
//   slot[new_off_b + i] = table[b][p / bs] * bs + p % bs,   p = ctx_b + i.
// Every CTA scans all requests itself (8 bytes each, from L2) and then
// writes the slots of its own tokens: one launch and no communication
// between CTAs. The token at p % bs == 0 of a new block writes that block's
// table entry; the other tokens of the block take its id from the free list,
// so no CTA reads an entry that another one writes. Latency bounds it (three
// dependent reads and a scan): 16 requests 3 us, 4,000 requests with 270,000
// tokens 8 us (11 with the lengths read from L2 in both passes).
//
// append_kv_kernel. A pure stream: each query, key and value row is read
// once and written once. A thread owns one pair of 16-byte vectors of a
// token's rows and walks one or two heads, so that the 64 bytes of cosines and
// sines stay in its registers. Copy bandwidth bounds it: 39,322 tokens of 16 + 4
// heads of 128 take 85 us, 5.93 TB/s of their own bytes (89 % of a measured
// plain copy); 16 tokens 2.6 us, latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sp_device.cuh"
#include "sp_internal.h"
#include "sp_paged.h"

namespace sp {
namespace {

// ------------------------------------------------------------ block tables

constexpr int kTabThreads = 512;

struct TabArgs {
    const int32_t* ctx_len;
    const int32_t* new_off;
    const int32_t* free_blocks;
    const int32_t* n_free;
    int32_t* table;
    int32_t* slot_map;
    int32_t* kv_len;
    int32_t* n_left;
    int32_t* status;
    int B, bs, table_stride, cap, free_cap, pool_blocks;
    int shift;   // log2(bs), or -1
};

__device__ __forceinline__ void raise_status(int32_t* status, int code) {
    if (status) atomicMax(status, code);
}

// x / d for x < 2^31: a shift where d is a power of two, as block sizes mostly are.
__device__ __forceinline__ uint32_t blocks_below(const TabArgs& a, uint32_t x) {
    return a.shift >= 0 ? x >> a.shift : x / static_cast<uint32_t>(a.bs);
}

__device__ __forceinline__ uint32_t blocks_for(const TabArgs& a, uint32_t tokens) {
    const uint32_t full = blocks_below(a, tokens);
    return full + (tokens - full * a.bs != 0);
}

// Last request b in [lo, hi) with off[b] <= t.
__device__ __forceinline__ int request_of(const int32_t* off, int lo, int hi, int t) {
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) block_tables_kernel(const TabArgs a) {
    extern __shared__ int32_t tab_smem[];
    int32_t* off = tab_smem;             // [B + 1] token offsets
    int32_t* ctx = off + a.B + 1;        // [B] cached tokens
    int32_t* pre = ctx + a.B;            // [B] blocks taken by earlier requests
    __shared__ int64_t warp_sum[kTabThreads / 32];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i <= a.B; i += kTabThreads) {
        off[i] = a.new_off[i];
        if (i < a.B) ctx[i] = a.ctx_len[i];
    }
    const int64_t n_free = *a.n_free;
    __syncthreads();
    // each thread takes a run of requests, of odd length (no bank conflicts)
    const int per = (a.B + kTabThreads - 1) / kTabThreads | 1;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    bool ok = n_free >= 0 && n_free <= a.free_cap && off[0] == 0;
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int lo = off[b], hi = off[b + 1], c = ctx[b];
        const int64_t all = static_cast<int64_t>(c) + hi - lo;
        if (hi < lo || hi > a.cap || c < 0 || all > INT32_MAX) {
            ok = false;
            break;
        }
        const uint32_t need = blocks_for(a, static_cast<uint32_t>(all));
        if (need > static_cast<uint32_t>(a.table_stride)) ok = false;
        mine += need - blocks_for(a, c);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    ok = __syncthreads_and(ok);
    int64_t sum = lane < kTabThreads / 32 ? warp_sum[lane] : 0;
    const int64_t own = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    const int64_t total = __shfl_sync(0xffffffffu, sum, 31);
    const int64_t before = __shfl_sync(0xffffffffu, sum - own, warp);
    const bool go = ok && total <= n_free;   // (the same on every thread)
    if (go) {
        int run = static_cast<int>(before + incl - mine);
        for (int b = b0; b < b1; ++b) {
            pre[b] = run;
            run += blocks_for(a, ctx[b] + (off[b + 1] - off[b])) - blocks_for(a, ctx[b]);
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        *a.n_left = static_cast<int32_t>(go ? n_free - total : n_free);
        if (!ok) raise_status(a.status, SP_ERR_DEVICE);
        else if (!go) raise_status(a.status, SP_ERR_CAPACITY);
    }
    __syncthreads();
    for (int b = blockIdx.x * kTabThreads + tid; b < a.B; b += gridDim.x * kTabThreads)
        a.kv_len[b] = go ? ctx[b] + (off[b + 1] - off[b]) : 0;
    // slots of this CTA's run of tokens
    const int64_t per_cta = (static_cast<int64_t>(a.cap) + gridDim.x - 1) / gridDim.x;
    const int t0 = static_cast<int>(min(per_cta * blockIdx.x, static_cast<int64_t>(a.cap)));
    const int t1 = static_cast<int>(min(t0 + per_cta, static_cast<int64_t>(a.cap)));
    const int n_new = go ? off[a.B] : 0;
    const int live = min(t1, n_new);
    int first = 0, last = 0;
    if (t0 < live) {
        first = request_of(off, 0, a.B, t0);
        last = request_of(off, first, a.B, live - 1) + 1;
    }
    for (int t = t0 + tid; t < t1; t += kTabThreads) {
        int32_t slot = -1;
        if (t < live) {
            // the request with off[b] <= t < off[b + 1]
            const int b = request_of(off, first, last, t);
            const uint32_t c = ctx[b], p = c + (t - off[b]);
            const uint32_t k = blocks_below(a, p), r = p - k * a.bs, held = blocks_for(a, c);
            int32_t* entry = a.table + static_cast<int64_t>(b) * a.table_stride + k;
            const int32_t id = k < held ? *entry : a.free_blocks[n_free - 1 - (pre[b] + static_cast<int64_t>(k - held))];
            if (k >= held && r == 0) *entry = id;
            if (id < 0 || id >= a.pool_blocks) raise_status(a.status, SP_ERR_DEVICE);
            else slot = id * a.bs + static_cast<int32_t>(r);
        }
        a.slot_map[t] = slot;
    }
}

// ------------------------------------------------------------ rotate and store

constexpr int kAppThreads = 256;
// Resident CTAs of an SM and the grid's: one full wave (five per SM, a second
// wave of a quarter: 112 us in place of 84).
constexpr int kAppCtas = 4;

struct AppArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* slot_map;
    const int32_t* positions;
    const float* cos_sin;
    const int32_t* n_new;
    uint16_t* q_out;
    uint16_t* k_pool;
    uint16_t* v_pool;
    int32_t* status;
    int64_t q_st, q_sh, qo_st, qo_sh, k_st, k_sh, v_st, v_sh, kp_st, kp_sh, vp_st, vp_sh;
    int64_t pool_tokens;
    int cap, hq, hk, d, half, max_pos;
    int heads_per, groups;  // heads walked by one thread, and groups of them
};

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
    if constexpr (kBf16) {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<const __half2*>(&x));
    }
}

// (rounded to nearest even, the one rounding of the rotated value)
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    if constexpr (kBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// (a, b) -> (a cos - b sin, b cos + a sin) on the 8 elements of each vector.
template <bool kBf16>
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
    uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
    uint32_t* pb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = unpack2<kBf16>(pa[i]), y = unpack2<kBf16>(pb[i]);
        pa[i] = pack2<kBf16>(x.x * c[2 * i] - y.x * s[2 * i], x.y * c[2 * i + 1] - y.y * s[2 * i + 1]);
        pb[i] = pack2<kBf16>(y.x * c[2 * i] + x.x * s[2 * i], y.y * c[2 * i + 1] + x.y * s[2 * i + 1]);
    }
}

template <bool kBf16>
__global__ void __launch_bounds__(kAppThreads, kAppCtas) append_kv_kernel(const AppArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    int64_t n = a.cap;
    if (a.n_new) {
        const int64_t given = *a.n_new;
        n = given < 0 ? 0 : (given < n ? given : n);
    }
    const int pairs = a.d / 16;            // pairs of vectors of a row
    const int per_token = pairs * a.groups;
    const int heads = a.hq + 2 * a.hk;
    const int64_t total = n * per_token;
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * kAppThreads + threadIdx.x; w < total;
         w += static_cast<int64_t>(gridDim.x) * kAppThreads) {
        const int64_t t = w / per_token;
        const int rest = static_cast<int>(w - t * per_token);
        const int group = rest / pairs, i = rest - group * pairs;
        const int64_t slot = a.slot_map[t];
        const bool stored = slot >= 0 && slot < a.pool_tokens;
        if (slot >= a.pool_tokens && rest == 0) raise_status(a.status, SP_ERR_DEVICE);
        // vectors (e0, e1) in elements: a rotated pair, or two neighbours behind it
        const bool turn = i < a.half / 8;
        const int p0 = i * 8, p1 = p0 + a.half;
        const int n0 = 2 * a.half + (i - a.half / 8) * 16;   // neighbours of q and k
        float c[8], s[8];
        if (a.half) {
            const int64_t pos = a.positions[t];
            if (pos < 0 || pos >= a.max_pos) {
                if (rest == 0) raise_status(a.status, SP_ERR_DEVICE);
                continue;
            }
            if (turn) {
                const float* row = a.cos_sin + pos * 2 * a.half + p0;
#pragma unroll
                for (int u = 0; u < 8; u += 4) {
                    const float4 x = __ldg(reinterpret_cast<const float4*>(row + u));
                    const float4 y = __ldg(reinterpret_cast<const float4*>(row + a.half + u));
                    c[u] = x.x, c[u + 1] = x.y, c[u + 2] = x.z, c[u + 3] = x.w;
                    s[u] = y.x, s[u + 1] = y.y, s[u + 2] = y.z, s[u + 3] = y.w;
                }
            }
        }
        const int h1 = min((group + 1) * a.heads_per, heads);
#pragma unroll 2
        for (int h = group * a.heads_per; h < h1; ++h) {
            const uint16_t* src;
            uint16_t* dst;
            const bool is_v = h >= a.hq + a.hk;
            if (h < a.hq) {
                src = a.q + t * a.q_st + h * a.q_sh;
                dst = a.q_out + t * a.qo_st + h * a.qo_sh;
            } else {
                if (!stored) continue;
                const int g = is_v ? h - a.hq - a.hk : h - a.hq;
                src = is_v ? a.v + t * a.v_st + g * a.v_sh : a.k + t * a.k_st + g * a.k_sh;
                dst = is_v ? a.v_pool + slot * a.vp_st + g * a.vp_sh : a.k_pool + slot * a.kp_st + g * a.kp_sh;
            }
            const bool rot = turn && !is_v;
            const int e0 = is_v ? i * 16 : (turn ? p0 : n0), e1 = rot ? p1 : e0 + 8;
            uint4 x = __ldcs(reinterpret_cast<const uint4*>(src + e0));
            uint4 y = __ldcs(reinterpret_cast<const uint4*>(src + e1));
            if (rot) rotate<kBf16>(x, y, c, s);
            *reinterpret_cast<uint4*>(dst + e0) = x;
            *reinterpret_cast<uint4*>(dst + e1) = y;
        }
    }
}

}  // namespace

cudaError_t launch_block_tables(const sp_block_shape* s, const int32_t* ctx_len, const int32_t* new_off,
                                const int32_t* free_blocks, const int32_t* n_free, int32_t* table,
                                int32_t* slot_map, int32_t* kv_len, int32_t* n_left, int32_t* status,
                                cudaStream_t st) {
    TabArgs a;
    a.ctx_len = ctx_len;
    a.new_off = new_off;
    a.free_blocks = free_blocks;
    a.n_free = n_free;
    a.table = table;
    a.slot_map = slot_map;
    a.kv_len = kv_len;
    a.n_left = n_left;
    a.status = status;
    a.B = s->n_seqs;
    a.bs = s->block_size;
    a.table_stride = s->table_stride;
    a.cap = s->n_tokens;
    a.free_cap = s->free_capacity;
    a.pool_blocks = s->pool_blocks;
    a.shift = (a.bs & (a.bs - 1)) == 0 ? __builtin_ctz(a.bs) : -1;
    const size_t smem = (3 * static_cast<size_t>(a.B) + 1) * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    const int64_t work = a.cap > a.B ? a.cap : a.B;
    int64_t grid = (work + kTabThreads - 1) / kTabThreads;
    const int sms = device_sms();
    if (grid > sms) grid = sms;
    return launch_k(block_tables_kernel, static_cast<unsigned>(grid), kTabThreads, smem, st, a);
}

cudaError_t launch_append_kv(const sp_append_shape* s, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                             const int32_t* slot_map, const int32_t* positions, const float* cos_sin,
                             const int32_t* n_new, uint16_t* q_out, uint16_t* k_pool, uint16_t* v_pool,
                             int32_t* status, cudaStream_t st) {
    AppArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.slot_map = slot_map;
    a.positions = positions;
    a.cos_sin = cos_sin;
    a.n_new = n_new;
    a.q_out = q_out;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.status = status;
    a.q_st = s->q_stride_token, a.q_sh = s->q_stride_head;
    a.qo_st = s->qo_stride_token, a.qo_sh = s->qo_stride_head;
    a.k_st = s->k_stride_token, a.k_sh = s->k_stride_head;
    a.v_st = s->v_stride_token, a.v_sh = s->v_stride_head;
    a.kp_st = s->kp_stride_token, a.kp_sh = s->kp_stride_head;
    a.vp_st = s->vp_stride_token, a.vp_sh = s->vp_stride_head;
    a.pool_tokens = s->pool_tokens;
    a.cap = s->n_tokens;
    a.hq = q ? s->n_q_heads : 0;
    a.hk = s->n_kv_heads;
    a.d = s->head_dim;
    a.half = s->rotary_dim / 2;
    a.max_pos = s->max_pos;
    const int heads = a.hq + 2 * a.hk, pairs = a.d / 16, sms = device_sms();
    // two heads a thread once that still fills the GPU (39,322 tokens of 16 + 4
    // heads of 128: one 101 us, two 84, four 92), else one, so that a decode
    // step's few rows are all in flight at once (16 tokens of 8 + 2 heads of 256:
    // one 2.1 us, two 2.6)
    a.heads_per = static_cast<int64_t>(a.cap) * pairs * heads >= int64_t(2) * kAppThreads * kAppCtas * sms ? 2 : 1;
    a.groups = (heads + a.heads_per - 1) / a.heads_per;
    int64_t grid = (static_cast<int64_t>(a.cap) * pairs * a.groups + kAppThreads - 1) / kAppThreads;
    if (grid > int64_t(kAppCtas) * sms) grid = int64_t(kAppCtas) * sms;
    auto kern = s->dtype == SP_DTYPE_BF16 ? append_kv_kernel<true> : append_kv_kernel<false>;
    return launch_k(kern, static_cast<unsigned>(grid), kAppThreads, 0, st, a);
}

}  // namespace sp
