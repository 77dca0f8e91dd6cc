// Attention of new tokens over a block-paged cache ("SpecPrefill —
// Implementation Guide", §How It Works / Sparse Prefill: the target's
// attention over the kept tokens, and its decode steps after them).
//
// For a query row (token i of request b, head h) with visible cache indices
// [lo, hi), and KV head g = h / G,
//   out = sum_j exp2(y_j - m) v_j / sum_j exp2(y_j - m),  y_j = scale log2(e) <q, k_j>,
// in one pass over the keys: m is the running maximum, and the sum and the
// accumulator are scaled by exp2(m_old - m_new) when it grows.
//
// One warp per row, the head dimension spread over its lanes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "sp_device.cuh"
#include "sp_internal.h"
#include "sp_paged.h"

namespace sp {
namespace {

constexpr int kAttnThreads = 256;

struct AttnArgs {
    const int32_t* q_off;
    const int32_t* kv_len;
    const int32_t* table;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* out;
    float* lse;
    int32_t* status;
    int64_t q_st, q_sh, o_st, o_sh, k_st, k_sh, v_st, v_sh, pool_tokens;
    int B, hq, hk, G, bs, table_stride, cap, causal, window;
    float scale2;
};

template <bool kBf16>
__device__ __forceinline__ float to_f32(uint16_t x) {
    if constexpr (kBf16) return __uint_as_float(static_cast<uint32_t>(x) << 16);
    return __half2float(__ushort_as_half(x));
}

template <bool kBf16>
__device__ __forceinline__ uint16_t from_f32(float x) {
    if constexpr (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    return __half_as_ushort(__float2half_rn(x));
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(kAttnThreads) attn_rows_kernel(const AttnArgs a) {
    grid_dep_wait();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    // (a request's lengths are checked by every row of the batch: nothing is
    // computed for an inconsistent batch)
    int bad = a.q_off[0] != 0;
    for (int b = threadIdx.x; b < a.B; b += kAttnThreads) {
        const int lo = a.q_off[b], hi = a.q_off[b + 1], kv = a.kv_len[b];
        bad |= hi < lo || hi > a.cap || kv < 0 || (static_cast<int64_t>(kv) + a.bs - 1) / a.bs > a.table_stride;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
        return;
    }
    const int64_t rows = static_cast<int64_t>(a.q_off[a.B]) * a.hq;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAttnThreads / 32);
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kAttnThreads / 32) + (threadIdx.x >> 5); w < rows;
         w += warps) {
        const int t = static_cast<int>(w / a.hq), h = static_cast<int>(w - static_cast<int64_t>(t) * a.hq);
        int b = 0, e = a.B;
        while (e - b > 1) {
            const int mid = (b + e) >> 1;
            if (a.q_off[mid] <= t) b = mid; else e = mid;
        }
        const int kv = a.kv_len[b];
        int hi = kv, lo = 0;
        if (a.causal) {
            hi = kv - a.q_off[b + 1] + t + 1;
            if (hi < 0) hi = 0;
            if (a.window > 0 && hi > a.window) lo = hi - a.window;
        }
        float q[E], acc[E];
        const uint16_t* qr = a.q + t * a.q_st + h * a.q_sh + lane * E;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            q[i] = to_f32<kBf16>(qr[i]);
            acc[i] = 0.0f;
        }
        float m = -INFINITY, l = 0.0f;
        const int g = h / a.G;
        for (int j = lo; j < hi; ++j) {
            const int id = a.table[static_cast<int64_t>(b) * a.table_stride + j / a.bs];
            int64_t row = static_cast<int64_t>(id) * a.bs + j % a.bs;
            if (id < 0 || row >= a.pool_tokens) {
                atomicCAS(a.status, 0, static_cast<int32_t>(SP_ERR_DEVICE));
                row = 0;
            }
            const uint16_t* kr = a.k + row * a.k_st + g * a.k_sh + lane * E;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) s += q[i] * to_f32<kBf16>(kr[i]);
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            s *= a.scale2;
            const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.0f : mn;
            const float f = exp2f(m - base), p = exp2f(s - base);
            l = l * f + p;
            const uint16_t* vr = a.v + row * a.v_st + g * a.v_sh + lane * E;
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = acc[i] * f + p * to_f32<kBf16>(vr[i]);
            m = mn;
        }
        uint16_t* o = a.out + t * a.o_st + h * a.o_sh + lane * E;
        const float inv = hi > lo ? 1.0f / l : 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = from_f32<kBf16>(acc[i] * inv);
        if (a.lse && lane == 0)
            a.lse[w] = hi > lo ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

}  // namespace

size_t attn_workspace(const sp_paged_shape*) { return sizeof(WsHeader); }

cudaError_t launch_paged_attention(const sp_paged_shape* s, const sp_attn_params* p, const int32_t* q_off,
                                   const int32_t* kv_len, const int32_t* table, const uint16_t* q,
                                   const uint16_t* k_pool, const uint16_t* v_pool, uint16_t* out, float* lse,
                                   void* ws, cudaStream_t st) {
    AttnArgs a;
    a.q_off = q_off;
    a.kv_len = kv_len;
    a.table = table;
    a.q = q;
    a.k = k_pool;
    a.v = v_pool;
    a.out = out;
    a.lse = lse;
    a.status = &ws_ptr<WsHeader>(ws, 0)->status;
    a.q_st = s->q_stride_token, a.q_sh = s->q_stride_head;
    a.o_st = s->o_stride_token, a.o_sh = s->o_stride_head;
    a.k_st = s->k_stride_token, a.k_sh = s->k_stride_head;
    a.v_st = s->v_stride_token, a.v_sh = s->v_stride_head;
    a.pool_tokens = s->pool_tokens;
    a.B = s->n_seqs;
    a.hq = s->n_q_heads;
    a.hk = s->n_kv_heads;
    a.G = a.hq / a.hk;
    a.bs = s->block_size;
    a.table_stride = s->table_stride;
    a.cap = s->n_tokens;
    a.causal = p->causal;
    a.window = p->window;
    const double scale = p->scale > 0.0f ? static_cast<double>(p->scale) : 1.0 / std::sqrt(static_cast<double>(s->head_dim));
    a.scale2 = static_cast<float>(scale * 1.4426950408889634);
    const bool bf = s->dtype == SP_DTYPE_BF16;
    auto kern = s->head_dim == 64    ? (bf ? attn_rows_kernel<64, true> : attn_rows_kernel<64, false>)
                : s->head_dim == 128 ? (bf ? attn_rows_kernel<128, true> : attn_rows_kernel<128, false>)
                                     : (bf ? attn_rows_kernel<256, true> : attn_rows_kernel<256, false>);
    return launch_k(kern, static_cast<unsigned>(8 * device_sms()), kAttnThreads, 0, st, a);
}

}  // namespace sp
