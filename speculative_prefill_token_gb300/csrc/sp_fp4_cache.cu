// Rows of the 4-bit cache ("SpecPrefill — Implementation Guide", §How It
// Works / Sparse Prefill: the target prefills the kept tokens, each at its
// original position): the store of a step's rotated keys and values, and rows
// read back as 16-bit values.
//
// append_kv_fp4_kernel. A thread owns pairs of 16-byte vectors of query rows, or two
// groups of 16 elements of a key or value row: the groups that are rotated with one
// another, or neighbours. It needs no other thread for a group's largest element, its
// scale and its 8 bytes of codes. (Where half the rotated elements are no whole
// number of groups, a key's threads read the partners of their neighbours' groups.)
// Every operation of the stored value is one of 32 bits, rounded as the definition in
// specprefill.h has it: the division by the scale as r = 1 / s, q = y r, q - (q s - y) r
// with fused operations, which is the rounded quotient (Markstein: r is rounded
// correctly, and no quotient here overflows; one that underflows is far below the
// smallest code's border).
//
// 39,322 tokens of 16/4 heads of 128 (bf16) are 322 MB of queries and 81 + 23 MB of
// keys and values; the queries take 54 us (6.0 TB/s, the memory), keys and values 36 us, 2.4 times
// their bytes at a copy's rate: no pipe is full (17 instructions an element, issue slots 55 % busy), the
// loads in flight wait in registers, 24 warps an SM (a thread's elements are under way before its slot and
// position are known, 93 to 90 us in all; the next row's read ahead as well: no gain). 16 tokens of 8/2 heads of
// 256: 2.3 us, a launch and three reads that follow one another.
//
// unpack_fp4_kernel. A thread turns 8 bytes of codes and a scale into 32 bytes (39,424 rows of 4 heads
// of 128, 52 MB: 11.7 us, 4.4 TB/s, most of it writes).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sp_device.cuh"
#include "sp_fp4.cuh"
#include "sp_fp4.h"
#include "sp_internal.h"
#include "sp_paged.h"

namespace sp {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void raise_status(int32_t* status, int code) {
    if (status) atomicMax(status, code);
}

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
    if constexpr (kBf16) {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<const __half2*>(&x));
    }
}

// (rounded to nearest even, the one rounding of the value)
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

template <bool kBf16>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<kBf16>(w[i]);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}

// ------------------------------------------------------------ rotate and store

struct AppArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* slot_map;
    const int32_t* positions;
    const float* cos_sin;
    const int32_t* n_new;
    uint16_t* q_out;
    uint8_t* k_pool;
    uint8_t* v_pool;
    int32_t* status;
    int64_t q_st, q_sh, qo_st, qo_sh, k_st, k_sh, v_st, v_sh, kp_sb, kp_sh, vp_sb, vp_sh;
    int64_t pool_tokens;
    int cap, hq, hk, d, half, max_pos, bs;
    int heads_per, groups;  // heads walked by one thread, and groups of them
    float k_inverse, v_inverse;   // of the pools' factors
};

// cos and sin of 8 neighbouring elements.
__device__ __forceinline__ void angles(const float* row, int half, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int u = 0; u < 8; u += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(row + u));
        const float4 y = __ldg(reinterpret_cast<const float4*>(row + half + u));
        c[u] = x.x, c[u + 1] = x.y, c[u + 2] = x.z, c[u + 3] = x.w;
        s[u] = y.x, s[u + 1] = y.y, s[u + 2] = y.z, s[u + 3] = y.w;
    }
}

// The largest magnitude, or NaN where one of them is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The codes (8 bytes) and scale of a group of 16 values.
__device__ __forceinline__ uint2 encode(const float (&x)[16], uint32_t* scale_byte) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) most = max_abs3(most, x[i], x[i + 1]);
    const uint32_t top = __float_as_uint(most);
    if (top >= 0x7f800000u) {   // an infinity or NaN among them
        *scale_byte = kFp4NoNumber;
        return make_uint2(0u, 0u);
    }
    // (at most 448, and at least the smallest scale: 2^-9, code 1)
    const uint32_t byte = max(fp8_pack(__fdiv_rn(__uint_as_float(top), 6.0f)), 1u);
    *scale_byte = byte;
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(fp8_unpack(byte))));
    const float r = __frcp_rn(s);
    auto over = [&](float y) {   // (the error negated: a zero keeps its sign)
        const float q = __fmul_rn(y, r);
        return __fmaf_rn(-__fmaf_rn(q, s, -y), r, q);
    };
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4] |= fp4_pack2(over(x[2 * i]), over(x[2 * i + 1])) << (8 * (i % 4));
    return make_uint2(w[0], w[1]);
}

// A group of a row to its record, its pool's factor taken out.
__device__ __forceinline__ void store_group(float (&x)[16], float inverse, uint8_t* rec, int d, int r, int group) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], inverse);
    uint32_t byte;
    const uint2 codes = encode(x, &byte);
    *reinterpret_cast<uint2*>(rec + r * (d / 2) + 8 * group) = codes;
    rec[fp4_codes(d) + r * (d / 16) + group] = static_cast<uint8_t>(byte);
}

// 8 elements of x and of their partners y: (x cos - y sin, y cos + x sin), each
// product and sum rounded.
__device__ __forceinline__ void turn8(const float* row, int half, float* x, float* y) {
    float c[8], s[8];
    angles(row, half, c, s);
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        const float a = x[v], b = y[v];
        x[v] = __fadd_rn(__fmul_rn(a, c[v]), __fmul_rn(-b, s[v]));
        y[v] = __fadd_rn(__fmul_rn(b, c[v]), __fmul_rn(a, s[v]));
    }
}

// 16 elements, as they are.
__device__ __forceinline__ void load16(const uint16_t* p, uint4* raw) {
#pragma unroll
    for (int u = 0; u < 2; ++u) raw[u] = __ldg(reinterpret_cast<const uint4*>(p) + u);
}

template <bool kBf16>
__device__ __forceinline__ void unpack16(const uint4* raw, float (&x)[16]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) unpack8<kBf16>(raw[u], *reinterpret_cast<float(*)[8]>(x + 8 * u));
}

// Which rows a launch takes. Many tokens go in two launches, queries and then keys and
// values: a thread of a query row needs 64 registers, one that encodes 80, and the
// queries' stream wants more warps than those leave room for (39,322 tokens of 16/4 heads of
// 128: one launch 103 us, two 96). Few tokens are one wave of blocks: they take the registers
// that spare them all spills (16 tokens of 8/2 heads of 256: 2.3 us, 2.5 with three blocks
// an SM; many tokens by two blocks: 97 us, by three 90, by 640 threads an SM 92).
enum Part { kAllRows, kQueryRows, kCacheRows };
constexpr int ctas_of(Part part) { return part == kQueryRows ? 4 : part == kCacheRows ? 3 : 2; }   // resident, of an SM

template <bool kBf16, Part kPart>
__global__ void __launch_bounds__(kThreads, ctas_of(kPart)) append_kv_fp4_kernel(const AppArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    int64_t n = a.cap;
    if (a.n_new) {
        const int64_t given = *a.n_new;
        n = given < 0 ? 0 : (given < n ? given : n);
    }
    // threads of a token: those of the queries, then of the keys, then of the values
    const int pairs = a.d / 16, halves = a.d / 32;
    const int of_q = kPart == kCacheRows ? 0 : pairs * a.groups, of_k = kPart == kQueryRows ? 0 : a.hk * halves;
    const int per_token = of_q + 2 * of_k;
    const int64_t total = n * per_token;
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; w < total;
         w += static_cast<int64_t>(gridDim.x) * kThreads) {
        // (keys and values of a token take other ways through the code: where they are many,
        // those of all tokens follow one another)
        const bool late = kPart == kCacheRows && w >= n * of_k;
        const int64_t v = late ? w - n * of_k : w;
        const int of_t = kPart == kCacheRows ? of_k : per_token;
        const int64_t t = total >> 32 ? v / of_t : static_cast<uint32_t>(v) / static_cast<uint32_t>(of_t);
        const int rest = static_cast<int>(v - t * of_t) + (late ? of_k : 0);
        const bool is_q = kPart != kCacheRows && rest < of_q;
        // a key's or value's 32 elements, under way before its slot and position are known
        const bool is_v = rest >= of_q + of_k;
        const int unit = rest - of_q - (is_v ? of_k : 0), g = unit / halves, j = unit - g * halves;
        const int half = is_v ? 0 : a.half, turned = half / kFp4Group;
        const bool whole = half % kFp4Group == 0;   // rotated groups have groups as partners
        const bool pair = whole && j < turned;
        const int g0 = !whole ? 2 * j : pair ? j : 2 * turned + 2 * (j - turned), g1 = pair ? j + turned : g0 + 1;
        const uint16_t* from = is_v ? a.v + t * a.v_st + g * a.v_sh : a.k + t * a.k_st + g * a.k_sh;
        uint4 raw[4] = {};
        if (kPart != kQueryRows && !is_q) {
            load16(from + 16 * g0, raw);
            load16(from + 16 * g1, raw + 2);
        }
        const float* row = nullptr;
        const int64_t slot = kPart == kQueryRows ? -1 : a.slot_map[t];
        const int64_t pos = a.half ? a.positions[t] : 0;
        if (slot >= a.pool_tokens && rest == 0) raise_status(a.status, SP_ERR_DEVICE);
        if (a.half) {
            if (pos < 0 || pos >= a.max_pos) {
                if (rest == 0) raise_status(a.status, SP_ERR_DEVICE);
                continue;
            }
            row = a.cos_sin + pos * 2 * a.half;
        }
        if (is_q) {
            // vectors (e0, e1) in elements: a rotated pair, or two neighbours behind it
            const int group = rest / pairs, i = rest - group * pairs;
            const bool turn = i < a.half / 8;
            const int e0 = turn ? i * 8 : 2 * a.half + (i - a.half / 8) * 16, e1 = turn ? e0 + a.half : e0 + 8;
            float c[8], s[8];
            if (turn) angles(row + e0, a.half, c, s);
            const int h0 = group * a.heads_per, h1 = min(h0 + a.heads_per, a.hq);
#pragma unroll 2
            for (int h = h0; h < h1; ++h) {
                const uint16_t* src = a.q + t * a.q_st + h * a.q_sh;
                uint16_t* dst = a.q_out + t * a.qo_st + h * a.qo_sh;
                uint4 x = __ldcs(reinterpret_cast<const uint4*>(src + e0));
                uint4 y = __ldcs(reinterpret_cast<const uint4*>(src + e1));
                if (turn) {
                    uint32_t* px = reinterpret_cast<uint32_t*>(&x);
                    uint32_t* py = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float2 f = unpack2<kBf16>(px[u]), g = unpack2<kBf16>(py[u]);
                        px[u] = pack2<kBf16>(f.x * c[2 * u] - g.x * s[2 * u], f.y * c[2 * u + 1] - g.y * s[2 * u + 1]);
                        py[u] = pack2<kBf16>(g.x * c[2 * u] + f.x * s[2 * u], g.y * c[2 * u + 1] + f.y * s[2 * u + 1]);
                    }
                }
                *reinterpret_cast<uint4*>(dst + e0) = x;
                *reinterpret_cast<uint4*>(dst + e1) = y;
            }
            continue;
        }
        if (kPart == kQueryRows || slot < 0 || slot >= a.pool_tokens) continue;
        const uint32_t at = static_cast<uint32_t>(slot), blk = at / static_cast<uint32_t>(a.bs);
        const int within = static_cast<int>(at - blk * a.bs), r = within % kFp4Rows;
        uint8_t* rec = (is_v ? a.v_pool + blk * a.vp_sb + g * a.vp_sh : a.k_pool + blk * a.kp_sb + g * a.kp_sh) +
                       static_cast<int64_t>(within / kFp4Rows) * fp4_record(a.d);
        const float inverse = is_v ? a.v_inverse : a.k_inverse;
        float x[16], y[16];
        unpack16<kBf16>(raw, x);
        unpack16<kBf16>(raw + 2, y);
        if (pair) {
#pragma unroll
            for (int u = 0; u < 2; ++u) turn8(row + 16 * g0 + 8 * u, half, x + 8 * u, y + 8 * u);
        } else if (!whole) {
#pragma unroll 1
            for (int u = 0; u < 4; ++u) {
                const int e = 32 * j + 8 * u;
                if (e >= 2 * half) break;
                const bool second = e >= half;
                const int k = second ? e - half : e;
                float o[8];
                unpack8<kBf16>(__ldg(reinterpret_cast<const uint4*>(from + (second ? k : e + half))), o);
                // (four places, so that the elements stay in registers)
                if (u == 0) second ? turn8(row + k, half, o, x) : turn8(row + k, half, x, o);
                if (u == 1) second ? turn8(row + k, half, o, x + 8) : turn8(row + k, half, x + 8, o);
                if (u == 2) second ? turn8(row + k, half, o, y) : turn8(row + k, half, y, o);
                if (u == 3) second ? turn8(row + k, half, o, y + 8) : turn8(row + k, half, y + 8, o);
            }
        }
        store_group(x, inverse, rec, a.d, r, g0);
        store_group(y, inverse, rec, a.d, r, g1);
    }
}

// ------------------------------------------------------------ read back

struct UnpackArgs {
    const uint8_t* pool;
    const int32_t* slots;
    uint16_t* out;
    int32_t* status;
    int64_t rows, sb, sh, o_st, o_sh, pool_tokens;
    int hk, d, bs;
    float scale;
};

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) unpack_fp4_kernel(const UnpackArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const int groups = a.d / 16, per_row = groups * a.hk;
    const int64_t total = a.rows * per_row;
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; w < total;
         w += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t t = total >> 32 ? w / per_row : static_cast<uint32_t>(w) / static_cast<uint32_t>(per_row);
        const int rest = static_cast<int>(w - t * per_row);
        const int h = rest / groups, i = rest - h * groups;
        const int64_t slot = a.slots ? a.slots[t] : t;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (slot >= 0 && slot < a.pool_tokens) {
            const uint32_t at = static_cast<uint32_t>(slot), blk = at / static_cast<uint32_t>(a.bs);
            const int within = static_cast<int>(at - blk * a.bs), r = within % kFp4Rows;
            const uint8_t* rec = a.pool + blk * a.sb + h * a.sh + static_cast<int64_t>(within / kFp4Rows) * fp4_record(a.d);
            const uint2 codes = __ldg(reinterpret_cast<const uint2*>(rec + r * (a.d / 2) + 8 * i));
            const uint32_t s = fp8_unpack(rec[fp4_codes(a.d) + r * groups + i] * 0x101u);
            uint32_t n[8], o[8];
            fp4_unpack(codes.x, *reinterpret_cast<uint32_t(*)[4]>(n));
            fp4_unpack(codes.y, *reinterpret_cast<uint32_t(*)[4]>(n + 4));
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float2 f = unpack2<false>(mul_f16x2(n[u], s));
                o[u] = pack2<kBf16>(f.x * a.scale, f.y * a.scale);
            }
            x = make_uint4(o[0], o[1], o[2], o[3]);
            y = make_uint4(o[4], o[5], o[6], o[7]);
        } else if (slot != -1 && rest == 0) {
            raise_status(a.status, SP_ERR_DEVICE);
        }
        uint4* dst = reinterpret_cast<uint4*>(a.out + t * a.o_st + h * a.o_sh + 16 * i);
        dst[0] = x;
        dst[1] = y;
    }
}

}  // namespace

cudaError_t launch_append_kv_fp4(const sp_append_fp4_shape* s, const uint16_t* q, const uint16_t* k,
                                 const uint16_t* v, const int32_t* slot_map, const int32_t* positions,
                                 const float* cos_sin, const int32_t* n_new, uint16_t* q_out, uint8_t* k_pool,
                                 uint8_t* v_pool, int32_t* status, cudaStream_t st) {
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
    a.kp_sb = s->kp_stride_block, a.kp_sh = s->kp_stride_head;
    a.vp_sb = s->vp_stride_block, a.vp_sh = s->vp_stride_head;
    a.pool_tokens = s->pool_blocks * s->block_size;
    a.cap = s->n_tokens;
    a.hq = q ? s->n_q_heads : 0;
    a.hk = s->n_kv_heads;
    a.d = s->head_dim;
    a.half = s->rotary_dim / 2;
    a.max_pos = s->max_pos;
    a.bs = s->block_size;
    a.k_inverse = 1.0f / s->k_scale;
    a.v_inverse = 1.0f / s->v_scale;
    const bool bf16 = s->dtype == SP_DTYPE_BF16;
    const int pairs = a.d / 16;
    const int64_t of_q = static_cast<int64_t>(a.cap) * pairs * a.hq, of_kv = static_cast<int64_t>(a.cap) * 2 * a.hk * (a.d / 32);
    const int sms = device_sms();
    auto launch = [&](Part part, int64_t work, void (*kern)(const AppArgs)) {
        const int64_t most = int64_t(ctas_of(part)) * sms, need = (work + kThreads - 1) / kThreads;
        return launch_k(kern, static_cast<unsigned>(need < most ? need : most), kThreads, 0, st, a);
    };
    // two heads a thread and two launches once either fills the GPU
    const bool many = of_q / 2 >= int64_t(kThreads) * ctas_of(kQueryRows) * sms;
    a.heads_per = many ? 2 : 1;
    a.groups = (a.hq + a.heads_per - 1) / a.heads_per;
    const int64_t units = static_cast<int64_t>(a.cap) * pairs * a.groups;
    if (!many)
        return launch(kAllRows, units + of_kv, bf16 ? append_kv_fp4_kernel<true, kAllRows> : append_kv_fp4_kernel<false, kAllRows>);
    const cudaError_t e = launch(kQueryRows, units, bf16 ? append_kv_fp4_kernel<true, kQueryRows> : append_kv_fp4_kernel<false, kQueryRows>);
    if (e != cudaSuccess) return e;
    return launch(kCacheRows, of_kv, bf16 ? append_kv_fp4_kernel<true, kCacheRows> : append_kv_fp4_kernel<false, kCacheRows>);
}

cudaError_t launch_unpack_fp4(const sp_unpack_fp4_shape* s, const uint8_t* pool, const int32_t* slots, uint16_t* out,
                              int32_t* status, cudaStream_t st) {
    UnpackArgs a;
    a.pool = pool;
    a.slots = slots;
    a.out = out;
    a.status = status;
    a.rows = s->n_rows;
    a.sb = s->stride_block, a.sh = s->stride_head;
    a.o_st = s->o_stride_token, a.o_sh = s->o_stride_head;
    a.pool_tokens = s->pool_blocks * s->block_size;
    a.hk = s->n_kv_heads;
    a.d = s->head_dim;
    a.bs = s->block_size;
    a.scale = s->scale;
    const int64_t work = a.rows * a.hk * (a.d / 16);
    int64_t grid = (work + kThreads - 1) / kThreads;
    const int64_t most = int64_t(8) * device_sms();
    if (grid > most) grid = most;
    auto kern = s->dtype == SP_DTYPE_BF16 ? unpack_fp4_kernel<true> : unpack_fp4_kernel<false>;
    return launch_k(kern, static_cast<unsigned>(grid), kThreads, 0, st, a);
}

}  // namespace sp
