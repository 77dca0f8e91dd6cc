// C ABI of the 4-bit cache and of the page operators: argument checks of
// sp_append_kv_fp4, sp_unpack_fp4, sp_paged_attention_fp4, sp_copy_kv,
// sp_fork_blocks and sp_free_blocks of specprefill.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "sp_fp4.cuh"
#include "sp_fp4.h"
#include "sp_internal.h"
#include "sp_paged.h"
#include "specprefill.h"

namespace sp {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

using Pointers = std::initializer_list<const void*>;

bool all_aligned(Pointers all, uintptr_t n) {
    for (const void* p : all)
        if (!aligned(p, n)) return false;
    return true;
}

// Whether an output is one of the inputs, or another output (null ones aside).
bool shared(Pointers outs, Pointers ins) {
    for (const void* const* o = outs.begin(); o != outs.end(); ++o) {
        if (!*o) continue;
        for (const void* i : ins)
            if (i == *o) return true;
        for (const void* const* other = outs.begin(); other != o; ++other)
            if (*other == *o) return true;
    }
    return false;
}

int to_status(cudaError_t e) { return e == cudaSuccess ? SP_OK : SP_ERR_CUDA; }

bool fp4_head_dim(int d) { return d == 64 || d == 128 || d == 256; }
bool fp4_block_size(int bs) { return bs == 8 || bs == 16 || bs == 32 || bs == 64 || (bs > 0 && bs % 128 == 0); }
// (a NaN is in no range)
bool factor(float f) { return f >= 0x1p-60f && f <= 0x1p60f; }
bool is_type(int dtype) { return dtype == SP_DTYPE_BF16 || dtype == SP_DTYPE_F16; }

// An axis whose entries are at least `width` apart, in steps of `step`: a stride
// counts only where the axis has more than one entry.
int check_stride(int64_t extent, int64_t stride, int64_t width, int64_t step) {
    if (extent <= 1) return SP_OK;
    if (stride < width) return SP_ERR_INVALID_ARG;
    return stride % step == 0 ? SP_OK : SP_ERR_UNSUPPORTED;
}

// Blocks and heads of a 4-bit pool, in either order.
int check_pool(int64_t blocks, int hk, int bs, int d, int64_t sb, int64_t sh) {
    const int64_t page = static_cast<int64_t>(bs) / kFp4Rows * fp4_record(d);
    int rc = check_stride(blocks, sb, page, 16);
    if (rc == SP_OK) rc = check_stride(hk, sh, page, 16);
    if (rc == SP_OK && ((blocks > 1 && sb > UINT32_MAX) || (hk > 1 && sh > UINT32_MAX))) rc = SP_ERR_UNSUPPORTED;
    return rc;
}

int check_fp4(const sp_fp4_shape* s) {
    if (!s) return SP_ERR_INVALID_ARG;
    if (s->n_seqs < 1 || s->n_q_heads < 1 || s->n_kv_heads < 1 || s->table_stride < 1 || s->n_tokens < 1 ||
        s->block_size < 1 || s->pool_blocks < 1 || s->max_new < 0 || s->max_new > s->n_tokens || s->reserved != 0 ||
        s->dense_tokens < 0 || !is_type(s->dtype) || s->n_q_heads % s->n_kv_heads != 0)
        return SP_ERR_INVALID_ARG;
    if (!fp4_head_dim(s->head_dim) || !fp4_block_size(s->block_size)) return SP_ERR_UNSUPPORTED;
    if (s->pool_blocks > INT32_MAX / s->block_size) return SP_ERR_INVALID_ARG;
    if (s->n_seqs > kMaxSeqs || s->n_q_heads / s->n_kv_heads > 128 || s->n_q_heads > kMaxHeads ||
        s->n_tokens > kMaxCached || static_cast<int64_t>(s->n_tokens) * s->n_q_heads > INT32_MAX ||
        s->dense_tokens > kMaxCached)
        return SP_ERR_UNSUPPORTED;
    const int d = s->head_dim;
    int rc = check_stride(s->n_tokens, s->q_stride_token, d, 8);
    if (rc == SP_OK) rc = check_stride(s->n_q_heads, s->q_stride_head, d, 8);
    if (rc == SP_OK) rc = check_stride(s->n_tokens, s->o_stride_token, d, 8);
    if (rc == SP_OK) rc = check_stride(s->n_q_heads, s->o_stride_head, d, 8);
    if (rc == SP_OK) rc = check_pool(s->pool_blocks, s->n_kv_heads, s->block_size, d, s->k_stride_block, s->k_stride_head);
    if (rc == SP_OK) rc = check_pool(s->pool_blocks, s->n_kv_heads, s->block_size, d, s->v_stride_block, s->v_stride_head);
    return rc;
}

int check_pages(const sp_pages_shape* s) {
    if (!s) return SP_ERR_INVALID_ARG;
    if (s->n_seqs < 1 || s->block_size < 1 || s->table_stride < 1 || s->pool_blocks < 1 || s->free_capacity < 0 ||
        (s->alone != 0 && s->alone != 1) || static_cast<int64_t>(s->pool_blocks) * s->block_size > INT32_MAX)
        return SP_ERR_INVALID_ARG;
    return s->n_seqs > kMaxTableSeqs ? SP_ERR_UNSUPPORTED : SP_OK;
}

}  // namespace
}  // namespace sp

using namespace sp;

extern "C" {

int sp_append_kv_fp4(const sp_append_fp4_shape* s, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                     const int32_t* slot_map, const int32_t* positions, const float* cos_sin, const int32_t* n_new,
                     uint16_t* q_out, uint8_t* k_pool, uint8_t* v_pool, int32_t* status, sp_stream_t stream) {
    if (!s || !k || !v || !slot_map || !k_pool || !v_pool || (q != nullptr) != (q_out != nullptr))
        return SP_ERR_INVALID_ARG;
    if (s->n_tokens < 1 || s->n_kv_heads < 1 || s->head_dim < 1 || (q && s->n_q_heads < 1) || s->rotary_dim < 0 ||
        s->rotary_dim > s->head_dim || s->pool_blocks < 1 || s->block_size < 1 || !factor(s->k_scale) ||
        !factor(s->v_scale) || !is_type(s->dtype))
        return SP_ERR_INVALID_ARG;
    if (!fp4_head_dim(s->head_dim) || !fp4_block_size(s->block_size) || s->rotary_dim % 16 != 0)
        return SP_ERR_UNSUPPORTED;
    if (s->pool_blocks > INT32_MAX / s->block_size) return SP_ERR_INVALID_ARG;
    if (s->rotary_dim > 0 && (!positions || !cos_sin || s->max_pos < 1)) return SP_ERR_INVALID_ARG;
    if ((q ? static_cast<int64_t>(s->n_q_heads) : 0) + 2 * static_cast<int64_t>(s->n_kv_heads) > kMaxHeads)
        return SP_ERR_UNSUPPORTED;
    if (!all_aligned({q, q_out, k, v, k_pool, v_pool}, 16) || (s->rotary_dim > 0 && !aligned(cos_sin, 16)) ||
        !all_aligned({slot_map, positions, n_new, status}, 4) ||
        shared({k_pool, v_pool, q_out, status}, {k, v, slot_map, positions, cos_sin, n_new}) ||
        shared({k_pool, v_pool, status}, {q}))
        return SP_ERR_INVALID_ARG;
    if (q && q_out == q &&
        ((s->n_tokens > 1 && s->qo_stride_token != s->q_stride_token) ||
         (s->n_q_heads > 1 && s->qo_stride_head != s->q_stride_head)))
        return SP_ERR_INVALID_ARG;
    const int d = s->head_dim;
    const int64_t tq = q ? s->n_tokens : 1, hq = q ? s->n_q_heads : 1;
    const int64_t ext[8] = {tq, hq, tq, hq, s->n_tokens, s->n_kv_heads, s->n_tokens, s->n_kv_heads};
    const int64_t st[8] = {s->q_stride_token, s->q_stride_head, s->qo_stride_token, s->qo_stride_head,
                           s->k_stride_token, s->k_stride_head, s->v_stride_token, s->v_stride_head};
    for (int i = 0; i < 8; ++i) {
        const int rc = check_stride(ext[i], st[i], d, 8);
        if (rc != SP_OK) return rc;
    }
    int rc = check_pool(s->pool_blocks, s->n_kv_heads, s->block_size, d, s->kp_stride_block, s->kp_stride_head);
    if (rc == SP_OK) rc = check_pool(s->pool_blocks, s->n_kv_heads, s->block_size, d, s->vp_stride_block, s->vp_stride_head);
    if (rc != SP_OK) return rc;
    return to_status(launch_append_kv_fp4(s, q, k, v, slot_map, positions, cos_sin, n_new, q_out, k_pool, v_pool,
                                          status, reinterpret_cast<cudaStream_t>(stream)));
}

int sp_unpack_fp4(const sp_unpack_fp4_shape* s, const uint8_t* pool, const int32_t* slots, uint16_t* out,
                  int32_t* status, sp_stream_t stream) {
    if (!s || !pool || !out || s->n_rows < 1 || s->n_kv_heads < 1 || s->pool_blocks < 1 || s->block_size < 1 ||
        s->reserved != 0 || !is_type(s->dtype) || !std::isfinite(s->scale))
        return SP_ERR_INVALID_ARG;
    if (!fp4_head_dim(s->head_dim) || !fp4_block_size(s->block_size) || s->n_kv_heads > kMaxHeads)
        return SP_ERR_UNSUPPORTED;
    if (s->pool_blocks > INT32_MAX / s->block_size || (!slots && s->n_rows != s->pool_blocks * s->block_size))
        return SP_ERR_INVALID_ARG;
    if (!all_aligned({pool, out}, 16) || !all_aligned({slots, status}, 4) || shared({out, status}, {pool, slots}))
        return SP_ERR_INVALID_ARG;
    int rc = check_stride(s->n_rows, s->o_stride_token, s->head_dim, 8);
    if (rc == SP_OK) rc = check_stride(s->n_kv_heads, s->o_stride_head, s->head_dim, 8);
    if (rc == SP_OK) rc = check_pool(s->pool_blocks, s->n_kv_heads, s->block_size, s->head_dim, s->stride_block, s->stride_head);
    if (rc != SP_OK) return rc;
    return to_status(launch_unpack_fp4(s, pool, slots, out, status, reinterpret_cast<cudaStream_t>(stream)));
}

int sp_paged_attention_fp4_workspace(const sp_fp4_shape* shape, size_t* bytes) {
    const int rc = check_fp4(shape);
    if (rc != SP_OK) return rc;
    if (!bytes) return SP_ERR_INVALID_ARG;
    *bytes = attn_fp4_workspace(shape);
    return SP_OK;
}

int sp_paged_attention_fp4(const sp_fp4_shape* shape, const sp_fp4_params* params, const int32_t* q_off,
                           const int32_t* kv_len, const int32_t* block_table, const uint16_t* q,
                           const uint8_t* k_pool, const uint8_t* v_pool, uint16_t* out, float* lse, void* ws,
                           size_t ws_bytes, sp_stream_t stream) {
    const int rc = check_fp4(shape);
    if (rc != SP_OK) return rc;
    if (!params || !q_off || !kv_len || !block_table || !q || !k_pool || !v_pool || !out) return SP_ERR_INVALID_ARG;
    if ((params->causal != 0 && params->causal != 1) || params->window < 0 ||
        (params->window > 0 && !params->causal) || !(std::isfinite(params->scale) && params->scale >= 0.0f) ||
        !factor(params->k_scale) || !factor(params->v_scale))
        return SP_ERR_INVALID_ARG;
    const double logit = params->scale * static_cast<double>(params->k_scale);
    if (params->scale > 0.0f && (logit < 0x1p-126 || logit > 0x1p126)) return SP_ERR_INVALID_ARG;
    if (!all_aligned({q, k_pool, v_pool, out}, 16) || !all_aligned({q_off, kv_len, block_table, lse}, 4) ||
        shared({out, lse}, {q_off, kv_len, block_table, q, k_pool, v_pool, ws}))
        return SP_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 256) || ws_bytes < attn_fp4_workspace(shape)) return SP_ERR_WORKSPACE;
    return to_status(launch_paged_attention_fp4(shape, params, q_off, kv_len, block_table, q, k_pool, v_pool, out,
                                                lse, ws, reinterpret_cast<cudaStream_t>(stream)));
}

int sp_copy_kv(const sp_copy_shape* s, void* const* pools, const int32_t* src, const int32_t* dst,
               const int32_t* block_table, const int32_t* src_off, const int32_t* n_used, int32_t* status,
               sp_stream_t stream) {
    if (!s || !pools || !src || !dst || (block_table != nullptr) != (src_off != nullptr)) return SP_ERR_INVALID_ARG;
    if (s->n_pools < 1 || s->n_entries < 1 || s->block_size < 1 || s->n_kv_heads < 1 || s->head_dim < 1 ||
        s->pool_blocks < 1 || s->reserved != 0 || (s->fp4 != 0 && s->fp4 != 1) ||
        (s->rows != 1 && s->rows != s->block_size) ||
        (block_table && (s->rows != 1 || s->n_seqs < 1 || s->table_stride < 1)))
        return SP_ERR_INVALID_ARG;
    if (s->n_pools > SP_MAX_COPY_POOLS || s->n_kv_heads > kMaxHeads ||
        (s->fp4 ? !fp4_head_dim(s->head_dim) || !fp4_block_size(s->block_size)
                : s->head_dim % 8 != 0 || s->head_dim > 1024))
        return SP_ERR_UNSUPPORTED;
    if (s->pool_blocks > INT32_MAX / s->block_size) return SP_ERR_INVALID_ARG;
    int rc;
    if (s->fp4) {
        rc = check_pool(s->pool_blocks, s->n_kv_heads, s->block_size, s->head_dim, s->stride_block, s->stride_head);
    } else {
        rc = check_stride(s->pool_blocks, s->stride_block, 2 * s->head_dim, 16);
        if (rc == SP_OK) rc = check_stride(s->block_size, s->stride_token, 2 * s->head_dim, 16);
        if (rc == SP_OK) rc = check_stride(s->n_kv_heads, s->stride_head, 2 * s->head_dim, 16);
    }
    if (rc != SP_OK) return rc;
    if (!all_aligned({src, dst, block_table, src_off, n_used, status}, 4) ||
        shared({status}, {src, dst, block_table, src_off, n_used}))
        return SP_ERR_INVALID_ARG;
    for (int i = 0; i < s->n_pools; ++i) {
        if (!pools[i] || !aligned(pools[i], 16) || shared({pools[i]}, {src, dst, block_table, src_off, n_used, status}))
            return SP_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (pools[j] == pools[i]) return SP_ERR_INVALID_ARG;
    }
    return to_status(launch_copy_kv(s, pools, src, dst, block_table, src_off, n_used, status,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

int sp_fork_blocks(const sp_pages_shape* s, const int32_t* src, const int32_t* dst, const int32_t* ctx_len,
                   int32_t* block_table, int32_t* shared_count, const int32_t* free_blocks, const int32_t* n_free,
                   int32_t* kv_len, int32_t* copy_src, int32_t* copy_dst, int32_t* n_left, int32_t* status,
                   sp_stream_t stream) {
    const int rc = check_pages(s);
    if (rc != SP_OK) return rc;
    if (s->n_forks < 1 || s->alone != 0 || !src || !dst || !ctx_len || !block_table || !shared_count || !n_free || !kv_len ||
        !copy_src || !copy_dst || !n_left || (s->free_capacity > 0 && !free_blocks))
        return SP_ERR_INVALID_ARG;
    if (s->n_forks > kMaxForks) return SP_ERR_UNSUPPORTED;
    if (!all_aligned({src, dst, ctx_len, block_table, shared_count, free_blocks, n_free, kv_len, copy_src, copy_dst,
                      n_left, status}, 4) ||
        shared({block_table, shared_count, kv_len, copy_src, copy_dst, n_left, status},
               {src, dst, ctx_len, free_blocks, n_free}))
        return SP_ERR_INVALID_ARG;
    return to_status(launch_fork_blocks(s, src, dst, ctx_len, block_table, shared_count, free_blocks, n_free, kv_len,
                                        copy_src, copy_dst, n_left, status, reinterpret_cast<cudaStream_t>(stream)));
}

int sp_free_blocks(const sp_pages_shape* s, const int32_t* ctx_len, const int32_t* new_len,
                   const int32_t* block_table, int32_t* shared_count, int32_t* free_blocks, const int32_t* n_free,
                   int32_t* kv_len, int32_t* n_left, int32_t* status, sp_stream_t stream) {
    const int rc = check_pages(s);
    if (rc != SP_OK) return rc;
    if (!ctx_len || !new_len || !block_table || !shared_count || !n_free || !kv_len || !n_left ||
        (s->free_capacity > 0 && !free_blocks))
        return SP_ERR_INVALID_ARG;
    if (!all_aligned({ctx_len, new_len, block_table, shared_count, free_blocks, n_free, kv_len, n_left, status}, 4) ||
        shared({shared_count, free_blocks, kv_len, n_left, status}, {ctx_len, new_len, block_table, n_free}))
        return SP_ERR_INVALID_ARG;
    return to_status(launch_free_blocks(s, ctx_len, new_len, block_table, shared_count, free_blocks, n_free, kv_len,
                                        n_left, status, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
