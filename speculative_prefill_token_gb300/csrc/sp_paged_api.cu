// C ABI of the paged-cache operators: argument checks of the entry points
// sp_block_tables, sp_append_kv and sp_paged_attention of specprefill.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "sp_internal.h"
#include "sp_paged.h"
#include "specprefill.h"

namespace sp {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

using Pointers = std::initializer_list<const void*>;

// Whether all of them (null or not) are aligned to their 32-bit entries.
bool words(Pointers all) {
    for (const void* p : all)
        if (!aligned(p, 4)) return false;
    return true;
}

// Whether an output is one of the inputs, or another output.
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

// (extent, stride) of one axis of bf16/fp16 rows of `width` elements: a
// stride counts only where the axis has more than one entry.
int check_stride(int64_t extent, int64_t stride, int64_t width) {
    if (extent <= 1) return SP_OK;
    if (stride < width) return SP_ERR_INVALID_ARG;
    return stride % 8 == 0 ? SP_OK : SP_ERR_UNSUPPORTED;
}

int check_paged(const sp_paged_shape* s) {
    if (!s) return SP_ERR_INVALID_ARG;
    if (s->n_seqs < 1 || s->n_q_heads < 1 || s->n_kv_heads < 1 || s->table_stride < 1 || s->n_tokens < 1 ||
        s->block_size < 1 || s->pool_tokens < 1 || s->pool_tokens > INT32_MAX)
        return SP_ERR_INVALID_ARG;
    if (s->n_q_heads % s->n_kv_heads != 0) return SP_ERR_INVALID_ARG;
    if (s->dtype != SP_DTYPE_BF16 && s->dtype != SP_DTYPE_F16) return SP_ERR_INVALID_ARG;
    if (s->head_dim != 64 && s->head_dim != 128 && s->head_dim != 256) return SP_ERR_UNSUPPORTED;
    if (s->n_seqs > kMaxSeqs || s->n_q_heads / s->n_kv_heads > 128 || s->n_q_heads > kMaxHeads ||
        s->n_tokens > kMaxCached)
        return SP_ERR_UNSUPPORTED;
    const int bs = s->block_size;
    if (!(bs == 8 || bs == 16 || bs == 32 || bs == 64 || bs % 128 == 0)) return SP_ERR_UNSUPPORTED;
    if (s->pool_tokens < bs) return SP_ERR_INVALID_ARG;
    const int64_t st[8] = {s->q_stride_token, s->o_stride_token, s->k_stride_token, s->v_stride_token,
                           s->q_stride_head,  s->o_stride_head,  s->k_stride_head,  s->v_stride_head};
    const int64_t ext[8] = {s->n_tokens,  s->n_tokens,  s->pool_tokens, s->pool_tokens,
                            s->n_q_heads, s->n_q_heads, s->n_kv_heads,  s->n_kv_heads};
    for (int i = 0; i < 8; ++i) {
        const int rc = check_stride(ext[i], st[i], s->head_dim);
        if (rc != SP_OK) return rc;
    }
    return SP_OK;
}

}  // namespace
}  // namespace sp

using namespace sp;

extern "C" {

int sp_block_tables(const sp_block_shape* s, const int32_t* ctx_len, const int32_t* new_off,
                    const int32_t* free_blocks, const int32_t* n_free, int32_t* block_table,
                    int32_t* slot_map, int32_t* kv_len, int32_t* n_left, int32_t* status,
                    sp_stream_t stream) {
    if (!s || !ctx_len || !new_off || !n_free || !block_table || !kv_len || !n_left) return SP_ERR_INVALID_ARG;
    if (s->n_seqs < 1 || s->block_size < 1 || s->table_stride < 1 || s->n_tokens < 0 || s->free_capacity < 0 ||
        s->pool_blocks < 1 || static_cast<int64_t>(s->pool_blocks) * s->block_size > INT32_MAX)
        return SP_ERR_INVALID_ARG;
    if ((s->n_tokens > 0 && !slot_map) || (s->free_capacity > 0 && !free_blocks)) return SP_ERR_INVALID_ARG;
    if (s->n_seqs > kMaxTableSeqs) return SP_ERR_UNSUPPORTED;
    if (!words({ctx_len, new_off, free_blocks, n_free, block_table, slot_map, kv_len, n_left, status}) ||
        shared({block_table, slot_map, kv_len, n_left, status}, {ctx_len, new_off, free_blocks, n_free}))
        return SP_ERR_INVALID_ARG;
    return to_status(launch_block_tables(s, ctx_len, new_off, free_blocks, n_free, block_table, slot_map, kv_len,
                                         n_left, status, reinterpret_cast<cudaStream_t>(stream)));
}

int sp_append_kv(const sp_append_shape* s, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                 const int32_t* slot_map, const int32_t* positions, const float* cos_sin,
                 const int32_t* n_new, uint16_t* q_out, uint16_t* k_pool, uint16_t* v_pool,
                 int32_t* status, sp_stream_t stream) {
    if (!s || !k || !v || !slot_map || !k_pool || !v_pool || (q != nullptr) != (q_out != nullptr))
        return SP_ERR_INVALID_ARG;
    if (s->n_tokens < 1 || s->n_kv_heads < 1 || s->head_dim < 1 || (q && s->n_q_heads < 1) ||
        s->rotary_dim < 0 || s->rotary_dim > s->head_dim || s->pool_tokens < 1 || s->pool_tokens > INT32_MAX ||
        s->reserved != 0)
        return SP_ERR_INVALID_ARG;
    if (s->dtype != SP_DTYPE_BF16 && s->dtype != SP_DTYPE_F16) return SP_ERR_INVALID_ARG;
    if (s->head_dim % 16 != 0 || s->head_dim > 1024 || s->rotary_dim % 16 != 0) return SP_ERR_UNSUPPORTED;
    if (s->rotary_dim > 0 && (!positions || !cos_sin || s->max_pos < 1)) return SP_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_pool, 16) ||
        !aligned(v_pool, 16) || (s->rotary_dim > 0 && !aligned(cos_sin, 16)))
        return SP_ERR_INVALID_ARG;
    if ((q ? static_cast<int64_t>(s->n_q_heads) : 0) + 2 * static_cast<int64_t>(s->n_kv_heads) > kMaxHeads)
        return SP_ERR_UNSUPPORTED;
    if (!words({slot_map, positions, n_new, status}) ||
        shared({k_pool, v_pool, q_out, status}, {k, v, slot_map, positions, cos_sin, n_new}) ||
        shared({k_pool, v_pool, status}, {q}))
        return SP_ERR_INVALID_ARG;
    if (q && q_out == q &&
        ((s->n_tokens > 1 && s->qo_stride_token != s->q_stride_token) ||
         (s->n_q_heads > 1 && s->qo_stride_head != s->q_stride_head)))
        return SP_ERR_INVALID_ARG;
    const int64_t hq = q ? s->n_q_heads : 1;
    const int64_t ext[12] = {q ? s->n_tokens : 1, hq, q ? s->n_tokens : 1, hq, s->n_tokens, s->n_kv_heads,
                             s->n_tokens, s->n_kv_heads, s->pool_tokens, s->n_kv_heads, s->pool_tokens,
                             s->n_kv_heads};
    const int64_t st[12] = {s->q_stride_token, s->q_stride_head, s->qo_stride_token, s->qo_stride_head,
                            s->k_stride_token, s->k_stride_head, s->v_stride_token, s->v_stride_head,
                            s->kp_stride_token, s->kp_stride_head, s->vp_stride_token, s->vp_stride_head};
    for (int i = 0; i < 12; ++i) {
        const int rc = check_stride(ext[i], st[i], s->head_dim);
        if (rc != SP_OK) return rc;
    }
    return to_status(launch_append_kv(s, q, k, v, slot_map, positions, cos_sin, n_new, q_out, k_pool, v_pool, status,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

int sp_paged_attention_workspace(const sp_paged_shape* shape, size_t* bytes) {
    const int rc = check_paged(shape);
    if (rc != SP_OK) return rc;
    if (!bytes) return SP_ERR_INVALID_ARG;
    *bytes = attn_workspace(shape);
    return SP_OK;
}

int sp_paged_attention(const sp_paged_shape* shape, const sp_attn_params* params, const int32_t* q_off,
                       const int32_t* kv_len, const int32_t* block_table, const uint16_t* q,
                       const uint16_t* k_pool, const uint16_t* v_pool, uint16_t* out, float* lse,
                       void* ws, size_t ws_bytes, sp_stream_t stream) {
    const int rc = check_paged(shape);
    if (rc != SP_OK) return rc;
    if (!params || !q_off || !kv_len || !block_table || !q || !k_pool || !v_pool || !out) return SP_ERR_INVALID_ARG;
    if ((params->causal != 0 && params->causal != 1) || params->window < 0 ||
        (params->window > 0 && !params->causal) || !(std::isfinite(params->scale) && params->scale >= 0.0f))
        return SP_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(out, 16) ||
        !words({q_off, kv_len, block_table, lse}) ||
        shared({out, lse}, {q_off, kv_len, block_table, q, k_pool, v_pool, ws}))
        return SP_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 256) || ws_bytes < attn_workspace(shape)) return SP_ERR_WORKSPACE;
    return to_status(launch_paged_attention(shape, params, q_off, kv_len, block_table, q, k_pool, v_pool, out, lse,
                                            ws, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
