// Internal declarations of the 4-bit cache and of the page operators:
// launchers of sp_fp4_cache.cu, sp_fp4_attn.cu and sp_pages.cu, called by
// sp_fp4_api.cu after its checks.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "specprefill.h"

namespace sp {

constexpr int kMaxForks = 16384;   // forks whose scan fits a CTA's shared memory

cudaError_t launch_append_kv_fp4(const sp_append_fp4_shape* s, const uint16_t* q, const uint16_t* k,
                                 const uint16_t* v, const int32_t* slot_map, const int32_t* positions,
                                 const float* cos_sin, const int32_t* n_new, uint16_t* q_out, uint8_t* k_pool,
                                 uint8_t* v_pool, int32_t* status, cudaStream_t st);

cudaError_t launch_unpack_fp4(const sp_unpack_fp4_shape* s, const uint8_t* pool, const int32_t* slots, uint16_t* out,
                              int32_t* status, cudaStream_t st);

// Bytes of workspace of the attention (header included).
size_t attn_fp4_workspace(const sp_fp4_shape* s);

cudaError_t launch_paged_attention_fp4(const sp_fp4_shape* s, const sp_fp4_params* p, const int32_t* q_off,
                                       const int32_t* kv_len, const int32_t* table, const uint16_t* q,
                                       const uint8_t* k_pool, const uint8_t* v_pool, uint16_t* out, float* lse,
                                       void* ws, cudaStream_t st);

cudaError_t launch_copy_kv(const sp_copy_shape* s, void* const* pools, const int32_t* src, const int32_t* dst,
                           const int32_t* block_table, const int32_t* src_off, const int32_t* n_entries,
                           int32_t* status, cudaStream_t st);

cudaError_t launch_fork_blocks(const sp_pages_shape* s, const int32_t* src, const int32_t* dst,
                               const int32_t* ctx_len, int32_t* table, int32_t* shared, const int32_t* free_blocks,
                               const int32_t* n_free, int32_t* kv_len, int32_t* copy_src, int32_t* copy_dst,
                               int32_t* n_left, int32_t* status, cudaStream_t st);

cudaError_t launch_free_blocks(const sp_pages_shape* s, const int32_t* ctx_len, const int32_t* new_len,
                               const int32_t* table, int32_t* shared, int32_t* free_blocks, const int32_t* n_free,
                               int32_t* kv_len, int32_t* n_left, int32_t* status, cudaStream_t st);

}  // namespace sp
