// Internal declarations of the paged-cache operators: launchers of
// sp_cache.cu and sp_attn.cu, called by sp_paged_api.cu after its checks.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "specprefill.h"

namespace sp {

constexpr int kMaxCached = 1 << 30;   // cached tokens of a request, and new tokens of an attention call
constexpr int kMaxHeads = 1 << 16;    // heads of all kinds that one call walks
constexpr int kMaxTableSeqs = 16384;  // requests whose scan fits a CTA's shared memory

// Multiprocessors of the current device.
inline int device_sms() {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms > 0 ? sms : 1;
}

cudaError_t launch_block_tables(const sp_block_shape* s, const int32_t* ctx_len, const int32_t* new_off,
                                const int32_t* free_blocks, const int32_t* n_free, int32_t* table,
                                int32_t* slot_map, int32_t* kv_len, int32_t* n_left, int32_t* status,
                                cudaStream_t st);

cudaError_t launch_append_kv(const sp_append_shape* s, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                             const int32_t* slot_map, const int32_t* positions, const float* cos_sin,
                             const int32_t* n_new, uint16_t* q_out, uint16_t* k_pool, uint16_t* v_pool,
                             int32_t* status, cudaStream_t st);

// Bytes of workspace of the attention (header included).
size_t attn_workspace(const sp_paged_shape* s);

cudaError_t launch_paged_attention(const sp_paged_shape* s, const sp_attn_params* p, const int32_t* q_off,
                                   const int32_t* kv_len, const int32_t* table, const uint16_t* q,
                                   const uint16_t* k_pool, const uint16_t* v_pool, uint16_t* out, float* lse,
                                   void* ws, cudaStream_t st);

}  // namespace sp
