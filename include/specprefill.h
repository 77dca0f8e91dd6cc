/*
 * specprefill.h — C ABI of the SpecPrefill token-importance and
 * chunk-selection path, hand-written CUDA for sm_103a (GB300).
 *
 * The path (pages: "SpecPrefill — Implementation Guide" of the
 * sliding-specprefill project, versions v2 and v3.1, and the llama.cpp pull
 * request "Speculative prefill"):
 *
 *   logits    s = scale * <q, k> for every lookahead query vector q of every
 *             attention layer and query head, against the prompt's cached
 *             keys k (GQA: query head h reads KV head h / (Hq/Hk))
 *   softmax   over the prompt's keys                    (guide §How It Works /
 *                                                        Attention Capture)
 *   importance  max over heads, max over layers, mean over lookahead steps
 *                                                       (guide §How It Works /
 *                                                        Token Importance)
 *   pool      centred average over W tokens (W = 13)    (PR §Approach item 3)
 *   normalise min-max to [0, 1] (optional)              (guide v3.1 item 5)
 *   boost     first 64 tokens x1.5, last 128 x1.3      (guide v3 item 2)
 *   chunks    mean score of 32-token chunks             (guide §Chunk Selection)
 *   select    top k = max(1, ceil(nc * p)) chunks, or the shortest ranked
 *             prefix holding `mass` of the total score  (guide v3 item 1)
 *   force     BOS and each prompt's final chunk         (PR §Approach item 4)
 *   gather    kept token indices + original position IDs (guide §How It
 *                                                        Works / Sparse Prefill)
 *
 * Conventions for every entry point
 * - Pointers marked (device) are device memory owned by the caller; the
 *   library never allocates, frees or retains them, and keeps no state
 *   between calls. Pointers marked (host) are host memory read during the
 *   call.
 * - Work is enqueued on `stream` and runs asynchronously; no entry point
 *   synchronises except sp_get_device_status.
 * - Return value: SP_OK, or an sp_status code for an argument the host can
 *   check (nothing is enqueued then) or a launch error. Faults the device
 *   detects itself (a bounded wait that gave up) set a sticky status word in
 *   the workspace, read with sp_get_device_status.
 * - Ranking ties break by ascending chunk index; the fixed mode keeps
 *   exactly k ranked chunks.
 * - Prompts are packed along the token axis: prompt b owns global tokens
 *   [seq_off[b], seq_off[b+1]). Chunks never cross prompts; prompt b owns
 *   chunks [chunk_off[b], chunk_off[b+1]), chunk_off[b+1]-chunk_off[b] =
 *   ceil(n_b / chunk).
 */
#ifndef SPECPREFILL_H
#define SPECPREFILL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same underlying type as cudaStream_t / cudaEvent_t. */
typedef struct CUstream_st* sp_stream_t;
typedef struct CUevent_st* sp_event_t;

typedef enum sp_status {
    SP_OK = 0,
    SP_ERR_INVALID_ARG = 1,   /* null pointer, inconsistent shape, parameter out of range */
    SP_ERR_UNSUPPORTED = 2,   /* head_dim not in {64,128,256}, L*G > 64, misaligned strides */
    SP_ERR_WORKSPACE = 3,     /* workspace null, misaligned (256 B) or smaller than required */
    SP_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed */
    SP_ERR_TIMEOUT = 5,       /* (device status) a bounded device wait gave up */
    SP_ERR_DEVICE = 6,        /* (device status) the kernel found an inconsistent input */
    SP_ERR_CAPACITY = 7       /* (device status) the free list holds too few blocks */
} sp_status;

enum { SP_MODE_FIXED = 0, SP_MODE_MASS = 1 };

/* Selection rule.
 * SP_RULE_EXACT: exactly k chunks in fixed mode (ties broken by ascending
 *   chunk index), token 0 and the final chunk forced (force_bos,
 *   force_last_chunk); the SpecPrefill scoring contract.
 * SP_RULE_LISTING: the rule of the pages' own tool ("SpecPrefill —
 *   Implementation Guide", v2 listing `select_chunks` and the cap in `main`):
 *   k = max(1, ceil(nc * p)) with the product rounded to float32, every
 *   chunk scoring at least the k-th largest score kept (ties can keep more
 *   than k), tokens {0, 1, 2, 3, n-2, n-1} forced (the last two when
 *   n > 4; force_bos and force_last_chunk are ignored), then a fill of the
 *   smallest unselected tokens up to eff_min = min(min_tok, max(4, n / 10))
 *   tokens, everything kept when p >= 1 (fixed mode) or n <= eff_min, and
 *   finally, when max_keep > 0 and more than max_keep tokens are kept, every
 *   step-th kept token (step = count / max_keep) up to max_keep of them with
 *   the last one replaced by the prompt's last kept token. Mass mode keeps
 *   its ranking prefix and then applies the forced tokens, the fill and the
 *   cap. Only sp_specprefill_score and sp_select_from_importance take this
 *   rule, and only with pool_w / 2 <= 64 and chunk dividing 128
 *   (SP_ERR_UNSUPPORTED otherwise). */
enum { SP_RULE_EXACT = 0, SP_RULE_LISTING = 1 };

/* Where the W-wide average pool applies (llama.cpp PR "Speculative
 * prefill", §Approach item 3, lists the smoothing together with the max over
 * heads and layers without fixing the order).
 * SP_POOL_TOKEN: on the per-token importance, after the mean over the
 *   lookahead steps (the scoring contract).
 * SP_POOL_HEAD: on every attention row (layer, step, query head) before the
 *   max over heads and layers; the later pooling step is then the identity
 *   (sp_pool_chunk and the fused call treat pool_w as 1 after it). Requires
 *   pool_w / 2 <= 64 (SP_ERR_UNSUPPORTED otherwise). */
enum { SP_POOL_TOKEN = 0, SP_POOL_HEAD = 1 };

/* Shapes and strides. Strides are in elements; the head_dim axis is
 * contiguous (stride 1).
 * K: bf16 keys of layer l, global token t, KV head g at
 *    k[l*k_stride_layer + t*k_stride_token + g*k_stride_head + j]
 *    (a token-major KV cache, e.g. [Ly][Ntot][Hk][d] contiguous).
 * Q: bf16 lookahead queries of prompt b, layer l, step s, query head h at
 *    q[b*q_stride_seq + l*q_stride_layer + s*q_stride_step + h*q_stride_head + j]
 *    (e.g. [B][Ly][L][Hq][d] contiguous).
 * Every stride times 2 bytes must be a multiple of 16 and both base
 * pointers 16-byte aligned (tensor-memory-accelerator tiles). */
typedef struct sp_shape {
    int32_t n_seqs;          /* B >= 1 prompts */
    int32_t n_layers;        /* Ly >= 1 attention layers */
    int32_t n_q_heads;       /* Hq >= 1 */
    int32_t n_kv_heads;      /* Hk >= 1, Hq % Hk == 0, G = Hq / Hk */
    int32_t head_dim;        /* d in {64, 128, 256} */
    int32_t n_lookahead;     /* L >= 1 query vectors per layer and head; L*G <= 64 */
    int32_t n_tokens_total;  /* Ntot = seq_off[B] >= 1 */
    int32_t max_seq_len;     /* 0 (no bound), or the longest prompt the caller
                                allows: a prompt with more tokens makes the
                                call's device status SP_ERR_DEVICE (checked on
                                the device with seq_off); < 0 is invalid */
    int64_t k_stride_layer, k_stride_token, k_stride_head;
    int64_t q_stride_seq, q_stride_layer, q_stride_step, q_stride_head;
} sp_shape;

typedef struct sp_params {
    int32_t pool_w;            /* odd, >= 1 (13); 1 = no smoothing */
    int32_t chunk;             /* C >= 1 (32) */
    int32_t mode;              /* SP_MODE_FIXED or SP_MODE_MASS */
    float keep_p;              /* fixed mode, in (0, 1] (0.30) */
    float mass;                /* mass mode, in (0, 1] (0.85) */
    int32_t normalize;         /* 1: min-max normalise each prompt's pooled scores */
    float boost_first_mult;    /* > 0 (1.5); 1 = off */
    int32_t boost_first_n;     /* >= 0 (64) */
    float boost_last_mult;     /* > 0 (1.3); 1 = off */
    int32_t boost_last_n;      /* >= 0 (128) */
    int32_t force_bos;         /* 1: token 0 of every prompt is kept */
    int32_t force_last_chunk;  /* 1: every prompt's final chunk is kept */
    float scale;               /* logit scale; 0 selects 1/sqrt(head_dim) */
    int32_t spin_limit;        /* polls before a device wait gives up; <= 0 selects the default */
    int32_t rule;              /* SP_RULE_EXACT (0) or SP_RULE_LISTING */
    int32_t min_tok;           /* SP_RULE_LISTING: >= 0 (128), bound of eff_min */
    int32_t max_keep;          /* SP_RULE_LISTING: >= 0 (2000 in the pages' tool); 0 = no cap */
    int32_t pool_at;           /* SP_POOL_TOKEN (0) or SP_POOL_HEAD */
    int32_t wave_mib;          /* >= 0; 0 selects the default (2048). The logits
                                  of all slabs are kept in the workspace between
                                  the two passes of the softmax; when they need
                                  more than this many MiB the slabs are scored in
                                  waves that each fit it (smaller workspace, one
                                  more pair of kernels per wave) */
} sp_params;

/* Optional profiling hook: when non-null, `logits_start`/`logits_stop` are
 * recorded on `stream` immediately around the logits kernel(s). */
typedef struct sp_profile {
    sp_event_t logits_start;
    sp_event_t logits_stop;
} sp_profile;

/* Number of kernels one sp_specprefill_score call with this shape and these
 * parameters launches on its stream (all of them this library's own), so a
 * caller can account for the launches it issues. */
int sp_kernels_per_call(const sp_shape* shape, const sp_params* params, int32_t* n_kernels);

/* Upper bound on the number of chunks of a packed batch:
 * floor(Ntot / chunk) + B. Chunk arrays must hold this many entries. */
int sp_max_chunks(const sp_shape* shape, const sp_params* params, int64_t* n_chunks);

/* Bytes of device workspace the entry points below need for this shape on
 * the current device (writes *bytes). */
int sp_workspace_size(const sp_shape* shape, const sp_params* params, size_t* bytes);

/* Zero the workspace's status word. Call once on a new workspace (or use
 * zero-filled memory) before the first call that uses it. */
int sp_workspace_init(void* ws, size_t ws_bytes, sp_stream_t stream);

/* Token importance (logits, softmax, max over heads and layers, mean over
 * steps): imp[t] for every global token t (device, Ntot floats).
 * Defined by "SpecPrefill — Implementation Guide", §How It Works / Attention
 * Capture (one post-softmax attention row per head and lookahead step over
 * the prompt's keys) and §How It Works / Token Importance (max over heads,
 * then max over layers, then the mean over the lookahead steps); the draft's
 * L lookahead queries and full-attention layers are those of llama.cpp PR
 * "Speculative prefill", §Approach items 1-2.
 * seq_off (device, B+1 int32, non-decreasing from 0 to Ntot), q and k
 * (device, bf16 bits) as described at sp_shape. */
int sp_attn_importance(const sp_shape* shape, const sp_params* params,
                       const int32_t* seq_off, const uint16_t* q, const uint16_t* k,
                       float* imp, void* ws, size_t ws_bytes, sp_stream_t stream);

/* Same contract as sp_attn_importance, but the logits come from a CUDA-core
 * (FP32 FMA) kernel instead of the tensor-core one. It exists as an
 * independent cross-check of the tensor-core kernel in the GPU tests. */
int sp_attn_importance_simt(const sp_shape* shape, const sp_params* params,
                            const int32_t* seq_off, const uint16_t* q, const uint16_t* k,
                            float* imp, void* ws, size_t ws_bytes, sp_stream_t stream);

/* Smoothing and chunk scores from imp (device, Ntot floats).
 * Defined by llama.cpp PR "Speculative prefill", §Approach item 3 (the
 * W-wide average pool), "SpecPrefill — Implementation Guide" v3.1, §v3.1
 * Optimizations item 5 (min-max normalisation), v3 §v3 Improvements item 2
 * (structural boost of the first and last tokens) and §Chunk Selection (a
 * chunk's score is the mean of its tokens' scores).
 * tok_score (device, Ntot floats, nullable): pooled score before
 * normalisation and boost. chunk_score (device, sp_max_chunks floats): the
 * final chunk scores. chunk_off (device, B+1 int32): written. */
int sp_pool_chunk(const sp_shape* shape, const sp_params* params, const int32_t* seq_off,
                  const float* imp, float* tok_score, float* chunk_score, int32_t* chunk_off,
                  void* ws, size_t ws_bytes, sp_stream_t stream);

/* Allocation-free variant of sp_pool_chunk (the pages have no counterpart;
 * this entry point exists for callers that cannot allocate device memory:
 * code running under a memory pool that owns all device memory and forbids
 * allocations after start-up, plugins whose host runtime gives them no
 * allocator, or loops that must not risk the device synchronisation a
 * cudaMalloc/cudaFree can cause). Same results as sp_pool_chunk, without a
 * workspace: its scratch lives in a fixed 1 MiB array inside the library on
 * every GPU that loads it, kept until the process exits. It calls no
 * allocation routine.
 * - tok_score, chunk_score (sp_max_chunks floats) and chunk_off (B+1) are
 *   required device outputs.
 * - status_out (device, one int32, nullable) receives this call's device
 *   status in stream order: SP_OK, or SP_ERR_DEVICE when seq_off is invalid.
 * - Batches whose scratch does not fit return SP_ERR_UNSUPPORTED before
 *   anything is enqueued. The scratch is a 256-byte header, four offset
 *   tables of 4*(B+1) bytes each (each rounded up to 256 bytes) and 8 bytes
 *   per pooling block of floor(1024 / chunk) * chunk tokens (one block per
 *   1024 tokens at chunk 32, plus one per prompt); it depends on B, Ntot and
 *   chunk only. At chunk 32 that admits, for example, 16,000 prompts of 1K
 *   tokens or one prompt of 100M tokens.
 * - Each call looks up the array's device address in the calling thread's
 *   current CUDA context (a new context after cudaDeviceReset, or another
 *   context on the same GPU, has its own copy of the array) unless the
 *   stream is being captured; a call made during stream capture reuses the
 *   address the last uncaptured call on that context found, so make one
 *   uncaptured call per context first.
 * - All calls on one GPU share the array and each leaves its contents
 *   behind: calls that overlap on the GPU (unordered streams or threads)
 *   race, so order them on one stream. */
int sp_pool_chunk_noalloc(const sp_shape* shape, const sp_params* params,
                          const int32_t* seq_off, const float* imp, float* tok_score,
                          float* chunk_score, int32_t* chunk_off, int32_t* status_out,
                          sp_stream_t stream);

/* Chunk selection per prompt, defined by "SpecPrefill — Implementation
 * Guide", §Chunk Selection (the top k = max(1, ceil(nc * p)) chunks by
 * score), v3 §v3 Improvements item 1 (cumulative attention mass: the
 * shortest ranked prefix holding `mass` of the total) and llama.cpp PR
 * "Speculative prefill", §Approach item 4 (BOS and the final chunk are always
 * kept). chunk_keep (device, one byte per chunk):
 * bit 0 = chosen by the ranking, bit 1 = forced final chunk.
 * SP_RULE_LISTING is not a chunk-level rule: SP_ERR_UNSUPPORTED (likewise
 * for sp_gather_kept). */
int sp_select(const sp_shape* shape, const sp_params* params, const int32_t* seq_off,
              const int32_t* chunk_off, const float* chunk_score, uint8_t* chunk_keep,
              void* ws, size_t ws_bytes, sp_stream_t stream);

/* Stream compaction of kept tokens, defined by "SpecPrefill —
 * Implementation Guide", §How It Works / Sparse Prefill (the target
 * prefills only the kept tokens, each at its original position ID). For
 * prompt b, its kept tokens (those
 * in a chunk with chunk_keep != 0, plus token 0 when force_bos) in
 * increasing order occupy [kept_off[b], kept_off[b+1]) of kept_idx (global
 * token index) and kept_pos (position within the prompt, i.e. the original
 * position ID). kept_idx/kept_pos: device, capacity Ntot int32 each;
 * kept_off: device, B+1 int32; n_kept: device, 1 int32 (= kept_off[B]). */
int sp_gather_kept(const sp_shape* shape, const sp_params* params, const int32_t* seq_off,
                   const int32_t* chunk_off, const uint8_t* chunk_keep, int32_t* kept_idx,
                   int32_t* kept_pos, int32_t* kept_off, int32_t* n_kept, void* ws,
                   size_t ws_bytes, sp_stream_t stream);

/* Sparse-prefill consumer: the rows of the kept tokens of a token-major
 * cache tensor ("SpecPrefill — Implementation Guide", §How It Works / Sparse
 * Prefill: the target prefills only the kept tokens, each at its original
 * position), so that keys or values built from the draft can be handed to
 * the target compactly.
 * - src (device, bf16 bits): [Ly][Ntot][Hk][d] with the k_stride_* strides
 *   of `shape` (d contiguous); only Ly, Ntot, Hk, d and those strides of
 *   `shape` are used.
 * - kept_idx (device, int32): packed token indices, e.g. from
 *   sp_specprefill_score; n_kept (device, one int32): how many of them to
 *   gather. Both are read on the device, so no host synchronisation is
 *   needed between the selection and this call.
 * - dst (device, bf16 bits): [Ly][dst_rows][Hk][d], dense; row i of layer l
 *   receives src[l][kept_idx[i]]. dst_rows must be at least Ntot (the
 *   largest possible kept count); rows past n_kept are left untouched.
 * - An index outside [0, Ntot) gives a zero row; n_kept is clamped to
 *   [0, Ntot].
 * Returns SP_ERR_INVALID_ARG for a bad shape, a null pointer, a pointer that
 * is not 16-byte aligned or dst_rows < Ntot. */
int sp_gather_rows(const sp_shape* shape, const int32_t* kept_idx, const int32_t* n_kept,
                   const uint16_t* src, uint16_t* dst, int64_t dst_rows, sp_stream_t stream);

/* Kept token ids for the target's batch (same section): out[i] =
 * token_ids[kept_idx[i]] for i < *n_kept (n_kept read on the device and
 * clamped to [0, n_tokens_total]); an index outside [0, n_tokens_total)
 * gives -1. token_ids holds the packed prompts' ids, n_tokens_total of them;
 * out must hold n_tokens_total entries. All pointers are device pointers.
 * Returns SP_ERR_INVALID_ARG for a null pointer or a bad size. */
int sp_gather_tokens(const int32_t* token_ids, int64_t n_tokens_total, const int32_t* kept_idx,
                     const int32_t* n_kept, int32_t* out, sp_stream_t stream);

/* Keys read in place from a draft engine's cache (in-situ scoring): one
 * key pool per layer, as draft engines allocate them, instead of one
 * [Ly][Ntot][Hk][d] tensor.
 * - layer_k: host array of n_layers (<= 64) device pointers, 16-byte
 *   aligned; pool row r, KV head g, element j of layer l at
 *   layer_k[l][r*k_stride_token + g*k_stride_head + j] (the shape's
 *   k_stride_token and k_stride_head; k_stride_layer is not used).
 * - block_table NULL: pool row = packed token index (seq_off[b] + t);
 *   pool_tokens >= n_tokens_total.
 * - block_table non-NULL (device, [n_seqs][table_stride] int32): a
 *   block-paged cache; token t of prompt b is pool row
 *   block_table[b*table_stride + t/block_size]*block_size + t%block_size.
 *   block_size is 8, 16, 32 or 64, or a multiple of 128; every prompt's
 *   blocks must fit in its table row (else the call's device status is
 *   SP_ERR_DEVICE and nothing is scored); a block id whose rows fall outside
 *   [0, pool_tokens) sets SP_ERR_DEVICE and reads pool row 0 instead.
 * - pool_tokens: rows of each layer's pool (num_blocks * block_size), at
 *   most 2^31 - 1. */
typedef struct sp_kv_source {
    const uint16_t* const* layer_k;
    const int32_t* block_table;
    int32_t block_size;
    int32_t table_stride;
    int64_t pool_tokens;
} sp_kv_source;

/* sp_attn_importance and sp_specprefill_score with the keys from `kv`
 * (the tensor-core path; same outputs, same workspace size for the same
 * shape). */
int sp_attn_importance_kv(const sp_shape* shape, const sp_params* params, const int32_t* seq_off,
                          const uint16_t* q, const sp_kv_source* kv, float* imp, void* ws,
                          size_t ws_bytes, sp_stream_t stream);
int sp_specprefill_score_kv(const sp_shape* shape, const sp_params* params,
                            const int32_t* seq_off, const uint16_t* q, const sp_kv_source* kv,
                            float* imp, float* tok_score, float* chunk_score, int32_t* chunk_off,
                            uint8_t* chunk_keep, int32_t* kept_idx, int32_t* kept_pos,
                            int32_t* kept_off, int32_t* n_kept, void* ws, size_t ws_bytes,
                            sp_stream_t stream);

/* Sliding-window scoring of the pages' tool ("SpecPrefill — Implementation
 * Guide", v3.1 §Sliding Window Loop and §Bug Fixes in v3.1): a prompt longer
 * than the draft's context is scored in windows of `window` tokens starting
 * every `stride` tokens, each window on its own (its own keys and lookahead
 * queries); window w contributes the scores of its first `stride` tokens,
 * the last window (the first one that reaches the end of the prompt) all of
 * its own, so every token is scored by exactly one window.
 *
 * sp_auto_window (host only): the guide's sizing for a draft context of
 * spec_ctx tokens (v2 listing `main`): a requested window <= 0 becomes
 * min(spec_ctx - 512, 500 MiB / (spec_ctx * 32)), the result is raised to
 * at least 512 and then lowered to at most spec_ctx - 128, and the stride is
 * half of it. SP_ERR_INVALID_ARG when spec_ctx < 130 (the window would be
 * below 2) or an output pointer is null.
 *
 * sp_window_plan (host only): the windows of a prompt of n tokens, in scoring
 * order: window w covers tokens [start[w], end[w]) and contributes its first
 * kept[w] scores. Writes *n_windows; the arrays (host, `capacity` entries
 * each, nullable when capacity is 0) receive min(capacity, *n_windows)
 * windows. SP_ERR_INVALID_ARG unless 1 <= stride <= window and n >= 0.
 *
 * sp_merge_windows (device): out[t] for t < n (device, n floats) from the
 * per-window importance vectors packed back to back in window order
 * (imp_windows, device, sum of the window lengths: every window but the
 * last has `window` tokens), i.e. out[t] = imp_windows[w * window + t -
 * w * stride] with w = min(t / stride, last window). Feed the window batch
 * to sp_attn_importance as a batch of prompts (one per window), merge, then
 * select with sp_select_from_importance. */
int sp_auto_window(int32_t spec_ctx, int32_t window_request, int32_t* window, int32_t* stride);
int sp_window_plan(int64_t n, int32_t window, int32_t stride, int32_t* start, int32_t* end,
                   int32_t* kept, int32_t capacity, int32_t* n_windows);
int sp_merge_windows(int64_t n, int32_t window, int32_t stride, const float* imp_windows,
                     float* out, sp_stream_t stream);

/* Pooling, normalisation, boost, chunk scores, selection and the kept
 * lists from a given per-token importance imp (device, Ntot floats): the
 * part of sp_specprefill_score after the importance, for importance that
 * comes from elsewhere (merged windows, another scorer). `shape` needs only
 * n_seqs and n_tokens_total to be meaningful (the attention dimensions must
 * still pass the checks; sp_workspace_size with the same shape gives the
 * workspace). Outputs as for sp_specprefill_score. */
int sp_select_from_importance(const sp_shape* shape, const sp_params* params,
                              const int32_t* seq_off, const float* imp, float* tok_score,
                              float* chunk_score, int32_t* chunk_off, uint8_t* chunk_keep,
                              int32_t* kept_idx, int32_t* kept_pos, int32_t* kept_off,
                              int32_t* n_kept, void* ws, size_t ws_bytes, sp_stream_t stream);

/* The whole path in one call: sp_attn_importance, sp_pool_chunk, sp_select
 * and sp_gather_kept in sequence, defined by the passages cited at each of
 * them ("SpecPrefill — Implementation Guide", §How It Works / Attention
 * Capture, Token Importance, Sparse Prefill, §Chunk Selection, v3 §v3
 * Improvements items 1-2, v3.1 §v3.1 Optimizations item 5; llama.cpp PR
 * "Speculative prefill", §Approach items 1-4). imp, tok_score, chunk_score, chunk_off and
 * chunk_keep are optional outputs (nullable; kept in the workspace when
 * null); kept_idx, kept_pos, kept_off and n_kept are required. `prof` is
 * optional (nullable). */
int sp_specprefill_score(const sp_shape* shape, const sp_params* params,
                         const int32_t* seq_off, const uint16_t* q, const uint16_t* k,
                         float* imp, float* tok_score, float* chunk_score, int32_t* chunk_off,
                         uint8_t* chunk_keep, int32_t* kept_idx, int32_t* kept_pos,
                         int32_t* kept_off, int32_t* n_kept, void* ws, size_t ws_bytes,
                         sp_stream_t stream, const sp_profile* prof);

/* ---------------------------------------------------------------------
 * Sparse prefill on a block-paged cache ("SpecPrefill — Implementation
 * Guide", §How It Works / Sparse Prefill: the target prefills only the kept
 * tokens, each at its original position ID, and then decodes). Three
 * operators carry a step of the target from the kept lists above:
 *
 *   sp_block_tables     cache blocks and slots for the step's new tokens,
 *                       from lengths that only the device knows (kept_off)
 *   sp_append_kv        queries and keys rotated to their original positions
 *                       (kept_pos), keys and values stored at those slots
 *   sp_paged_attention  attention of the new tokens over their requests'
 *                       cached tokens, the new ones included
 *
 * A cache layer is a key pool and a value pool of pool_tokens rows (blocks of
 * block_size rows) in the layout of sp_kv_source; block_table (device,
 * [n_seqs][table_stride] int32) maps logical block j of request b to pool
 * block block_table[b * table_stride + j]. The pages have no counterpart of
 * these operators; the paged layout is that of sp_kv_source.
 *
 * A request's cached tokens are its kept tokens in increasing original
 * position, so causality over cache indices is causality over positions.
 */
enum { SP_DTYPE_BF16 = 0, SP_DTYPE_F16 = 1 };

typedef struct sp_block_shape {
    int32_t n_seqs;        /* 1 <= B <= 16384 requests (SP_ERR_UNSUPPORTED above) */
    int32_t block_size;    /* >= 1 tokens of a block */
    int32_t table_stride;  /* >= 1 table entries of a request */
    int32_t n_tokens;      /* >= 0 entries of slot_map; the step's new tokens may be fewer */
    int32_t free_capacity; /* >= 0 entries of free_blocks */
    int32_t pool_blocks;   /* >= 1 blocks of the pool; pool_blocks * block_size <= 2^31 - 1 */
} sp_block_shape;

/* Block tables and slots of a step. Request b holds ctx_len[b] cached tokens
 * (in ceil(ctx_len[b] / block_size) blocks, the first entries of its table
 * row) and gets new_off[b+1] - new_off[b] new ones.
 * - ctx_len (device, B int32), new_off (device, B+1 int32, from 0, at most
 *   n_tokens; kept_off of the scoring call, or 0..B for a decode step).
 * - free_blocks (device, free_capacity int32), n_free (device, one int32):
 *   the free block ids are free_blocks[0, *n_free). Blocks are taken from
 *   the end, request by request and in order within a request, so
 *   free_blocks[0, *n_left) are the ones that stay free.
 * - block_table (device, in/out): the entries of the blocks taken are
 *   written, all others keep their values.
 * - slot_map (device, n_tokens int32): pool row of every new token, in
 *   order; -1 behind the last one.
 * - kv_len (device, B int32): ctx_len plus the new tokens.
 * - n_left (device, one int32): blocks that stay free.
 * - status (device, one int32, nullable): raised to SP_ERR_CAPACITY when
 *   n_free is too small, to SP_ERR_DEVICE when a length, an offset or n_free
 *   is out of range or a request outgrows its table row; the call then takes
 *   no block, leaves the table as it was, sets kv_len to 0 and every slot to
 *   -1. A block id outside [0, pool_blocks) also raises SP_ERR_DEVICE; the
 *   tokens of that block get slot -1. The word is never lowered: zero it
 *   before the first call.
 * A step that took nothing has to leave the lengths as they are: its kv_len is
 * no length of the cache, and as the next call's ctx_len it would have every
 * request begin anew over the blocks that it holds. Where steps are chained on
 * the device, let kv_len and n_left become ctx_len and n_free only where status
 * is still 0 (ctx_len and n_free themselves are inputs, so they hold what was
 * before the step, and the same step can be taken again). A block that a
 * request fills further belongs to it alone; full ones may be shared.
 * Nothing is allocated and no other memory is used, so a captured call can
 * be replayed. Outputs may not overlap inputs (block_table aside) or one
 * another: equal pointers are SP_ERR_INVALID_ARG, and so are pointers that
 * are not 4-byte aligned. */
int sp_block_tables(const sp_block_shape* shape, const int32_t* ctx_len, const int32_t* new_off,
                    const int32_t* free_blocks, const int32_t* n_free, int32_t* block_table,
                    int32_t* slot_map, int32_t* kv_len, int32_t* n_left, int32_t* status,
                    sp_stream_t stream);

/* Shapes and strides (in elements, head_dim contiguous) of sp_append_kv. */
typedef struct sp_append_shape {
    int32_t n_tokens;      /* >= 1 rows of q, k, v and slot_map */
    int32_t n_q_heads;     /* >= 1 with queries; ignored without */
    int32_t n_kv_heads;    /* >= 1; queries, keys and values have at most 65536 heads together */
    int32_t head_dim;      /* a multiple of 16, at most 1024 */
    int32_t rotary_dim;    /* 0 (no rotation) or a multiple of 16, at most head_dim */
    int32_t max_pos;       /* rows of cos_sin (ignored when rotary_dim is 0) */
    int32_t dtype;         /* SP_DTYPE_BF16 or SP_DTYPE_F16, of every tensor */
    int32_t reserved;      /* 0 */
    int64_t pool_tokens;   /* rows of each pool */
    int64_t q_stride_token, q_stride_head, qo_stride_token, qo_stride_head;
    int64_t k_stride_token, k_stride_head, v_stride_token, v_stride_head;
    int64_t kp_stride_token, kp_stride_head, vp_stride_token, vp_stride_head;
} sp_append_shape;

/* Rotation and cache store of the new tokens of one layer. Row t of q and k
 * is rotated to position positions[t] (rotate-half layout: elements j and
 * j + rotary_dim/2, j < rotary_dim/2, become a cos - b sin and b cos + a sin,
 * in 32 bits and rounded once; the others are copied); rotated queries go to
 * row t of q_out, rotated keys and the values to pool row slot_map[t].
 * - q, q_out (device, nullable together): [n_tokens][n_q_heads][head_dim];
 *   q_out may be q itself with the same strides.
 * - k, v (device): [n_tokens][n_kv_heads][head_dim]; k_pool, v_pool (device):
 *   [pool_tokens][n_kv_heads][head_dim].
 * - slot_map (device, n_tokens int32): -1 stores nothing (queries are still
 *   rotated). Slots of different rows must differ, as sp_block_tables makes
 *   them: a slot given twice holds a mixture of both rows.
 * - positions (device, n_tokens int32) and cos_sin (device, fp32,
 *   [max_pos][rotary_dim]: rotary_dim/2 cosines, then as many sines):
 *   required when rotary_dim > 0.
 * - n_new (device, one int32, nullable): the rows in use, clamped to
 *   [0, n_tokens]; rows behind are neither read nor written.
 * - status (device, one int32, nullable): raised to SP_ERR_DEVICE by a slot
 *   at or past pool_tokens (nothing is stored for the row) or a position
 *   outside [0, max_pos) (the row is skipped). Never lowered.
 * Outputs may not overlap inputs (q_out = q aside) or one another; equal
 * pointers are SP_ERR_INVALID_ARG. Base pointers of the 16-bit tensors and
 * cos_sin are 16-byte aligned, the others 4-byte aligned
 * (SP_ERR_INVALID_ARG), and strides multiples of 8 (SP_ERR_UNSUPPORTED). */
int sp_append_kv(const sp_append_shape* shape, const uint16_t* q, const uint16_t* k,
                 const uint16_t* v, const int32_t* slot_map, const int32_t* positions,
                 const float* cos_sin, const int32_t* n_new, uint16_t* q_out, uint16_t* k_pool,
                 uint16_t* v_pool, int32_t* status, sp_stream_t stream);

/* Shapes and strides (in elements, head_dim contiguous) of
 * sp_paged_attention. */
typedef struct sp_paged_shape {
    int32_t n_seqs;        /* 1 <= B <= 65536 requests */
    int32_t n_q_heads;     /* Hq <= 65536, Hq % Hk == 0, G = Hq / Hk <= 128 */
    int32_t n_kv_heads;    /* Hk >= 1 */
    int32_t head_dim;      /* d in {64, 128, 256} */
    int32_t dtype;         /* SP_DTYPE_BF16 or SP_DTYPE_F16: q, pools and out */
    int32_t block_size;    /* 8, 16, 32, 64 or a multiple of 128 */
    int32_t table_stride;  /* >= 1 table entries of a request */
    int32_t n_tokens;      /* 1 to 2^30 rows of q, out and lse; q_off[B] may be less */
    int64_t pool_tokens;   /* rows of each pool, at most 2^31 - 1 */
    int64_t q_stride_token, q_stride_head, o_stride_token, o_stride_head;
    int64_t k_stride_token, k_stride_head, v_stride_token, v_stride_head;
} sp_paged_shape;

typedef struct sp_attn_params {
    int32_t causal;        /* 1: a new token sees the cached tokens up to itself; 0: all of them */
    int32_t window;        /* with causal: > 0 sees only the last `window` of those; 0: all */
    float scale;           /* logit scale; 0 selects 1/sqrt(head_dim) */
    int32_t spin_limit;    /* polls before a device wait gives up; <= 0 selects the default */
} sp_attn_params;

/* Bytes of device workspace of sp_paged_attention for this shape on the
 * current device. The workspace is 256-byte aligned; prepare it once with
 * sp_workspace_init, read its status with sp_get_device_status. Calls that
 * share a workspace must be ordered (one stream, or events). */
int sp_paged_attention_workspace(const sp_paged_shape* shape, size_t* bytes);

/* Attention of new tokens over a block-paged cache: request b's new tokens
 * are rows [q_off[b], q_off[b+1]) of q, the last of its kv_len[b] cached
 * tokens (stored before this call). Row i of request b, at cache index
 * p = kv_len[b] - (q_off[b+1] - q_off[b]) + i, sees the cached tokens j with
 *   j <= p and (window == 0 or j > p - window)     when causal, else all,
 * and every query head h of it gives, over the tokens it sees,
 *   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale <q, k_j>,
 *   lse = m + log(sum_j exp(s_j - m)),                  m = max_j s_j,
 * with keys and values of KV head h / G. A row that sees no token (p < 0, or
 * a request without cached tokens) gives out = 0 and lse = -inf.
 * - q_off (device, B+1 int32, from 0, at most n_tokens): lengths from one
 *   token (a decode step) to a whole prompt, mixed in one call; 0 is allowed.
 * - kv_len (device, B int32): from sp_block_tables. It may be smaller than
 *   the number of new tokens (the first of them then see nothing).
 * - q (device): [n_tokens][Hq][d]; out (device): the same shape; lse (device,
 *   fp32 [n_tokens][Hq] dense, nullable). Rows at and behind q_off[B] are not
 *   written.
 * - Logits, softmax statistics and sums are held in 32 bits; the weights are
 *   rounded to the tensors' type for the product with the values.
 * - Cache rows at or behind kv_len[b], and rows that a query is masked from,
 *   may hold anything, infinities and NaN included: they do not reach its
 *   result. (Where a value of the new tokens, or at the edge of the window, is
 *   no number, the queries around it take a slow path: 0.1 s and more for a
 *   context of 40,000 tokens, in proportion to it; device waits do not run out
 *   meanwhile.) Table entries behind the request's last block are not read.
 * - A bad q_off or kv_len (out of range, over 2^30, or more tokens than a
 *   table row holds) sets the device status SP_ERR_DEVICE and nothing is computed; a
 *   block id outside the pool sets it and reads pool row 0 instead.
 * out and lse may not overlap the inputs or one another (equal pointers:
 * SP_ERR_INVALID_ARG). Strides times 2 bytes are multiples of 16
 * (SP_ERR_UNSUPPORTED otherwise); base pointers of the 16-bit tensors are
 * 16-byte aligned, the others 4-byte aligned (SP_ERR_INVALID_ARG otherwise). */
int sp_paged_attention(const sp_paged_shape* shape, const sp_attn_params* params,
                       const int32_t* q_off, const int32_t* kv_len, const int32_t* block_table,
                       const uint16_t* q, const uint16_t* k_pool, const uint16_t* v_pool,
                       uint16_t* out, float* lse, void* ws, size_t ws_bytes, sp_stream_t stream);

/* ------------------------------------------------------------------------
 * A cache in 4 bits
 *
 * The paged cache of the target's step ("SpecPrefill — Implementation Guide",
 * §How It Works / Sparse Prefill) held in 4.5 bits an element: a value is an
 * e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 or a negative of them) times an e4m3
 * scale shared by 16 neighbours of a row, times a factor that the caller gives
 * for the whole pool. Number times scale is exact in bf16 and fp16.
 *
 * A pool holds, for block b and KV head h, block_size / 8 records of 9 d / 2
 * bytes: 8 tokens' codes (d / 2 bytes each, element 2 i in the low and 2 i + 1 in
 * the high four bits of byte i; bit 3 of a code is the sign), then their scales
 * (d / 16 bytes each). The records of a block and head follow one another; blocks
 * and heads are `stride_block` and `stride_head` bytes apart, multiples of 16 below
 * 2^32 (SP_ERR_UNSUPPORTED).
 * head_dim is 64, 128 or 256, block_size 8, 16, 32, 64 or a multiple of 128. */

/* Shapes and strides of sp_append_kv_fp4 (16-bit tensors in elements, pools in
 * bytes). */
typedef struct sp_append_fp4_shape {
    int32_t n_tokens;      /* >= 1 rows of q, k, v and slot_map */
    int32_t n_q_heads;     /* >= 1 with queries; ignored without */
    int32_t n_kv_heads;    /* >= 1; queries, keys and values have at most 65536 heads together */
    int32_t head_dim;      /* 64, 128 or 256 */
    int32_t rotary_dim;    /* 0 (no rotation) or a multiple of 16, at most head_dim */
    int32_t max_pos;       /* rows of cos_sin (ignored when rotary_dim is 0) */
    int32_t dtype;         /* SP_DTYPE_BF16 or SP_DTYPE_F16, of q, k, v and q_out */
    int32_t block_size;
    int64_t pool_blocks;   /* blocks of each pool; pool_blocks * block_size < 2^31 */
    int64_t q_stride_token, q_stride_head, qo_stride_token, qo_stride_head;
    int64_t k_stride_token, k_stride_head, v_stride_token, v_stride_head;
    int64_t kp_stride_block, kp_stride_head, vp_stride_block, vp_stride_head;
    float k_scale, v_scale;  /* factors of the pools, from 2^-60 to 2^60 */
} sp_append_fp4_shape;

/* sp_append_kv into pools of 4 bits. Queries are rotated as there; a row x of
 * a rotated key (in 32 bits, not rounded before) or of a value is stored as
 *   y = x (1 / factor),   s_g = max(e4m3(min(max |y_g| / 6, 448)), 2^-9),
 *   code_i = e2m1(y_i / s_g)   for each group g of 16 neighbours,
 * every operation in 32 bits and rounded to nearest, e4m3() and e2m1() to the
 * nearest number with ties to even, e2m1 saturating at 6. A group that holds
 * an infinity or NaN gets the scale NaN, and reads back as NaN. The rest is as
 * for sp_append_kv: slot -1 stores nothing, slots of different rows must differ,
 * a bad slot or position raises SP_ERR_DEVICE in `status`, equal pointers and
 * misaligned ones are SP_ERR_INVALID_ARG, strides off 16 bytes
 * SP_ERR_UNSUPPORTED. */
int sp_append_kv_fp4(const sp_append_fp4_shape* shape, const uint16_t* q, const uint16_t* k,
                     const uint16_t* v, const int32_t* slot_map, const int32_t* positions,
                     const float* cos_sin, const int32_t* n_new, uint16_t* q_out, uint8_t* k_pool,
                     uint8_t* v_pool, int32_t* status, sp_stream_t stream);

typedef struct sp_unpack_fp4_shape {
    int32_t n_kv_heads;    /* >= 1, at most 65536 */
    int32_t head_dim;      /* 64, 128 or 256 */
    int32_t block_size;
    int32_t dtype;         /* of out */
    int64_t pool_blocks;
    int64_t stride_block, stride_head;          /* of the pool, in bytes */
    int64_t n_rows;        /* rows of out */
    int64_t o_stride_token, o_stride_head;      /* of out, in elements */
    float scale;           /* factor of the pool, finite */
    int32_t reserved;      /* 0 */
} sp_unpack_fp4_shape;

/* Rows of a 4-bit pool as 16-bit values (number * scale * factor in 32 bits,
 * rounded once; without a rounding when factor is a power of two and nothing
 * leaves the type's range). Row r of out is the pool's row slots[r]
 * (device, int32), or row r itself when slots is null (n_rows is then
 * pool_blocks * block_size). A slot of -1 gives zeros; one outside the pool
 * raises SP_ERR_DEVICE in `status` (device, one int32, nullable) and gives
 * zeros too. The values are what sp_attn_importance_kv, sp_paged_attention and
 * the gathers take as a 16-bit cache. */
int sp_unpack_fp4(const sp_unpack_fp4_shape* shape, const uint8_t* pool, const int32_t* slots,
                  uint16_t* out, int32_t* status, sp_stream_t stream);

/* Shapes and strides of sp_paged_attention_fp4 (q and out in elements, pools
 * in bytes). */
typedef struct sp_fp4_shape {
    int32_t n_seqs;        /* 1 <= B <= 65536 requests */
    int32_t n_q_heads;     /* Hq <= 65536, Hq % Hk == 0, G = Hq / Hk <= 128 */
    int32_t n_kv_heads;    /* Hk >= 1 */
    int32_t head_dim;      /* d in {64, 128, 256} */
    int32_t dtype;         /* SP_DTYPE_BF16 or SP_DTYPE_F16: q and out */
    int32_t block_size;    /* 8, 16, 32, 64 or a multiple of 128 */
    int32_t table_stride;  /* >= 1 table entries of a request */
    int32_t n_tokens;      /* 1 to 2^30 rows of q, out and lse; n_tokens * Hq < 2^31 */
    int32_t max_new;       /* most new tokens of a request, at most n_tokens; 0: n_tokens */
    int32_t reserved;      /* 0 */
    int64_t dense_tokens;  /* cached tokens that requests with many new ones may have together to be
                              read through 16 bits (below); 0: none */
    int64_t pool_blocks;   /* blocks of each pool; pool_blocks * block_size < 2^31 */
    int64_t q_stride_token, q_stride_head, o_stride_token, o_stride_head;
    int64_t k_stride_block, k_stride_head, v_stride_block, v_stride_head;
} sp_fp4_shape;

typedef struct sp_fp4_params {
    int32_t causal;        /* as in sp_attn_params */
    int32_t window;
    float scale;           /* logit scale; 0 selects 1/sqrt(head_dim). scale * k_scale lies between
                              2^-126 and 2^126 */
    float k_scale;         /* factors of the pools, from 2^-60 to 2^60 */
    float v_scale;
    int32_t spin_limit;    /* polls before a device wait gives up; <= 0 selects the default */
} sp_fp4_params;

/* Bytes of device workspace of sp_paged_attention_fp4 for this shape on the
 * current device (prepared and read as that of sp_paged_attention). It holds
 * 4 * Hk * head_dim bytes for each of dense_tokens. */
int sp_paged_attention_fp4_workspace(const sp_fp4_shape* shape, size_t* bytes);

/* sp_paged_attention over 4-bit pools: the same rows, masks, outputs and error
 * behaviour, with s_j = scale k_scale <q, k_j> and out = v_scale sum p v / sum p.
 * Logits, statistics and sums are held in 32 bits; weights are rounded to fp16
 * (scaled so that the largest is 2^6 to 2^14) for the product with the values. bf16 queries are
 * scaled by a power of two for each row and head and taken as fp16, which is
 * exact for elements down to 2^-31 of the row's largest.
 * Requests whose new tokens make many rows are computed over a 16-bit copy of
 * their cached tokens, in the workspace, as long as those of all such requests
 * of the call fit into dense_tokens (in the requests' order: from the first that does not
 * fit on, none is copied); the others, all decode steps, and calls that n_tokens and the
 * table's rows bound to little work are computed from the 4-bit rows. The same call gives
 * the same bits. A request's last bits may change with the requests beside it and with
 * the table's width, which decide where its context is cut and which way a chunk goes. A request with more new
 * tokens than max_new sets SP_ERR_DEVICE, and nothing is computed.
 * Cached rows that a query is masked from may hold anything, scales that are
 * NaN included; table entries of blocks that no row sees (behind the request's end,
 * before the first row's window) are not read. */
int sp_paged_attention_fp4(const sp_fp4_shape* shape, const sp_fp4_params* params,
                           const int32_t* q_off, const int32_t* kv_len, const int32_t* block_table,
                           const uint16_t* q, const uint8_t* k_pool, const uint8_t* v_pool,
                           uint16_t* out, float* lse, void* ws, size_t ws_bytes, sp_stream_t stream);

/* ------------------------------------------------------------------------
 * Pages of the cache
 *
 * A block may belong to several requests. `shared` (device, int32 [pool_blocks])
 * counts its holders beyond the first: 0 for a block of one request and for a
 * free one, so that blocks that sp_block_tables takes need no entry. */

typedef struct sp_copy_shape {
    int32_t n_pools;       /* 1 to SP_MAX_COPY_POOLS pools of one shape */
    int32_t n_entries;     /* entries of src and dst */
    int32_t rows;          /* consecutive slots of an entry: 1, or block_size */
    int32_t block_size;
    int32_t n_kv_heads;
    int32_t head_dim;      /* 16-bit pools: a multiple of 8; 4-bit pools: 64, 128 or 256 */
    int32_t fp4;           /* 0: 16-bit pools [blocks][block_size][Hk][d]; 1: 4-bit pools */
    int32_t n_seqs;        /* with block_table: its rows */
    int32_t table_stride;  /* with block_table: entries of a row */
    int32_t reserved;      /* 0 */
    int64_t pool_blocks;
    int64_t stride_block, stride_token, stride_head;   /* of every pool, in bytes (4-bit: no token stride) */
} sp_copy_shape;

#define SP_MAX_COPY_POOLS 256

/* Copies rows of the cache in every pool (keys and values of all layers).
 * Entry i copies the `rows` slots from src[i] * rows on to those from dst[i] * rows on:
 * single tokens, or whole blocks (the copies that sp_fork_blocks asks for). With
 * block_table and src_off (int32 [n_seqs + 1], from 0, non-decreasing; rows = 1),
 * entry i of request b, src_off[b] <= i < src_off[b + 1], copies the request's cached
 * token src[i], which lies in block block_table[b][src[i] / block_size]: with a
 * scoring call's kept_pos and kept_off, and slots that sp_block_tables gave for
 * new rows of the table, this moves the kept tokens of cached prompts to blocks
 * of their own.
 * - src, dst (device, n_entries int32): an entry with a negative src or dst
 *   copies nothing. The slots written differ from one another and from all that are
 *   read.
 * - n_used (device, one int32, nullable): the entries in use, clamped to
 *   [0, n_entries] (and to src_off[n_seqs] with block_table).
 * - status (device, one int32, nullable): raised to SP_ERR_DEVICE by a slot, a
 *   token or a block id out of range; that entry copies nothing.
 * - pools (host array of n_pools device pointers), 16-byte aligned. */
int sp_copy_kv(const sp_copy_shape* shape, void* const* pools, const int32_t* src, const int32_t* dst,
               const int32_t* block_table, const int32_t* src_off, const int32_t* n_used,
               int32_t* status, sp_stream_t stream);

typedef struct sp_pages_shape {
    int32_t n_seqs;        /* 1 <= B <= 16384 rows of the table */
    int32_t n_forks;       /* sp_fork_blocks: entries of src and dst, 1 to 16384 */
    int32_t block_size;    /* >= 1 */
    int32_t table_stride;  /* >= 1 entries of a table row */
    int32_t pool_blocks;   /* entries of shared; pool_blocks * block_size < 2^31 */
    int32_t free_capacity; /* entries of free_blocks */
    int32_t alone;         /* sp_free_blocks: 1 refuses cuts inside a block that others hold (below), 0 makes them;
                              sp_fork_blocks: 0 */
} sp_pages_shape;

/* Forks requests: row dst[i] of the table becomes a request with the cached
 * tokens of row src[i]. Its full blocks are src's own, each with one holder more;
 * a begun last block is taken anew, from the end of the free list, in the order
 * of i, and left to be copied: copy_src[i] and copy_dst[i] name the blocks (-1
 * where there is none), as sp_copy_kv takes them with rows = block_size.
 * - src, dst (device, n_forks int32): src[i] < 0 forks nothing. The rows dst of
 *   the others differ from one another and from all of src, and hold nothing
 *   (ctx_len 0).
 * - ctx_len (device, B int32): cached tokens of every row; kv_len (device, B
 *   int32, written): the same after the forks.
 * - block_table (device, int32 [B][table_stride]), shared (device, int32
 *   [pool_blocks]): written in place.
 * - free_blocks, n_free, n_left: as in sp_block_tables.
 * - status (device, one int32, nullable): raised to SP_ERR_CAPACITY when the free
 *   list is too short, to SP_ERR_DEVICE when an entry, a length or n_free is out of
 *   range or a dst breaks the rule above. The call then forks nothing: table and
 *   counts stay, kv_len is ctx_len, n_left is n_free and all copies are -1. A block
 *   id outside [0, pool_blocks) also raises SP_ERR_DEVICE, and is counted nowhere.
 * Outputs may not be inputs or one another (SP_ERR_INVALID_ARG). */
int sp_fork_blocks(const sp_pages_shape* shape, const int32_t* src, const int32_t* dst,
                   const int32_t* ctx_len, int32_t* block_table, int32_t* shared,
                   const int32_t* free_blocks, const int32_t* n_free, int32_t* kv_len,
                   int32_t* copy_src, int32_t* copy_dst, int32_t* n_left, int32_t* status,
                   sp_stream_t stream);

/* Cuts every request from ctx_len[b] to new_len[b] <= ctx_len[b] cached tokens
 * (0: the request ends) and lets go of the blocks behind them: a block's count of
 * holders goes down by the requests that let it go, and the blocks that nobody
 * holds any more are put behind the n_free free ones, in increasing order of
 * their ids, whatever the order of the requests.
 * - ctx_len, new_len (device, B int32); kv_len (device, B int32, written): new_len.
 * - block_table (device, int32 [B][table_stride]): read only; entries behind a
 *   request's last block count for nothing afterwards.
 * - shared, free_blocks (device): written in place; n_left (device, one int32,
 *   written): the blocks that are free after the call.
 * - status (device, one int32, nullable): raised to SP_ERR_DEVICE when a length or
 *   n_free is out of range, or a block is let go more often than it is held (as
 *   far as `shared`, whose entries are 0 or more, shows it); to SP_ERR_CAPACITY when
 *   free_blocks is too short. The call then frees nothing: counts and list stay,
 *   kv_len is ctx_len, n_left is n_free. A block id outside [0, pool_blocks) also
 *   raises SP_ERR_DEVICE, and is counted nowhere.
 * A cut may end inside a block that other requests hold as well (a request and its fork
 * share a block until both have let it go). A request cut like that may be read, cut further
 * and forked, but not filled further: sp_block_tables takes a begun block for the
 * request's own, and its next tokens would overwrite those of the others. To go on with it, fork it
 * into an empty row, which gets the begun block as a copy of its own, and free the row that was cut. With
 * alone = 1 such a cut counts as a length out of range: SP_ERR_DEVICE, and the call frees
 * nothing.
 * Outputs may not be inputs or one another (SP_ERR_INVALID_ARG). */
int sp_free_blocks(const sp_pages_shape* shape, const int32_t* ctx_len, const int32_t* new_len,
                   const int32_t* block_table, int32_t* shared, int32_t* free_blocks,
                   const int32_t* n_free, int32_t* kv_len, int32_t* n_left, int32_t* status,
                   sp_stream_t stream);

/* Synchronise `stream`, then read (and, when `clear` is non-zero, reset)
 * the workspace's sticky device status word into *status_host. */
int sp_get_device_status(void* ws, size_t ws_bytes, sp_stream_t stream, int clear,
                         int32_t* status_host);

/* Static description of a status code. */
const char* sp_status_string(int status);

/* Library build identification (architecture and kernel variant). */
const char* sp_build_info(void);

#ifdef __cplusplus
}
#endif

#endif /* SPECPREFILL_H */
