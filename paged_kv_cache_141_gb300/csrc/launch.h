// launch.h -- host-side interface between the C ABI (api.cu) and the kernel
// translation units. Arguments have been validated by the caller.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pagedkv.h"

namespace pagedkv {

struct DecodeParams {
    void* out;                    // single pass: [S, Hq, D] of the query type
    const void* query;            // [S, Hq, D]
    const void* k_cache;          // [num_blocks, Hkv, B, D]
    const void* v_cache;
    const int32_t* block_tables;  // [S, max_blocks]
    const int32_t* context_lens;  // [S]
    float* tmp_out;               // split: [S, Hq, max_parts, D]
    float* max_logits;            // split: [S, Hq, max_parts]
    float* exp_sums;              // split: [S, Hq, max_parts]
    uint32_t* status;             // may be null
    int64_t num_blocks;
    int max_blocks;
    int num_seqs;
    int num_q_heads;
    int num_kv_heads;
    int block_size;
    int max_context_len;
    int partition_size;           // split only
    int max_parts;                // split only
    int group;                    // Hq / Hkv
    int sub_groups;               // group / heads per work unit
    float q_mul;                  // scale * log2(e) * (E4M3 cache ? k_scale : 1)
    float v_mul;                  // E4M3 cache ? v_scale : 1
    // fused KV write (all null for a plain decode): each sequence's newest
    // key/value [S, Hkv, D] of the query type, stored at new_slots[s]
    const void* new_key;
    const void* new_value;
    const int64_t* new_slots;
    void* wk_cache;               // the caches, writable (same addresses as k_cache / v_cache)
    void* wv_cache;
    float k_scale_w;              // E4M3 quantisation scales of the write
    float v_scale_w;
    // multi-query attention on the CUDA cores (null for the decode): the
    // rows of query/out are query tokens; token t of sequence s (query_start[s]
    // <= t < query_start[s+1]) attends to the first L_s - Q_s + (t -
    // query_start[s]) + 1 keys. Single pass only, no fused write.
    const int32_t* query_start;   // [S + 1]
    int num_queries;              // rows of query / out
    int max_queries;              // max over s of Q_s (sizes the tensor-core multi-query grid)
    const int32_t* seq_order;     // null or [S]: launch position -> sequence (longest first)
    // shared-prefix partitions (tensor-core decode, split only; all null / 0
    // otherwise): skip_parts[s] leading partitions of sequence s are computed
    // by the CTAs of the unit holding s (grid z < num_units, in the same
    // launch), whose members are unit_seqs[u * 4 .. u * 4 + 3] (-1 = none)
    // sharing unit_parts[u] partitions
    const int32_t* skip_parts;    // [S]
    const int32_t* unit_seqs;     // [num_units, 4]
    const int32_t* unit_parts;    // [num_units]
    int num_units;
    bool nan_codes;               // E4M3's NaN codes are read as NaN by the tensor cores too
};

// Generic CUDA-core decode; one launcher per (query type, cache type).
// head_size in {64, 128, 256}; heads_per_unit in {1, 2, 4, 8}.
cudaError_t launch_decode_simt_f32(const DecodeParams& p, int head_size, int heads_per_unit,
                                   bool split, cudaStream_t stream);
cudaError_t launch_decode_simt_f16(const DecodeParams& p, int head_size, int heads_per_unit,
                                   bool split, cudaStream_t stream);
cudaError_t launch_decode_simt_bf16(const DecodeParams& p, int head_size, int heads_per_unit,
                                    bool split, cudaStream_t stream);
cudaError_t launch_decode_simt_f16_e4m3(const DecodeParams& p, int head_size, int heads_per_unit,
                                        bool split, cudaStream_t stream);
cudaError_t launch_decode_simt_bf16_e4m3(const DecodeParams& p, int head_size,
                                         int heads_per_unit, bool split, cudaStream_t stream);

// Tensor-TMA decode (rows of 128/256/512 bytes, block size 8, 16 or a
// multiple of 32); heads_per_unit <= 32 / (head_size / 32).
cudaError_t launch_decode_tma_f32(const DecodeParams& p, int head_size, int heads_per_unit,
                                  bool split, cudaStream_t stream);
cudaError_t launch_decode_tma_f16(const DecodeParams& p, int head_size, int heads_per_unit,
                                  bool split, cudaStream_t stream);
cudaError_t launch_decode_tma_bf16(const DecodeParams& p, int head_size, int heads_per_unit,
                                   bool split, cudaStream_t stream);
cudaError_t launch_decode_tma_f16_e4m3(const DecodeParams& p, int head_size, int heads_per_unit,
                                       bool split, cudaStream_t stream);
cudaError_t launch_decode_tma_bf16_e4m3(const DecodeParams& p, int head_size, int heads_per_unit,
                                        bool split, cudaStream_t stream);

// Tensor-core decode for 16-bit caches (query type = cache type), TMA-eligible
// shapes, heads_per_unit in {1, 2, 4, 8}.
cudaError_t launch_decode_mma_f16(const DecodeParams& p, int head_size, int heads_per_unit,
                                  bool split, cudaStream_t stream);
cudaError_t launch_decode_mma_bf16(const DecodeParams& p, int head_size, int heads_per_unit,
                                   bool split, cudaStream_t stream);
// E4M3 caches (rows of 128 or 256 bytes) with a 16-bit query, MMAs in f16.
cudaError_t launch_decode_mma_f16_e4m3(const DecodeParams& p, int head_size, int heads_per_unit,
                                       bool split, cudaStream_t stream);
cudaError_t launch_decode_mma_bf16_e4m3(const DecodeParams& p, int head_size, int heads_per_unit,
                                        bool split, cudaStream_t stream);
// Multi-query paged attention for a few query rows per (sequence, KV head)
// (max_queries * group <= 32 at head_size <= 128, <= 16 at 256) on
// warp-level MMA: 16-bit query with a cache of
// the same type (head_size 64/128/256) or E4M3 (128/256), TMA-eligible shapes.
// Uses the multi-query fields of DecodeParams; single pass.
cudaError_t launch_prefill_mma_f16(const DecodeParams& p, int head_size, cudaStream_t stream);
cudaError_t launch_prefill_mma_bf16(const DecodeParams& p, int head_size, cudaStream_t stream);
cudaError_t launch_prefill_mma_f16_e4m3(const DecodeParams& p, int head_size, cudaStream_t stream);
cudaError_t launch_prefill_mma_bf16_e4m3(const DecodeParams& p, int head_size, cudaStream_t stream);

// Multi-query paged attention on the tensor cores (tcgen05): 16-bit query and
// cache of the same type (head_size in {64, 128, 256}) or E4M3 (64, 128),
// block size a power of two in [8, 256], group <= 128.
struct PrefillParams {
    void* out;                    // [T, Hq, D], query type
    const void* query;            // [T, Hq, D]
    const int32_t* query_start;   // [S + 1]
    const void* k_cache;          // [num_blocks, Hkv, B, D]
    const void* v_cache;
    const int32_t* block_tables;  // [S, max_blocks]
    const int32_t* context_lens;  // [S]
    uint32_t* status;             // may be null
    int64_t num_blocks;
    int max_blocks;
    int num_seqs;
    int num_q_heads;
    int num_kv_heads;
    int block_size;
    int group;                    // Hq / Hkv
    int max_context_len;
    int max_queries;              // max over s of Q_s (sizes the grid)
    int tokens_per_tile;          // floor(128 / G)
    int q_tiles;                  // ceil(max_queries / tokens_per_tile)
    float q_mul;                  // scale * log2(e) * (E4M3 cache ? k_scale : 1)
    float v_mul;                  // E4M3 cache ? v_scale : 1
    const int32_t* seq_order;     // null or [S]: launch position -> sequence (longest first)
};

cudaError_t launch_prefill_tc_f16(const PrefillParams& p, int head_size, cudaStream_t stream);
cudaError_t launch_prefill_tc_bf16(const PrefillParams& p, int head_size, cudaStream_t stream);
// E4M3 caches with a 16-bit query, head_size 64 or 128 (MMAs in binary16).
cudaError_t launch_prefill_tc_f16_e4m3(const PrefillParams& p, int head_size, cudaStream_t stream);
cudaError_t launch_prefill_tc_bf16_e4m3(const PrefillParams& p, int head_size, cudaStream_t stream);

// The KV append with norms and rotation (rope_and_cache.cu).
struct RopeParams {
    void* query_out;              // [T, Hq, D]
    const void* query;            // rows of Hq * D elements, query_stride apart
    const void* key;
    const void* value;
    int64_t query_stride;         // elements between tokens
    int64_t key_stride;
    int64_t value_stride;
    void* k_cache;                // [num_blocks, Hkv, B, D]
    void* v_cache;
    const float* cos_sin;         // [max_position, rotary_dim]: cosines, then sines
    const int64_t* positions;     // [num_axes, T]
    const int64_t* slots;         // [T]
    const float* q_weight;        // [D] or null
    const float* k_weight;
    uint32_t* status;             // may be null
    int64_t total_tokens;         // T
    int64_t max_position;
    int64_t num_blocks;
    int num_axes;                 // 1..4
    int rotary_dim;
    int adjacent_pairs;           // pairs (2i, 2i + 1) instead of (i, i + rotary_dim / 2)
    int num_q_heads;
    int num_kv_heads;
    int block_size;
    float eps;
    float k_scale;
    float v_scale;
    int group_shift;              // set by the launcher: log2 of a token's row groups
    float k_inv;                  // 1 / scale, or 0 where that is no normal number
    float v_inv;
    uint32_t freq_axes[8];        // two bits per frequency
};

cudaError_t launch_rope_and_cache(const RopeParams& p, int head_size, pa_dtype in_dtype,
                                  pa_dtype cache_dtype, cudaStream_t stream);

// Per-block key bounds (key_bounds.cu).
struct BoundsParams {
    void* k_bounds;               // [num_blocks, Hkv, 2, D]: minimum, maximum
    const void* k_cache;          // [num_blocks, Hkv, B, D]
    const int32_t* block_tables;  // [S, max_blocks]
    const int32_t* context_lens;  // [S]
    const int32_t* new_tokens;    // [S], or null: one each
    uint32_t* status;             // may be null
    int64_t num_blocks;
    int max_blocks;
    int num_seqs;
    int num_kv_heads;
    int block_size;
    int max_context_len;
    int max_new_tokens;
    int touched;                  // blocks that max_new_tokens tokens can touch
};

// A warp each in the grid's x, whose thread indices are 32-bit.
constexpr int64_t kMaxBoundsUnits = 1ll << 27;    // touched blocks x KV heads

cudaError_t launch_key_bounds(const BoundsParams& p, int head_size, pa_dtype cache_dtype,
                              pa_dtype bounds_dtype, cudaStream_t stream);

// Block scores and selection of the block-sparse decode (sparse_select.cuh).
// A slab is one (block, KV head) pair of the cache, block * Hkv + head; the
// selection of (sequence s, KV head h) is row s * Hkv + h of slab_tables.
struct SelectParams {
    const void* query;            // [S, Hq, D]
    const void* k_bounds;         // [num_blocks, Hkv, 2, D], the query's type
    const int32_t* block_tables;  // [S, max_blocks]
    const int32_t* context_lens;  // [S]
    float* scores;                // [S * Hkv, max_ctx_blocks]: where they exceed shared memory
    uint64_t* exact_keys;         // [S * Hkv, max_ctx_blocks]: many undecided blocks
    int32_t* slab_tables;         // [S * Hkv, table_width]
    int32_t* slab_lens;           // [S * Hkv] tokens of the selection
    int32_t* selected;            // [S, Hkv, num_select] logical blocks, -1 padded; may be null
    uint32_t* status;             // may be null
    int64_t num_blocks;
    int max_blocks;
    int num_seqs;
    int num_q_heads;
    int num_kv_heads;
    int group;
    int block_size;
    int max_context_len;
    int max_ctx_blocks;           // ceil(max_context_len / block_size)
    int table_width;              // min(num_select, max_ctx_blocks)
    int num_select;
    int first_blocks;
    int recent_blocks;
    int side_bytes;               // set by the launcher: shared memory of the query's sides,
    int taken_bytes;              // of the candidates' bits,
    int keys_in_smem;             // and whether the scores are kept there
};

// The fused block-sparse decode (sparse_decode.cuh).
struct SparseParams {
    SelectParams sel;             // slab_tables, slab_lens unused
    void* out;                    // [S, Hq, D]
    const void* k_cache;
    const void* v_cache;
    float q_mul;                  // scale * log2(e) * (E4M3 cache ? k_scale : 1)
    float v_mul;                  // E4M3 cache ? v_scale : 1
    int list_bytes;               // set by the launcher
};

cudaError_t launch_sparse_decode_f16(const SparseParams& p, int head_size, cudaStream_t stream);
cudaError_t launch_sparse_decode_bf16(const SparseParams& p, int head_size, cudaStream_t stream);
cudaError_t launch_sparse_decode_f16_e4m3(const SparseParams& p, int head_size, cudaStream_t stream);
cudaError_t launch_sparse_decode_bf16_e4m3(const SparseParams& p, int head_size, cudaStream_t stream);

cudaError_t launch_select_blocks(const SelectParams& p, int head_size, pa_dtype q_dtype,
                                 cudaStream_t stream);

// len_cap: context lengths above it are clamped to it (and flagged
// PA_DEV_BAD_LEN), the clamp the partition kernel applied, so that only
// partitions it wrote are merged.
cudaError_t launch_merge(void* out, const float* tmp_out, const float* max_logits,
                         const float* exp_sums, const int32_t* context_lens, int num_seqs,
                         int num_q_heads, int head_size, int partition_size, int max_parts,
                         long long len_cap, pa_dtype out_dtype, uint32_t* status,
                         cudaStream_t stream);

cudaError_t launch_copy_blocks(void* k_cache, void* v_cache, const int64_t* pairs,
                               int64_t num_pairs, int64_t num_blocks, int64_t block_bytes,
                               uint32_t* status, cudaStream_t stream);

cudaError_t launch_wait_selftest(int arrive, uint32_t* status, cudaStream_t stream);

cudaError_t launch_reshape_and_cache(const void* key, const void* value, void* k_cache,
                                     void* v_cache, const int64_t* slots, int64_t num_tokens,
                                     int num_kv_heads, int head_size, int block_size,
                                     int64_t num_blocks, pa_dtype in_dtype, pa_dtype cache_dtype,
                                     float k_scale, float v_scale, uint32_t* status,
                                     cudaStream_t stream);

}  // namespace pagedkv
