// Parameters and launchers of the operators that keep a paged cache within a
// budget of tokens: rotary positions with the cache write (rope_cache.cu),
// the accumulated attention weights of decode (decode_weights.cu) and of
// prefill chunks (prefill_weights.cu), and eviction (evict.cu).
#pragma once

#include "pa_internal.h"

namespace pa {

struct RopeParams {
    const void* q;                 // [T] rows of Hq * D, q_stride elements apart (null: no q)
    const void* k;
    const void* v;
    const int64_t* positions;      // [T]
    const int64_t* slots;          // [T]
    const float* inv_freq;         // [rotary_dim / 2]
    void* q_out;
    void* k_cache;
    void* v_cache;
    int* err;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int64_t num_tokens;
    int64_t num_slots;
    int num_q_heads, num_kv_heads;
    int rotary_dim;
    float factor;
    float k_scale, v_scale;        // E4M3 cache only
};

cudaError_t launch_rope_and_cache(int dtype, int head_dim, bool fp8, bool interleaved,
                                  const RopeParams& p, cudaStream_t stream);

// Merge of the partitions written by the decode kernel's weights mode, and
// the weights themselves.
struct WeightsMergeParams {
    const float* tmp_out;          // [B][Hq][S][D]
    const float* max_logits;       // [B][Hq][S], log2 units
    const float* exp_sums;         // [B][Hq][S]
    const float* scores;           // [B][Hkv][S * P][G], log2 units
    const int32_t* context_lens;
    const float* weights;          // [B][Hkv][stride], null: none yet
    float* weights_out;            // [B][Hkv][stride]
    int64_t weights_stride;
    void* out;                     // [B][Hq][D]
    int num_q_heads, num_kv_heads, group;
    int partition_tokens, max_parts;
    int max_context;               // max_blocks_per_seq * block_size
};

cudaError_t launch_weights_merge(int dtype, int head_dim, const WeightsMergeParams& p,
                                 int num_seqs, cudaStream_t stream);

struct PrefillWeightsParams {
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_start;    // [B + 1]
    const float* weights;          // [B][Hkv][stride], null: none yet
    float* weights_out;
    int64_t weights_stride;
    int* err;
    float scale_log2;
    int num_seqs, num_kv_heads, group;
    int max_blocks_per_seq, block_size;
    int64_t num_blocks;
    int64_t num_tokens;            // rows of q
    int max_context;               // smaller of the table's and the caller's bound
    int max_counted;               // queries counted per sequence at most
    int window;                    // 0: every query of the chunk
    // filled by prefill_weights_plan
    int tile_tokens;               // query tokens per tile of 128 rows
    int max_query_tiles;
    int key_chunk, key_chunks;     // key tiles per unit of pass 1, units of the longest row
    int query_chunk, query_chunks; // query tiles per unit of pass 2, units of a column
    float* lse;                    // [B][Hkv][max_query_tiles][128], log2 units
    float2* stats;                 // [key_chunks] x the same: maximum and sum
    float* columns;                // [query_chunks][B][Hkv][columns_stride]
    int columns_stride;
#ifdef PA_TEST_HOOKS
    // Test builds only: CTA test_cta's loaders issue no streamed tile from
    // test_tile on, and waits give up after test_wait_limit_ns.
    int test_cta, test_tile;
    unsigned long long test_wait_limit_ns;
#endif
};

// Chooses the chunks, lays out the workspace and returns its bytes (needs
// the sizes: group, num_seqs, num_kv_heads, max_context, max_counted).
size_t prefill_weights_plan(PrefillWeightsParams& p, void* workspace);
// The case of at most one query tile per sequence (prefill_window.cu).
size_t window_weights_plan(PrefillWeightsParams& p, void* workspace);
cudaError_t launch_window_weights(int dtype, int head_dim, const CUtensorMap& tmk,
                                  const CUtensorMap& tmq, const PrefillWeightsParams& p,
                                  cudaStream_t stream);
// The same in one launch where the contexts fit the shared memory of one wave
// (prefill_short.cu); nothing is done where `launched` comes back false.
cudaError_t launch_short_weights(int dtype, int head_dim, const CUtensorMap& tmk,
                                 const CUtensorMap& tmq, const PrefillWeightsParams& p,
                                 cudaStream_t stream, bool* launched);
cudaError_t launch_prefill_weights(int dtype, int head_dim, const CUtensorMap& tmk,
                                   const CUtensorMap& tmq, const PrefillWeightsParams& p,
                                   cudaStream_t stream);

struct EvictParams {
    void* k_cache;
    void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* seen_lens;
    const int32_t* known_lens;     // null: 0
    const float* weights;          // [B][Hkv][stride]
    const int32_t* positions;
    float* weights_out;
    int32_t* positions_out;
    int64_t stride;
    int32_t* new_lens;
    int32_t* moves;                // [B][Hkv][2][moves_stride]: gaps, then movers
    int32_t* num_moves;            // [B][Hkv]
    int* err;
    int num_seqs, num_kv_heads;
    int max_blocks_per_seq, block_size;
    int64_t num_blocks;
    int row_bytes;                 // of one head's K (or V) of one token
    int budget, trigger, sinks, recent;
    int moves_stride;
    int cluster;                   // CTAs of the select kernel per (sequence, KV head)
    int own_moves;                 // moves that each makes itself
};

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);

}  // namespace pa
