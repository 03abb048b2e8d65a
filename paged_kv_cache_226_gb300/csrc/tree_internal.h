// Parameters and launchers of the operators of speculative decoding: attention
// of a tree of drafted tokens (tree_attention.cu), the accepted path and its
// commit (tree_path.cu).  Rotary positions behind a norm per head are in
// rope_cache.cu.
#pragma once

#include "pa_internal.h"

namespace pa {

struct TreeParams {
    const void* q;                 // [T][Hq][D]
    const void* k_cache;
    const void* v_cache;
    void* out;                     // [T][Hq][D]
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_start;    // [B + 1]
    const int32_t* parents;        // [T], null: a line
    int* err;
    float scale_log2;              // scale * k_scale * log2(e)
    float v_scale;
    int num_seqs, num_q_heads, num_kv_heads, group;
    int max_blocks_per_seq, block_size;
    int64_t num_blocks;
    int64_t num_tokens;            // rows of q
    int max_context;               // smaller of the table's and the caller's bound
    int max_query;                 // nodes per sequence at most
    // filled by tree_plan
    int sides, heads;              // a lane's CTAs: sides (256 rows of queries each) x KV heads
    int ctas;                      // lanes
    bool whole;                    // lanes are dealt whole sequences
    float* rec_o;                  // [ctas][sides][heads][2][2][D / 4][128][4]
    float2* rec_ml;                // [ctas][sides][heads][2][2][128]: reference (log2 units) and sum
#ifdef PA_TEST_HOOKS
    // Test builds only: CTA test_cta's loaders issue no tile from test_tile
    // on, and waits give up after test_wait_limit_ns.
    int test_cta, test_tile;
    unsigned long long test_wait_limit_ns;
#endif
};

// Lays out the work and the workspace, whose bytes it returns (needs the
// sizes: num_seqs, num_kv_heads, group, max_context, max_query).
size_t tree_plan(TreeParams& p, int head_dim, void* workspace);
cudaError_t launch_tree_attention(int dtype, int head_dim, bool fp8, const CUtensorMap& tmk,
                                  const CUtensorMap& tmv, const CUtensorMap& tmq, const TreeParams& p,
                                  cudaStream_t stream);
// Nodes of a query tile: the box of its map.
int tree_nodes_per_tile(int group);
// Keys of a tile, and what a (sequence, KV head) pair weighs beside its tiles
// in the dealing.  The weight of a call is counted in 31 bits.
constexpr int kTreeKeys = 64;
constexpr int kTreePairWeight = 4;

struct AcceptParams {
    const int64_t* draft;          // [T]
    const int64_t* target;         // [T]
    const int32_t* parents;        // [T]
    const int32_t* query_start;    // [B + 1]
    int32_t* path;                 // [B][max_query]
    int32_t* path_lens;            // [B]
    int64_t* next;                 // [B]
    int* err;
    int64_t num_tokens;
    int num_seqs, max_query;
};

cudaError_t launch_accept_tree(const AcceptParams& p, cudaStream_t stream);

constexpr int kCommitLayers = 64;  // per launch: their pointers are kernel arguments

struct CommitParams {
    void* caches[2 * kCommitLayers];   // K of each layer, then V
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* query_start;
    const int32_t* path;           // [B][path_stride]
    const int32_t* path_lens;
    int32_t* new_lens;
    int* err;
    int num_caches, num_seqs;
    int path_stride;
    int max_blocks_per_seq, block_size;
    int64_t num_blocks;
    int row_vectors;               // 16-byte vectors of a token's row in one cache
    bool report;                   // the launch that writes new_lens and flags errors
};

cudaError_t launch_commit_path(const CommitParams& p, cudaStream_t stream);

}  // namespace pa
