// C-ABI entry points of the operators of speculative decoding: host-side
// validation and dispatch.  Declarations and contracts: include/pa.h.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "tree_internal.h"

namespace {

constexpr int kMaxLayers = 1024;         // of one pa_commit_path

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether two buffers of `bytes` bytes have some in common.
bool overlap(const void* a, const void* b, uint64_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x == y || (x < y ? y - x : x - y) < bytes;
}

// A buffer of `count` elements of `size` bytes.
struct Span {
    const void* at;
    int64_t count;
    int size;
    bool meets(const Span& o) const {
        const uintptr_t x = reinterpret_cast<uintptr_t>(at), y = reinterpret_cast<uintptr_t>(o.at);
        return count > 0 && o.count > 0 && x < y + (uint64_t)o.count * o.size && y < x + (uint64_t)count * size;
    }
};

// Whether an output lies over an input or over another output.
template <size_t kOutputs, size_t kInputs>
bool written_over(const Span (&outputs)[kOutputs], const Span (&inputs)[kInputs]) {
    for (size_t i = 0; i < kOutputs; ++i) {
        for (const Span& in : inputs)
            if (in.at && outputs[i].meets(in)) return true;
        for (size_t j = 0; j < i; ++j)
            if (outputs[i].meets(outputs[j])) return true;
    }
    return false;
}

int finish(cudaError_t e) {
    if (e == cudaSuccess) return PA_OK;
    pa::record_cuda_error(static_cast<int>(e));
    return PA_ERR_CUDA;
}

// The sizes that the plan of pa_tree_attention depends on.
pa::TreeParams tree_sizes(const pa_shape* shp, int32_t max_query_len, int32_t max_context_len) {
    pa::TreeParams p{};
    p.num_seqs = shp->num_seqs, p.num_q_heads = shp->num_q_heads, p.num_kv_heads = shp->num_kv_heads;
    p.group = shp->num_q_heads / shp->num_kv_heads;
    p.max_context = std::min(max_context_len, shp->max_blocks_per_seq * shp->block_size);
    p.max_query = std::min(max_query_len, p.max_context);
    return p;
}

int check_tree(int32_t max_query_len, int32_t max_context_len) {
    if (max_query_len < 0 || max_context_len < 0) return PA_ERR_INVALID_ARG;
    return max_query_len > PA_TREE_NODES ? PA_ERR_UNSUPPORTED : PA_OK;
}

int tree_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                   const int32_t* context_lens, const int32_t* query_start, const int32_t* parents, float scale,
                   bool fp8, float k_scale, float v_scale, int64_t num_tokens, int32_t max_query_len,
                   int32_t max_context_len, void* workspace, size_t workspace_bytes, void* out,
                   const pa_shape* shp, void* stream) {
    // q and out may be empty: they are looked at below
    int st = pa::check_decode_args(k_cache, k_cache, v_cache, block_tables, context_lens, shp);
    if (st != PA_OK) return st;
    if (fp8 && (st = pa::check_fp8(shp, k_scale, v_scale)) != PA_OK) return st;
    const float scale_log2 = scale * (fp8 ? k_scale : 1.f) * pa::kLog2e;
    // a product that is zero would make NaN of scores that the mask sets to minus infinity
    if (num_tokens < 0 || num_tokens > 0x7fffffffll || !(scale_log2 >= FLT_MIN) || !std::isfinite(scale_log2))
        return PA_ERR_INVALID_ARG;
    if ((st = check_tree(max_query_len, max_context_len)) != PA_OK) return st;
    if (shp->num_seqs == 0) return PA_OK;
    if (!query_start || !aligned(query_start, 4) || !aligned(parents, 4) || !aligned(q, 16) || !aligned(out, 16) ||
        (num_tokens > 0 &&
         (!q || !out || overlap(q, out, 2ull * num_tokens * shp->num_q_heads * shp->head_dim))))
        return PA_ERR_INVALID_ARG;
    pa::TreeParams p = tree_sizes(shp, max_query_len, max_context_len);
    if (!workspace || workspace_bytes < pa::tree_plan(p, shp->head_dim, workspace)) return PA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0 || p.max_query == 0) return PA_OK;
    const int64_t tiles = (p.max_context + pa::kTreeKeys - 1) / pa::kTreeKeys;
    if ((tiles + pa::kTreePairWeight) * p.num_seqs * p.num_kv_heads >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
    CUtensorMap tmk, tmv, tmq;
    if ((st = pa::encode_cache_map(&tmk, k_cache, shp, fp8)) != PA_OK) return st;
    if ((st = pa::encode_cache_map(&tmv, v_cache, shp, fp8)) != PA_OK) return st;
    if ((st = pa::encode_query_map(&tmq, q, shp, num_tokens, p.group, pa::tree_nodes_per_tile(p.group))) != PA_OK)
        return st;
    cudaError_t e = pa::error_word(&p.err);
    if (e != cudaSuccess) return finish(e);
    p.q = q, p.k_cache = k_cache, p.v_cache = v_cache, p.out = out;
    p.block_tables = block_tables, p.context_lens = context_lens, p.query_start = query_start;
    p.parents = parents;
    p.scale_log2 = scale_log2, p.v_scale = v_scale;
    p.max_blocks_per_seq = shp->max_blocks_per_seq, p.block_size = shp->block_size;
    p.num_blocks = shp->num_blocks, p.num_tokens = num_tokens;
#ifdef PA_TEST_HOOKS
    const pa::TestFault fault = pa::test_fault();
    p.test_cta = fault.cta, p.test_tile = fault.tile, p.test_wait_limit_ns = fault.wait_limit_ns;
#endif
    return finish(pa::launch_tree_attention(shp->dtype, shp->head_dim, fp8, tmk, tmv, tmq, p,
                                            static_cast<cudaStream_t>(stream)));
}

int commit_path(void* const* k_caches, void* const* v_caches, int32_t num_layers, const int32_t* block_tables,
                const int32_t* context_lens, const int32_t* query_start, const int32_t* path,
                int32_t path_stride, const int32_t* path_lens, int32_t* new_lens, bool fp8,
                const pa_shape* shp, void* stream) {
    int st = pa::check_shape(shp, true);
    if (st != PA_OK) return st;
    if (fp8 && (st = pa::check_fp8(shp, 1.f, 1.f)) != PA_OK) return st;
    if (num_layers < 1 || path_stride < 0) return PA_ERR_INVALID_ARG;
    if (num_layers > kMaxLayers) return PA_ERR_UNSUPPORTED;
    if (shp->num_seqs == 0) return PA_OK;
    if (!k_caches || !v_caches || !block_tables || !context_lens || !query_start || !path_lens || !new_lens ||
        (path_stride > 0 && !path))
        return PA_ERR_INVALID_ARG;
    for (const int32_t* a : {block_tables, context_lens, query_start, path, path_lens, (const int32_t*)new_lens})
        if (!aligned(a, 4)) return PA_ERR_INVALID_ARG;
    // other CTAs, and the launches of further layers, read the inputs still
    const int64_t B = shp->num_seqs;
    if (written_over({{new_lens, B, 4}}, {{block_tables, B * shp->max_blocks_per_seq, 4}, {context_lens, B, 4},
                                          {query_start, B + 1, 4}, {path, B * path_stride, 4}, {path_lens, B, 4}}))
        return PA_ERR_INVALID_ARG;
    // no cache twice and none over another: two CTAs would move the same rows
    const uint64_t bytes = (uint64_t)shp->num_blocks * shp->block_size * shp->num_kv_heads * shp->head_dim * (fp8 ? 1 : 2);
    void* all[2 * kMaxLayers];
    void** const end = std::copy(v_caches, v_caches + num_layers, std::copy(k_caches, k_caches + num_layers, all));
    for (void** c = all; c < end; ++c)
        if (!*c || !aligned(*c, 16)) return PA_ERR_INVALID_ARG;
    std::sort(all, end);
    if (std::adjacent_find(all, end, [&](void* a, void* b) { return overlap(a, b, bytes); }) != end)
        return PA_ERR_INVALID_ARG;
    pa::CommitParams p{};
    cudaError_t e = pa::error_word(&p.err);
    if (e != cudaSuccess) return finish(e);
    p.block_tables = block_tables, p.context_lens = context_lens, p.query_start = query_start;
    p.path = path, p.path_lens = path_lens, p.new_lens = new_lens;
    p.num_seqs = shp->num_seqs, p.path_stride = path_stride;
    p.max_blocks_per_seq = shp->max_blocks_per_seq, p.block_size = shp->block_size;
    p.num_blocks = shp->num_blocks;
    p.row_vectors = shp->num_kv_heads * shp->head_dim * (fp8 ? 1 : 2) / 16;
    for (int32_t at = 0; at < num_layers; at += pa::kCommitLayers) {
        const int n = std::min(pa::kCommitLayers, num_layers - at);
        std::copy(k_caches + at, k_caches + at + n, p.caches);
        std::copy(v_caches + at, v_caches + at + n, p.caches + n);
        p.num_caches = 2 * n, p.report = at == 0;
        if ((e = pa::launch_commit_path(p, static_cast<cudaStream_t>(stream))) != cudaSuccess) break;
    }
    return finish(e);
}

}  // namespace

extern "C" {

size_t pa_tree_attention_workspace_size(const pa_shape* shp, int32_t max_query_len, int32_t max_context_len) {
    if (pa::check_shape(shp, true) != PA_OK || check_tree(max_query_len, max_context_len) != PA_OK) return 0;
    pa::TreeParams p = tree_sizes(shp, max_query_len, max_context_len);
    return pa::tree_plan(p, shp->head_dim, nullptr);
}

int pa_tree_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      const int32_t* context_lens, const int32_t* query_start, const int32_t* parents,
                      float scale, int64_t num_tokens, int32_t max_query_len, int32_t max_context_len,
                      void* workspace, size_t workspace_bytes, void* out, const pa_shape* shp, void* stream) {
    return tree_attention(q, k_cache, v_cache, block_tables, context_lens, query_start, parents, scale, false,
                          1.f, 1.f, num_tokens, max_query_len, max_context_len, workspace, workspace_bytes, out,
                          shp, stream);
}

int pa_tree_attention_fp8(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                          const int32_t* context_lens, const int32_t* query_start, const int32_t* parents,
                          float scale, float k_scale, float v_scale, int64_t num_tokens,
                          int32_t max_query_len, int32_t max_context_len, void* workspace,
                          size_t workspace_bytes, void* out, const pa_shape* shp, void* stream) {
    return tree_attention(q, k_cache, v_cache, block_tables, context_lens, query_start, parents, scale, true,
                          k_scale, v_scale, num_tokens, max_query_len, max_context_len, workspace,
                          workspace_bytes, out, shp, stream);
}

int pa_accept_tree(const int64_t* draft, const int64_t* target, const int32_t* parents,
                   const int32_t* query_start, int32_t num_seqs, int64_t num_tokens, int32_t max_query_len,
                   int32_t* path, int32_t* path_lens, int64_t* next, void* stream) {
    if (num_seqs < 0 || num_tokens < 0 || num_tokens > 0x7fffffffll || max_query_len < 1)
        return PA_ERR_INVALID_ARG;
    if (max_query_len > PA_TREE_NODES) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!query_start || !path || !path_lens || !next || (num_tokens > 0 && (!draft || !target)))
        return PA_ERR_INVALID_ARG;
    if (!aligned(draft, 8) || !aligned(target, 8) || !aligned(next, 8) || !aligned(parents, 4) ||
        !aligned(query_start, 4) || !aligned(path, 4) || !aligned(path_lens, 4))
        return PA_ERR_INVALID_ARG;
    const int64_t B = num_seqs;
    if (written_over({{path, B * max_query_len, 4}, {path_lens, B, 4}, {next, B, 8}},
                     {{draft, num_tokens, 8}, {target, num_tokens, 8}, {parents, num_tokens, 4}, {query_start, B + 1, 4}}))
        return PA_ERR_INVALID_ARG;
    pa::AcceptParams p{};
    cudaError_t e = pa::error_word(&p.err);
    if (e != cudaSuccess) return finish(e);
    p.draft = draft, p.target = target, p.parents = parents, p.query_start = query_start;
    p.path = path, p.path_lens = path_lens, p.next = next;
    p.num_tokens = num_tokens, p.num_seqs = num_seqs, p.max_query = max_query_len;
    return finish(pa::launch_accept_tree(p, static_cast<cudaStream_t>(stream)));
}

int pa_commit_path(void* const* k_caches, void* const* v_caches, int32_t num_layers,
                   const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
                   const int32_t* path, int32_t path_stride, const int32_t* path_lens, int32_t* new_lens,
                   const pa_shape* shp, void* stream) {
    return commit_path(k_caches, v_caches, num_layers, block_tables, context_lens, query_start, path,
                       path_stride, path_lens, new_lens, false, shp, stream);
}

int pa_commit_path_fp8(void* const* k_caches, void* const* v_caches, int32_t num_layers,
                       const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
                       const int32_t* path, int32_t path_stride, const int32_t* path_lens, int32_t* new_lens,
                       const pa_shape* shp, void* stream) {
    return commit_path(k_caches, v_caches, num_layers, block_tables, context_lens, query_start, path,
                       path_stride, path_lens, new_lens, true, shp, stream);
}

}  // extern "C"
