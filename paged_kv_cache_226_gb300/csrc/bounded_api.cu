// C-ABI entry points of the bounded-cache operators: host-side validation
// and dispatch.  Declarations and contracts: include/pa.h.
#include <cmath>

#include "bounded_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int finish(cudaError_t e) {
    if (e == cudaSuccess) return PA_OK;
    pa::record_cuda_error(static_cast<int>(e));
    return PA_ERR_CUDA;
}

int rope_and_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                   int64_t v_stride, const int64_t* positions, const int64_t* slot_mapping,
                   const float* inv_freq, int32_t rotary_dim, int32_t interleaved, float factor,
                   void* q_out, int64_t q_out_stride, void* k_cache, void* v_cache,
                   int64_t num_tokens, bool fp8, float k_scale, float v_scale,
                   const pa_shape* shp, void* stream) {
    int st = pa::check_shape(shp, false);
    if (st != PA_OK) return st;
    if (fp8 && (st = pa::check_fp8(shp, k_scale, v_scale)) != PA_OK) return st;
    if (num_tokens < 0 || num_tokens > 0x7fffffffll) return PA_ERR_INVALID_ARG;
    if (rotary_dim < 0 || rotary_dim > shp->head_dim || (interleaved != 0 && interleaved != 1) ||
        !std::isfinite(factor))
        return PA_ERR_INVALID_ARG;
    if (rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (q && shp->num_q_heads <= 0) return PA_ERR_INVALID_ARG;
    if (shp->num_q_heads > 65535 || shp->num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!k || !v || !positions || !slot_mapping || !k_cache || !v_cache || (q && !q_out) ||
        (rotary_dim > 0 && !inv_freq))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
        !aligned16(k_cache) || !aligned16(v_cache) || !aligned8(positions) ||
        !aligned8(slot_mapping) || !aligned4(inv_freq))
        return PA_ERR_INVALID_ARG;
    const int64_t kv_row = (int64_t)shp->num_kv_heads * shp->head_dim;
    const int64_t q_row = (int64_t)shp->num_q_heads * shp->head_dim;
    if (k_stride < kv_row || v_stride < kv_row || (k_stride | v_stride) % 8 != 0)
        return PA_ERR_INVALID_ARG;
    if (q && (q_stride < q_row || q_out_stride < q_row || (q_stride | q_out_stride) % 8 != 0 ||
              (q == q_out && q_stride != q_out_stride)))
        return PA_ERR_INVALID_ARG;
    pa::RopeParams p{};
    cudaError_t e = pa::error_word(&p.err);
    if (e != cudaSuccess) return finish(e);
    p.q = q, p.k = k, p.v = v, p.positions = positions, p.slots = slot_mapping;
    p.inv_freq = inv_freq, p.q_out = q_out, p.k_cache = k_cache, p.v_cache = v_cache;
    p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
    p.q_out_stride = q_out_stride;
    p.num_tokens = num_tokens, p.num_slots = shp->num_blocks * shp->block_size;
    p.num_q_heads = q ? shp->num_q_heads : 0, p.num_kv_heads = shp->num_kv_heads;
    p.rotary_dim = rotary_dim, p.factor = factor, p.k_scale = k_scale, p.v_scale = v_scale;
    return finish(pa::launch_rope_and_cache(shp->dtype, shp->head_dim, fp8, interleaved != 0, p,
                                            static_cast<cudaStream_t>(stream)));
}

// Parts of the decode-weights workspace, each 256-byte aligned.
struct WeightsWorkspace {
    size_t logits, sums, scores, bytes;      // offsets (tmp_out at 0) and the total
    int parts;
};

// 0 parts: invalid arguments.
WeightsWorkspace weights_layout(const pa_shape* s, int32_t max_context_len, int32_t partition_size) {
    WeightsWorkspace w{};
    if (max_context_len < 0 || partition_size <= 0 || partition_size % s->block_size != 0) return w;
    w.parts = max_context_len / partition_size + (max_context_len % partition_size != 0);
    if (w.parts == 0) w.parts = 1;
    const size_t rows = (size_t)s->num_seqs * s->num_q_heads * w.parts;
    w.logits = round256(rows * s->head_dim * sizeof(float));
    w.sums = w.logits + round256(rows * sizeof(float));
    w.scores = w.sums + round256(rows * sizeof(float));
    w.bytes = w.scores + round256(rows * partition_size * sizeof(float));
    return w;
}

// The state arrays [num_seqs][num_kv_heads][stride] cover every token the
// tables can hold.
int check_state(const void* in, const void* out, int64_t stride, const pa_shape* shp) {
    if (!out || !aligned16(out) || !aligned16(in)) return PA_ERR_INVALID_ARG;
    if (stride < (int64_t)shp->max_blocks_per_seq * shp->block_size) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

int decode_weights(const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, const int32_t* context_lens, float scale, bool fp8,
                   float k_scale, float v_scale, int32_t max_context_len, int32_t partition_size,
                   const float* weights, float* weights_out, int64_t weights_stride,
                   void* workspace, size_t workspace_bytes, void* out, const pa_shape* shp,
                   void* stream) {
    int st = pa::check_decode_args(q, k_cache, v_cache, block_tables, context_lens, shp);
    if (st != PA_OK) return st;
    if (fp8 && (st = pa::check_fp8(shp, k_scale, v_scale)) != PA_OK) return st;
    const WeightsWorkspace w = weights_layout(shp, max_context_len, partition_size);
    if (w.parts == 0) return PA_ERR_INVALID_ARG;
    // grids: a partition, or 256 tokens of the merge at least, along z
    if (w.parts > 65535 || max_context_len / 256 > 65000) return PA_ERR_UNSUPPORTED;
    if (shp->num_seqs == 0) return PA_OK;
    if (!out || !aligned16(out)) return PA_ERR_INVALID_ARG;
    if ((st = check_state(weights, weights_out, weights_stride, shp)) != PA_OK) return st;
    if (!workspace || workspace_bytes < w.bytes) return PA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PA_ERR_INVALID_ARG;
    CUtensorMap tmk, tmv;
    if ((st = pa::encode_cache_map(&tmk, k_cache, shp, fp8)) != PA_OK) return st;
    if ((st = pa::encode_cache_map(&tmv, v_cache, shp, fp8)) != PA_OK) return st;
    pa::DecodeParams p{};
    cudaError_t e = pa::error_word(&p.err);
    if (e != cudaSuccess) return finish(e);
    char* base = static_cast<char*>(workspace);
    p.q = q, p.block_tables = block_tables, p.context_lens = context_lens;
    p.scale_log2 = scale * (fp8 ? k_scale : 1.f) * pa::kLog2e;
    p.k_scale = k_scale, p.v_scale = v_scale;
    p.num_q_heads = shp->num_q_heads, p.num_kv_heads = shp->num_kv_heads;
    p.group = shp->num_q_heads / shp->num_kv_heads;
    p.max_blocks_per_seq = shp->max_blocks_per_seq, p.block_size = shp->block_size;
    p.num_blocks = shp->num_blocks;
    p.partition_tokens = partition_size, p.max_parts = w.parts;
    p.tmp_out = reinterpret_cast<float*>(base);
    p.max_logits = reinterpret_cast<float*>(base + w.logits);
    p.exp_sums = reinterpret_cast<float*>(base + w.sums);
    p.scores = reinterpret_cast<float*>(base + w.scores);
#ifdef PA_TEST_HOOKS
    const pa::TestFault fault = pa::test_fault();
    p.test_cta = fault.cta, p.test_tile = fault.tile, p.test_wait_limit_ns = fault.wait_limit_ns;
#endif
    const dim3 grid(shp->num_seqs, shp->num_kv_heads, w.parts);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // One launch, the partitions a cluster that joins them, for contexts of one
    // partition (us against decode + merge: 1216 pairs of 200 tokens 31.7 and
    // 35.4, 512 of 1040 53.5 and 55.5) or a few short ones (64 pairs of up to
    // 250 tokens in four 6.8 and 7.4; 8 pairs 5.9 and 5.6, but a launch less
    // to make).  Clusters of longer partitions hold their SM slots until the
    // slowest ends (512 pairs of up to 2048 in two 67 and 57).
    const bool join = (w.parts == 1 && partition_size <= 1024) || (w.parts <= 4 && partition_size <= 64);
    const int mode = join ? pa::kModeWeightsJoin : pa::kModeWeights;
    p.out = out, p.weights = weights, p.weights_out = weights_out, p.weights_stride = weights_stride;
    e = fp8 ? pa::launch_decode_fp8(shp->dtype, mode, tmk, tmv, p, grid, s)
            : pa::launch_decode(shp->dtype, shp->head_dim, mode, tmk, tmv, p, grid, s);
    if (e != cudaSuccess || join) return finish(e);
    pa::WeightsMergeParams m{};
    m.tmp_out = p.tmp_out, m.max_logits = p.max_logits, m.exp_sums = p.exp_sums;
    m.scores = p.scores, m.context_lens = context_lens;
    m.weights = weights, m.weights_out = weights_out, m.weights_stride = weights_stride;
    m.out = out;
    m.num_q_heads = p.num_q_heads, m.num_kv_heads = p.num_kv_heads, m.group = p.group;
    m.partition_tokens = partition_size, m.max_parts = w.parts;
    m.max_context = shp->max_blocks_per_seq * shp->block_size;
    return finish(pa::launch_weights_merge(shp->dtype, shp->head_dim, m, shp->num_seqs, s));
}

// The sizes that the plan of pa_prefill_weights depends on.
pa::PrefillWeightsParams prefill_weights_sizes(const pa_shape* shp, int32_t max_query_len,
                                               int32_t max_context_len, int32_t window) {
    pa::PrefillWeightsParams p{};
    const int table = shp->max_blocks_per_seq * shp->block_size;
    p.num_seqs = shp->num_seqs, p.num_kv_heads = shp->num_kv_heads;
    p.group = shp->num_q_heads / shp->num_kv_heads;
    p.max_context = max_context_len < table ? max_context_len : table;
    const int longest = max_query_len < p.max_context ? max_query_len : p.max_context;
    p.max_counted = window > 0 && window < longest ? window : longest;
    p.window = window;
    return p;
}

int evict_counted(const pa_shape* s, int32_t budget) {
    const int64_t over = (int64_t)s->max_blocks_per_seq * s->block_size - budget;
    return over <= 0 ? 0 : (int)(over < budget ? over : budget);
}

int evict(void* k_cache, void* v_cache, const int32_t* block_tables, const int32_t* context_lens,
          const int32_t* seen_lens, const int32_t* known_lens, const float* weights,
          const int32_t* positions, int64_t stride, int32_t budget, int32_t trigger, int32_t sinks,
          int32_t recent, float* weights_out, int32_t* positions_out, int32_t* new_lens,
          void* workspace, size_t workspace_bytes, bool fp8, const pa_shape* shp, void* stream) {
    int st = pa::check_decode_args(k_cache, k_cache, v_cache, block_tables, context_lens, shp);
    if (st != PA_OK) return st;
    if (fp8 && (st = pa::check_fp8(shp, 1.f, 1.f)) != PA_OK) return st;
    if (budget < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget || trigger < budget)
        return PA_ERR_INVALID_ARG;
    if (shp->num_seqs == 0) return PA_OK;
    if (!seen_lens || !aligned4(seen_lens) || !aligned4(known_lens) || !weights || !positions ||
        !new_lens || !aligned4(new_lens) || new_lens == context_lens || new_lens == known_lens ||
        new_lens == seen_lens)
        return PA_ERR_INVALID_ARG;
    if ((st = check_state(weights, weights_out, stride, shp)) != PA_OK) return st;
    if ((st = check_state(positions, positions_out, stride, shp)) != PA_OK) return st;
    if (!workspace || workspace_bytes < pa_evict_workspace_size(shp, budget)) return PA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PA_ERR_INVALID_ARG;
    pa::EvictParams p{};
    cudaError_t e = pa::error_word(&p.err);
    if (e != cudaSuccess) return finish(e);
    p.k_cache = k_cache, p.v_cache = v_cache, p.block_tables = block_tables;
    p.context_lens = context_lens, p.seen_lens = seen_lens, p.known_lens = known_lens;
    p.weights = weights, p.positions = positions, p.weights_out = weights_out;
    p.positions_out = positions_out, p.stride = stride, p.new_lens = new_lens;
    p.num_moves = static_cast<int32_t*>(workspace);
    p.moves = p.num_moves + round256((size_t)shp->num_seqs * shp->num_kv_heads * 4) / 4;
    p.num_seqs = shp->num_seqs, p.num_kv_heads = shp->num_kv_heads;
    p.max_blocks_per_seq = shp->max_blocks_per_seq, p.block_size = shp->block_size;
    p.num_blocks = shp->num_blocks;
    p.row_bytes = shp->head_dim * (fp8 ? 1 : 2);
    p.budget = budget, p.trigger = trigger, p.sinks = sinks, p.recent = recent;
    p.moves_stride = evict_counted(shp, budget);
    return finish(pa::launch_evict(p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int pa_rope_and_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const void* v, int64_t v_stride, const int64_t* positions,
                      const int64_t* slot_mapping, const float* inv_freq, int32_t rotary_dim,
                      int32_t interleaved, float factor, void* q_out, int64_t q_out_stride,
                      void* k_cache, void* v_cache, int64_t num_tokens, const pa_shape* shp,
                      void* stream) {
    return rope_and_cache(q, q_stride, k, k_stride, v, v_stride, positions, slot_mapping, inv_freq,
                          rotary_dim, interleaved, factor, q_out, q_out_stride, k_cache, v_cache,
                          num_tokens, false, 1.f, 1.f, shp, stream);
}

int pa_rope_and_cache_fp8(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int64_t* positions,
                          const int64_t* slot_mapping, const float* inv_freq, int32_t rotary_dim,
                          int32_t interleaved, float factor, void* q_out, int64_t q_out_stride,
                          void* k_cache, void* v_cache, int64_t num_tokens, float k_scale,
                          float v_scale, const pa_shape* shp, void* stream) {
    return rope_and_cache(q, q_stride, k, k_stride, v, v_stride, positions, slot_mapping, inv_freq,
                          rotary_dim, interleaved, factor, q_out, q_out_stride, k_cache, v_cache,
                          num_tokens, true, k_scale, v_scale, shp, stream);
}

size_t pa_decode_weights_workspace_size(const pa_shape* shp, int32_t max_context_len,
                                        int32_t partition_size) {
    if (pa::check_shape(shp, true) != PA_OK) return 0;
    return weights_layout(shp, max_context_len, partition_size).bytes;
}

int pa_decode_weights(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, const int32_t* context_lens, float scale,
                      int32_t max_context_len, int32_t partition_size, const float* weights,
                      float* weights_out, int64_t weights_stride, void* workspace,
                      size_t workspace_bytes, void* out, const pa_shape* shp, void* stream) {
    return decode_weights(q, k_cache, v_cache, block_tables, context_lens, scale, false, 1.f, 1.f,
                          max_context_len, partition_size, weights, weights_out, weights_stride,
                          workspace, workspace_bytes, out, shp, stream);
}

int pa_decode_weights_fp8(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens, float scale,
                          float k_scale, float v_scale, int32_t max_context_len,
                          int32_t partition_size, const float* weights, float* weights_out,
                          int64_t weights_stride, void* workspace, size_t workspace_bytes,
                          void* out, const pa_shape* shp, void* stream) {
    return decode_weights(q, k_cache, v_cache, block_tables, context_lens, scale, true, k_scale,
                          v_scale, max_context_len, partition_size, weights, weights_out,
                          weights_stride, workspace, workspace_bytes, out, shp, stream);
}

size_t pa_prefill_weights_workspace_size(const pa_shape* shp, int32_t max_query_len,
                                         int32_t max_context_len, int32_t window) {
    if (pa::check_shape(shp, true) != PA_OK || max_query_len < 0 || max_context_len < 0 || window < 0)
        return 0;
    pa::PrefillWeightsParams p = prefill_weights_sizes(shp, max_query_len, max_context_len, window);
    return pa::prefill_weights_plan(p, nullptr);
}

int pa_prefill_weights(const void* q, const void* k_cache, const int32_t* block_tables,
                       const int32_t* context_lens, const int32_t* query_start, float scale,
                       int64_t num_tokens, int32_t max_query_len, int32_t max_context_len,
                       int32_t window, const float* weights, float* weights_out,
                       int64_t weights_stride, void* workspace, size_t workspace_bytes,
                       const pa_shape* shp, void* stream) {
    int st = pa::check_decode_args(k_cache, k_cache, k_cache, block_tables, context_lens, shp);
    if (st != PA_OK) return st;
    if (num_tokens < 0 || num_tokens > 0x7fffffffll || max_query_len < 0 || max_context_len < 0 ||
        window < 0 || !(scale > 0.f) || !std::isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (shp->num_seqs == 0) return PA_OK;
    if (!query_start || !aligned4(query_start) || (num_tokens > 0 && !q) || !aligned16(q))
        return PA_ERR_INVALID_ARG;
    if ((st = check_state(weights, weights_out, weights_stride, shp)) != PA_OK) return st;
    pa::PrefillWeightsParams p = prefill_weights_sizes(shp, max_query_len, max_context_len, window);
    if (!workspace || workspace_bytes < pa::prefill_weights_plan(p, workspace)) return PA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PA_ERR_INVALID_ARG;
    if (p.max_context == 0) return PA_OK;
    // units of either pass, or key tiles, are counted in 32 bits
    const int64_t tiles = ((int64_t)p.max_context + 127) / 128 * p.num_seqs * p.num_kv_heads;
    const bool lone = p.max_query_tiles <= 1;
    if (tiles * (lone ? 1 : p.query_chunks) >= (1ll << 31) ||
        (!lone && (int64_t)p.max_query_tiles * p.key_chunks * p.num_seqs * p.num_kv_heads >= (1ll << 31)))
        return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) p.max_counted = 0;
    CUtensorMap tmk, tmq;
    if ((st = pa::encode_cache_map(&tmk, k_cache, shp, false)) != PA_OK) return st;
    // no queries: the map is not used, any address will do
    if ((st = pa::encode_query_map(&tmq, num_tokens > 0 ? q : k_cache, shp,
                                   num_tokens > 0 ? num_tokens : 1, p.group, p.tile_tokens)) != PA_OK)
        return st;
    cudaError_t e = pa::error_word(&p.err);
    if (e != cudaSuccess) return finish(e);
    p.block_tables = block_tables, p.context_lens = context_lens, p.query_start = query_start;
    p.weights = weights, p.weights_out = weights_out, p.weights_stride = weights_stride;
    p.scale_log2 = scale * pa::kLog2e;
    p.max_blocks_per_seq = shp->max_blocks_per_seq, p.block_size = shp->block_size;
    p.num_blocks = shp->num_blocks, p.num_tokens = num_tokens;
#ifdef PA_TEST_HOOKS
    const pa::TestFault fault = pa::test_fault();
    p.test_cta = fault.cta, p.test_tile = fault.tile, p.test_wait_limit_ns = fault.wait_limit_ns;
#endif
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    bool launched = false;
    if (lone) e = pa::launch_short_weights(shp->dtype, shp->head_dim, tmk, tmq, p, cs, &launched);
    if (e != cudaSuccess || launched) return finish(e);
    return finish((lone ? pa::launch_window_weights : pa::launch_prefill_weights)(
        shp->dtype, shp->head_dim, tmk, tmq, p, cs));
}

size_t pa_evict_workspace_size(const pa_shape* shp, int32_t budget) {
    if (pa::check_shape(shp, true) != PA_OK || budget < 1) return 0;
    const size_t pairs = (size_t)shp->num_seqs * shp->num_kv_heads;
    return round256(pairs * 4) + round256(pairs * 2 * evict_counted(shp, budget) * 4 + 1);
}

int pa_evict(void* k_cache, void* v_cache, const int32_t* block_tables,
             const int32_t* context_lens, const int32_t* seen_lens, const int32_t* known_lens,
             const float* weights, const int32_t* positions, int64_t stride, int32_t budget,
             int32_t trigger, int32_t sinks, int32_t recent, float* weights_out,
             int32_t* positions_out, int32_t* new_lens, void* workspace, size_t workspace_bytes,
             const pa_shape* shp, void* stream) {
    return evict(k_cache, v_cache, block_tables, context_lens, seen_lens, known_lens, weights,
                 positions, stride, budget, trigger, sinks, recent, weights_out, positions_out,
                 new_lens, workspace, workspace_bytes, false, shp, stream);
}

int pa_evict_fp8(void* k_cache, void* v_cache, const int32_t* block_tables,
                 const int32_t* context_lens, const int32_t* seen_lens, const int32_t* known_lens,
                 const float* weights, const int32_t* positions, int64_t stride, int32_t budget,
                 int32_t trigger, int32_t sinks, int32_t recent, float* weights_out,
                 int32_t* positions_out, int32_t* new_lens, void* workspace,
                 size_t workspace_bytes, const pa_shape* shp, void* stream) {
    return evict(k_cache, v_cache, block_tables, context_lens, seen_lens, known_lens, weights,
                 positions, stride, budget, trigger, sinks, recent, weights_out, positions_out,
                 new_lens, workspace, workspace_bytes, true, shp, stream);
}

}  // extern "C"
