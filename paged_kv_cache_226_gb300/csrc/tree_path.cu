// The end of a verification step: which drafted tokens the model agrees with,
// and the accepted path's rows closing up behind the context.
#include "tree_device.cuh"

namespace pa {

// One thread per node, one CTA per sequence.  With every node's line as a bit
// mask, a node is accepted where no bit of its line is a node that disagrees,
// its depth is the mask's bit count, and the path is the mask itself: parents
// stand before their children, so its ascending bits are the way down.
// What bounds it is its chain of dependent steps: bounds, tokens and parents
// from memory, up to seven rounds of masks, two reductions.  6.0 us with cold
// caches for 256 sequences (0.3 MB); calls back to back 4.9 to 5.1 us, which is
// the host's side of a call.
__global__ void __launch_bounds__(kLineThreads)
    accept_tree_kernel(const __grid_constant__ AcceptParams p) {
    __shared__ LineRoom room;
    __shared__ int64_t target_s[PA_TREE_NODES];
    __shared__ uint32_t wrong_s[kLineWords];
    __shared__ int best_s[kLineThreads / 32];
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.x, i = threadIdx.x;
    TreeSeq s;
    bool bad = false;
    tree_rows(p.query_start[b], p.query_start[b + 1], p.num_tokens, p.max_query, s, bad);
    if (bad && i == 0) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
    const bool live = i < s.C;
    const int64_t row = (int64_t)s.q0 + i;
    const int64_t draft = live ? p.draft[row] : 0, target = live ? p.target[row] : 0;
    const int up = live ? tree_parent(p.parents, s.q0, i, p.err) : -1;
    target_s[i] = target;
    const TreeLine line = tree_line(room, i, s.C, up, [](bool more) { return __syncthreads_or(more) != 0; });
    const bool agrees = live && (up < 0 ? i == 0 : draft == target_s[up]);
    const uint32_t wrong = __ballot_sync(0xffffffffu, !agrees);
    if ((i & 31) == 0) wrong_s[i >> 5] = wrong;
    __syncthreads();
    bool accepted = live;
    int depth = 0;
#pragma unroll
    for (int k = 0; k < kLineWords; ++k) {
        accepted = accepted && (line.w[k] & wrong_s[k]) == 0u;
        depth += __popc(line.w[k]);
    }
    // the deepest, the lowest among equals: 0 where there is none
    int best = accepted ? depth * PA_TREE_NODES + (PA_TREE_NODES - 1 - i) : 0;
    best = __reduce_max_sync(0xffffffffu, best);
    if ((i & 31) == 0) best_s[i >> 5] = best;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kLineThreads / 32; ++k) best = max(best, best_s[k]);
    const int length = best / PA_TREE_NODES, end = PA_TREE_NODES - 1 - best % PA_TREE_NODES;
    int32_t* path = p.path + (int64_t)b * p.max_query;
    if (i >= length && i < p.max_query) path[i] = -1;
    if (i == 0) {
        p.path_lens[b] = length;
        if (length == 0) p.next[b] = -1;
    }
    if (length > 0 && i == end) {
        p.next[b] = target;
        int at = 0;
#pragma unroll
        for (int k = 0; k < kLineWords; ++k)
            for (uint32_t m = line.w[k]; m != 0u; m &= m - 1u) path[at++] = 32 * k + __ffs((int)m) - 1;
    }
}

cudaError_t launch_accept_tree(const AcceptParams& p, cudaStream_t stream) {
    return launch_with_pdl(accept_tree_kernel, dim3((unsigned)p.num_seqs), dim3(kLineThreads), 0, stream, p);
}

// A CTA moves one sequence's rows in one cache; a thread owns 16-byte columns
// of the rows and makes the path's moves in order, a batch of loads before the
// batch's stores.  Entry j goes to base + j, and later entries lie above it
// (path[k] >= path[j] + (k - j) > j), so no row is written that is still to be
// read, within a thread's column or in another's.
// Loads that the path does not ask for are not made, and all layers go in one
// grid: 32 layers are 64 pointers in the arguments.
// Again a chain of loads (lengths and path, table, rows) and the launch: one
// layer 3.7 us a call, 32 layers 5.4 (9.3 us with cold caches, 4 MB read; a
// launch for each layer would take 32 times 3.7).
constexpr int kCommitThreads = 128;
constexpr int kCommitBatch = 8;

__global__ void __launch_bounds__(kCommitThreads)
    commit_path_kernel(const __grid_constant__ CommitParams p) {
    __shared__ int64_t src_s[PA_TREE_NODES], dst_s[PA_TREE_NODES];
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.x, t = threadIdx.x;
    const bool report = p.report && blockIdx.y == 0;
    const int max_context = p.max_blocks_per_seq * p.block_size;
    int L = p.context_lens[b], n = p.path_lens[b];
    const int entry = t < p.path_stride ? p.path[(int64_t)b * p.path_stride + t] : -1;
    const int before = t > 0 && t < p.path_stride ? p.path[(int64_t)b * p.path_stride + t - 1] : -1;
    int64_t C = (int64_t)p.query_start[b + 1] - p.query_start[b];
    // where the tree lies is not known, and nothing moves
    bool nowhere = false;
    if (L < 0 || L > max_context) nowhere = true, L = L < 0 ? 0 : max_context;
    if (C < 0 || C > L) nowhere = true, C = 0;
    const int base = L - (int)C, nodes = min((int)C, PA_TREE_NODES);
    if ((nowhere || nodes < C) && report && t == 0) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
    const bool wrong = n < 0 || n > nodes || n > p.path_stride || (t < n && (entry <= before || entry >= nodes));
    const bool refused = __syncthreads_or(wrong) != 0 || nowhere;
    if (report && t == 0) {
        if (refused && !nowhere) flag_error(p.err, PA_DEVERR_BAD_INDEX);
        p.new_lens[b] = refused ? L : base + n;
    }
    if (refused) return;
    if (t < n) {
        const int32_t* table = p.block_tables + (int64_t)b * p.max_blocks_per_seq;
        const int from = base + entry, to = base + t;
        const int fb = table[from / p.block_size], tb = table[to / p.block_size];
        const bool out = fb < 0 || fb >= p.num_blocks || tb < 0 || tb >= p.num_blocks;
        if (out && report) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
        src_s[t] = out || entry == t ? -1 : (int64_t)fb * p.block_size + from % p.block_size;
        dst_s[t] = (int64_t)tb * p.block_size + to % p.block_size;
    }
    __syncthreads();
    uint4* cache = static_cast<uint4*>(p.caches[blockIdx.y]);
    for (int c = t; c < p.row_vectors; c += kCommitThreads) {
        for (int j0 = 0; j0 < n; j0 += kCommitBatch) {
            uint4 v[kCommitBatch];
#pragma unroll
            for (int k = 0; k < kCommitBatch; ++k)
                if (j0 + k < n && src_s[j0 + k] >= 0) v[k] = cache[src_s[j0 + k] * p.row_vectors + c];
#pragma unroll
            for (int k = 0; k < kCommitBatch; ++k)
                if (j0 + k < n && src_s[j0 + k] >= 0) cache[dst_s[j0 + k] * p.row_vectors + c] = v[k];
        }
    }
}

cudaError_t launch_commit_path(const CommitParams& p, cudaStream_t stream) {
    return launch_with_pdl(commit_path_kernel, dim3((unsigned)p.num_seqs, (unsigned)p.num_caches),
                           dim3(kCommitThreads), 0, stream, p);
}

}  // namespace pa
