// A sequence's tree of drafted tokens on the device: its bounds, and the
// ancestors of its nodes as bit masks.
#pragma once

#include "pa_device.cuh"
#include "tree_internal.h"

namespace pa {

// Nodes [0, C) of a sequence in rows [q0, q0 + C) of the batch, its first
// L - C cached tokens being the context.
struct TreeSeq {
    int L, C, q0;
};

// Rows [start, end) of the batch as at most `most` nodes of a tree.
__device__ __forceinline__ void tree_rows(int start, int end, int64_t num_tokens, int most, TreeSeq& s,
                                          bool& bad) {
    int64_t c = (int64_t)end - start;
    if (c < 0) bad = true, c = 0;
    if (start < 0 || start + c > num_tokens) bad = true, c = 0;
    if (c > most) bad = true, c = most;
    s.q0 = start, s.C = (int)c;
}

// kL2: read past L1, by a kernel that runs ahead of the one before it.
template <bool kL2 = false>
__device__ __forceinline__ TreeSeq tree_sequence(const TreeParams& p, int b, bool report) {
    auto at = [](const int32_t* x) { return kL2 ? __ldcg(x) : *x; };
    TreeSeq s;
    bool bad = false;
    s.L = at(p.context_lens + b);
    const int start = at(p.query_start + b), end = at(p.query_start + b + 1);
    if (s.L < 0 || s.L > p.max_context) bad = true, s.L = s.L < 0 ? 0 : p.max_context;
    tree_rows(start, end, p.num_tokens, s.L, s, bad);
    // nodes past the first max_query are cut off, with their tokens: the others
    // stay where they are
    if (s.C > p.max_query) bad = true, s.L -= s.C - p.max_query, s.C = p.max_query;
    if (bad && report) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
    return s;
}

constexpr int kLineWords = PA_TREE_NODES / 32;

// A node's line: itself and its ancestors, a bit per node.
struct TreeLine {
    uint32_t w[kLineWords];
    __device__ __forceinline__ bool has(int i) const {
        const uint32_t lo = i & 32 ? w[1] : w[0], hi = i & 32 ? w[3] : w[2];
        return ((i & 64 ? hi : lo) >> (i & 31)) & 1u;
    }
};

// The lines of a tree's C nodes, thread `i` of kLineThreads making node i's:
// masks and parents double their reach in every round (node i's line joins
// its parent's, its parent becomes the parent's parent), so a tree of any
// depth takes at most seven.  `barrier` synchronises the threads and returns
// whether any of them passed true.  When the last thread has left, room.line
// holds every node's line; nobody may still read the room at the call.
constexpr int kLineThreads = PA_TREE_NODES;

struct LineRoom {
    uint4 line[PA_TREE_NODES];
    signed char above[PA_TREE_NODES];
};

template <typename Barrier>
__device__ __forceinline__ TreeLine tree_line(LineRoom& room, int i, int C, int parent, Barrier&& barrier) {
    uint32_t w[kLineWords];
#pragma unroll
    for (int k = 0; k < kLineWords; ++k) w[k] = i < C && (i >> 5) == k ? 1u << (i & 31) : 0u;
    int up = i < C && parent >= 0 ? parent : -1;
    room.line[i] = make_uint4(w[0], w[1], w[2], w[3]);
    room.above[i] = (signed char)up;
    while (barrier(up >= 0)) {
        if (up >= 0) {
            const uint4 o = room.line[up];
            w[0] |= o.x, w[1] |= o.y, w[2] |= o.z, w[3] |= o.w;
            up = room.above[up];
        }
        barrier(false);
        room.line[i] = make_uint4(w[0], w[1], w[2], w[3]);
        room.above[i] = (signed char)up;
    }
    return TreeLine{{w[0], w[1], w[2], w[3]}};
}

// Node i's parent, negative for the context's end.
__device__ __forceinline__ int tree_parent(const int32_t* parents, int q0, int i, int* err) {
    if (parents == nullptr) return i - 1;
    const int up = parents[(int64_t)q0 + i];
    if (up >= i) {
        flag_error(err, PA_DEVERR_BAD_INDEX);
        return -1;
    }
    return up;
}

}  // namespace pa
