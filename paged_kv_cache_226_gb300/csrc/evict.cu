// Eviction from a paged cache by accumulated attention weight.
//
// Per (sequence, KV head) with L tokens, L > trigger, K = min(L, budget)
// tokens stay: those at the first `sinks` positions, the `recent` newest
// positions, and for the rest the largest weights (ties: the lowest index).
// A kept token below K stays where it is; the n-th kept token at or past K
// moves into the n-th gap below K, so only the tokens that must move do, and
// no move reads what another writes.  Attention does not depend on the order
// of the tokens in the cache; their positions travel with them.
//
// The choice is a radix select on an order-preserving 32-bit image of the
// weight (protected tokens above every weight), 8 bits a pass.
#include "bounded_internal.h"
#include "pa_device.cuh"

namespace pa {

constexpr int kEvictThreads = 1024;
constexpr uint32_t kProtected = 0xffffffffu;

// Larger weight, larger image: -0 equals +0, NaN lies below everything.
__device__ __forceinline__ uint32_t weight_image(float w) {
    const uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
    if ((u & 0x7fffffffu) == 0u) return 0x80000000u;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct EvictSeq {
    int L, left, known, seen;
};

__device__ __forceinline__ EvictSeq evict_sequence(const EvictParams& p, int b, bool report) {
    EvictSeq s;
    const int max_ctx = p.max_blocks_per_seq * p.block_size;
    s.L = p.context_lens[b];
    if (s.L < 0 || s.L > max_ctx) {
        if (report) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
        s.L = s.L < 0 ? 0 : max_ctx;
    }
    s.left = s.L > p.trigger ? p.budget : s.L;
    s.known = p.known_lens ? p.known_lens[b] : 0;
    s.seen = p.seen_lens[b];
    return s;
}

__device__ __forceinline__ int evict_position(const EvictSeq& s, const int32_t* positions, int i) {
    return i < s.known ? positions[i] : i + (s.seen - s.L);
}

// Exclusive prefix of one packed count per thread over the block, and the
// total; `sums` holds a word per warp.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* sums, uint32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += u;
    }
    __syncthreads();                            // the previous call's reads of sums
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    uint32_t w = lane < kEvictThreads / 32 ? sums[lane] : 0u, wi = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, wi, d);
        if (lane >= d) wi += u;
    }
    *total = __shfl_sync(0xffffffffu, wi, 31);
    return __shfl_sync(0xffffffffu, wi - w, warp) + incl - v;
}

// One CTA per (sequence, KV head): which tokens stay, the gap and mover
// lists, and the state of the tokens that stay in place.
__global__ void __launch_bounds__(kEvictThreads)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sums[32];
    __shared__ uint32_t digit_s, above_s;
    grid_dependency_wait();
    allow_dependent_launch();
    const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const EvictSeq s = evict_sequence(p, b, tid == 0 && g == 0);
    const size_t pair = (size_t)b * p.num_kv_heads + g;
    const float* w = p.weights + pair * p.stride;
    const int32_t* pos = p.positions + pair * p.stride;
    float* wo = p.weights_out + pair * p.stride;
    int32_t* po = p.positions_out + pair * p.stride;
    if (g == 0 && tid == 0) p.new_lens[b] = s.left;
    if (s.left == s.L) {
        if (tid == 0) p.num_moves[pair] = 0;
        for (int i = tid; i < s.L; i += kEvictThreads) {
            wo[i] = w[i];
            po[i] = evict_position(s, pos, i);
        }
        return;
    }
    auto image = [&](int i) {
        const int at = evict_position(s, pos, i);
        return at < p.sinks || at >= s.seen - p.recent ? kProtected : weight_image(w[i]);
    };
    // the image of the left-th largest, and how many of its equals stay
    uint32_t prefix = 0, want = s.left;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < s.L; i += kEvictThreads) {
            const uint32_t k = image(i);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        const uint32_t mine = tid < 256 ? hist[255 - tid] : 0u;
        uint32_t total;
        const uint32_t before = block_prefix(mine, sums, &total);
        if (tid < 256 && before < want && before + mine >= want) digit_s = 255 - tid, above_s = before;
        __syncthreads();
        prefix |= digit_s << shift;
        want -= above_s;
    }
    // gaps below left and movers from left on, in order
    int32_t* gaps = p.moves + pair * 2 * p.moves_stride;
    int32_t* movers = gaps + p.moves_stride;
    uint32_t equal = 0, n_gaps = 0, n_movers = 0;
    for (int i0 = 0; i0 < s.L; i0 += kEvictThreads) {
        const int i = i0 + tid;
        const uint32_t k = i < s.L ? image(i) : 0u;
        const bool eq = i < s.L && k == prefix;
        uint32_t total;
        const uint32_t rank = equal + block_prefix(eq, sums, &total);
        equal += total;
        const bool keep = i < s.L && (k > prefix || (eq && rank < want));
        const bool gap = i < s.left && !keep, mover = i >= s.left && keep;
        // both counts of the block's 1024 tokens fit 16 bits
        const uint32_t at = block_prefix((uint32_t)gap | ((uint32_t)mover << 16), sums, &total);
        if (gap) gaps[n_gaps + (at & 0xffffu)] = i;
        if (mover) movers[n_movers + (at >> 16)] = i;
        n_gaps += total & 0xffffu, n_movers += total >> 16;
        if (i < s.left && keep) {
            wo[i] = w[i];
            po[i] = evict_position(s, pos, i);
        }
    }
    if (tid == 0) p.num_moves[pair] = n_gaps;
}

constexpr int kMoveThreads = 256;
constexpr int kMovesPerCta = 64;

// Grid (move chunks, KV heads, sequences): K and V rows, weight and position
// of each mover into its gap.
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const __grid_constant__ EvictParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const size_t pair = (size_t)b * p.num_kv_heads + g;
    const int n0 = blockIdx.x * kMovesPerCta, n1 = min(n0 + kMovesPerCta, p.num_moves[pair]);
    if (n0 >= n1) return;
    const EvictSeq s = evict_sequence(p, b, false);
    const int32_t* gaps = p.moves + pair * 2 * p.moves_stride;
    const int32_t* movers = gaps + p.moves_stride;
    const int32_t* table = p.block_tables + (size_t)b * p.max_blocks_per_seq;
    const int vecs = p.row_bytes / 16;
    auto row = [&](int i) -> int64_t {           // row of token i and this head, or -1
        const int blk = table[i / p.block_size];
        if (blk < 0 || blk >= p.num_blocks) return -1;
        return (((int64_t)blk * p.block_size + i % p.block_size) * p.num_kv_heads + g) * vecs;
    };
    for (int item = tid; item < (n1 - n0) * 2 * vecs; item += kMoveThreads) {
        const int n = n0 + item / (2 * vecs), c = item % vecs;
        const int64_t src = row(movers[n]), dst = row(gaps[n]);
        if (src < 0 || dst < 0) {
            flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
            continue;
        }
        uint4* cache = static_cast<uint4*>((item / vecs) & 1 ? p.v_cache : p.k_cache);
        cache[dst + c] = cache[src + c];
    }
    for (int n = n0 + tid; n < n1; n += kMoveThreads) {
        const int from = movers[n], to = gaps[n];
        p.weights_out[pair * p.stride + to] = p.weights[pair * p.stride + from];
        p.positions_out[pair * p.stride + to] = evict_position(s, p.positions + pair * p.stride, from);
    }
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
    cudaError_t e = launch_with_pdl(evict_select_kernel, dim3(p.num_kv_heads, p.num_seqs),
                                    dim3(kEvictThreads), 0, stream, p);
    if (e != cudaSuccess || p.moves_stride == 0) return e;
    const dim3 grid((p.moves_stride + kMovesPerCta - 1) / kMovesPerCta, p.num_kv_heads, p.num_seqs);
    return launch_with_pdl(evict_move_kernel, grid, dim3(kMoveThreads), 0, stream, p);
}

}  // namespace pa
