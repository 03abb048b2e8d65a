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
// weight (protected tokens above every weight) in digits of 8 bits, whose
// bins one warp scans (64 x 8 rows of 1040 tokens 11.1 us; digits of 11 bits
// that all warps scan together 13.3, of 8 that each scans for itself 13.0).
// Bound by instruction issue, half of the slots (27 warps an SM), and the
// chain of barriers.  A cluster of CTAs serves one (sequence, KV head), each
// CTA a contiguous slice of the tokens with its images in registers;
// histograms and counts are exchanged through distributed shared memory, and every CTA
// draws the same conclusions from them.  Few moves are made by the cluster
// itself; many are left to a second kernel that spreads them over the GPU.
#include "bounded_internal.h"
#include "pa_device.cuh"

namespace pa {

constexpr uint32_t kProtected = 0xffffffffu;
constexpr int kEvictKeys = 8;                // images a thread holds
constexpr int kEvictBins = 256;
constexpr int kEvictMaxCluster = 8;
// Moves per CTA that the select kernel makes itself where its CTAs do not fill
// the GPU: one round of rows for its warps; more are spread by the move kernel.
constexpr int kEvictOwnMoves = 64;

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

// ---- clusters -------------------------------------------------------------
// Four words at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint4 cluster_words(const uint32_t* local, int rank) {
    uint32_t addr;
    uint4 v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Exclusive prefix over the counts of a chunk's rows of kThreads tokens, warp
// by warp: line[row * kWarps + warp], `held` rows of them, read by every warp
// for itself.  at(before, row) is the prefix at this warp's count of that row.
template <int kWarps>
struct RowPrefix {
    static constexpr int kPer = kEvictKeys * kWarps / 32;        // counts of a lane
    static_assert(kWarps % kPer == 0, "a warp's counts sit at the same place in their lanes' shares");
    uint32_t before, total;
    __device__ __forceinline__ RowPrefix(const uint32_t* line, int held) {
        const int lane = threadIdx.x & 31, own = (threadIdx.x >> 5) % kPer;
        uint32_t v[kPer], sum = 0, part = 0;
        // a lane's counts are of one row; read in whole words, where single
        // ones would meet in the same banks
        if constexpr (kPer == 8) {
            const uint4 a = reinterpret_cast<const uint4*>(line)[2 * lane], b = reinterpret_cast<const uint4*>(line)[2 * lane + 1];
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            static_assert(kPer == 2, "8 or 32 warps");
            const uint2 a = reinterpret_cast<const uint2*>(line)[lane];
            v[0] = a.x, v[1] = a.y;
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (lane * kPer >= held * kWarps) v[k] = 0;
            part += k < own ? v[k] : 0u;
            sum += v[k];
        }
        uint32_t incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += u;
        }
        before = incl - sum + part;
        total = __shfl_sync(0xffffffffu, incl, 31);
    }
    __device__ __forceinline__ static uint32_t at(uint32_t before, int row) {
        return __shfl_sync(0xffffffffu, before, (row * kWarps + (threadIdx.x >> 5)) / kPer);
    }
};

// ---- moves ----------------------------------------------------------------
// Moves [n0, n1) of the lists, at most kMost: K and V rows, weight and
// position of each mover into its gap.  The rows' addresses go through shared
// memory first, so that a thread then has eight 16-byte loads in flight.
template <int kMost>
struct MoveRows {
    int64_t src[kMost], dst[kMost];
};

template <int kThreads, int kMost>
__device__ __forceinline__ void move_rows(const EvictParams& p, const EvictSeq& s, int b, int g,
                                          size_t pair, const int32_t* gaps, const int32_t* movers,
                                          int n0, int n1, MoveRows<kMost>& rows) {
    const int tid = threadIdx.x, vecs = p.row_bytes / 16, count = n1 - n0;
    const int32_t* table = p.block_tables + (size_t)b * p.max_blocks_per_seq;
    __syncthreads();                            // the previous batch's reads of rows
    for (int i = tid; i < count; i += kThreads) {
        const int from = movers[n0 + i], to = gaps[n0 + i];
        p.weights_out[pair * p.stride + to] = p.weights[pair * p.stride + from];
        p.positions_out[pair * p.stride + to] = evict_position(s, p.positions + pair * p.stride, from);
        const int fb = table[from / p.block_size], tb = table[to / p.block_size];
        const bool ok = fb >= 0 && fb < p.num_blocks && tb >= 0 && tb < p.num_blocks;
        if (!ok) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
        rows.src[i] = ok ? (((int64_t)fb * p.block_size + from % p.block_size) * p.num_kv_heads + g) * vecs : -1;
        rows.dst[i] = (((int64_t)tb * p.block_size + to % p.block_size) * p.num_kv_heads + g) * vecs;
    }
    __syncthreads();
    // items of a batch: move, K or V, 16-byte vector (vecs is 8 or 16)
    const int items = count * 2 * vecs, shift = vecs == 16 ? 4 : 3;
    for (int i0 = tid; i0 < items; i0 += 8 * kThreads) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= items || rows.src[i >> (shift + 1)] < 0) continue;
            const uint4* cache = static_cast<const uint4*>((i >> shift) & 1 ? p.v_cache : p.k_cache);
            v[k] = cache[rows.src[i >> (shift + 1)] + (i & (vecs - 1))];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= items || rows.src[i >> (shift + 1)] < 0) continue;
            uint4* cache = static_cast<uint4*>((i >> shift) & 1 ? p.v_cache : p.k_cache);
            cache[rows.dst[i >> (shift + 1)] + (i & (vecs - 1))] = v[k];
        }
    }
}

// ---- select ---------------------------------------------------------------
// Grid (KV heads * cluster, sequences): which tokens stay, the gap and mover
// lists, the state of the tokens that stay in place, and few moves.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : 1)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kWarps = kThreads / 32, kChunk = kThreads * kEvictKeys;
    __shared__ __align__(16) uint32_t hist[4][kEvictBins], joint[4][kEvictBins];
    __shared__ __align__(16) uint32_t counts[4];    // below left: above T, equal to T; past left: the same
    __shared__ int4 found[4];                   // per digit: it, tokens above its bin and inside
    __shared__ __align__(16) uint32_t line[2][kEvictKeys * kWarps];
    __shared__ int32_t own_gaps[kThreads], own_movers[kThreads];
    __shared__ MoveRows<kThreads> rows;
    const int C = p.cluster, rank = blockIdx.x % C;
    const int g = blockIdx.x / C, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 4 * kEvictBins / 4; i += kThreads)
        reinterpret_cast<uint4*>(&hist[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < 4) counts[tid] = 0;
    grid_dependency_wait();
    allow_dependent_launch();
    const EvictSeq s = evict_sequence(p, b, tid == 0 && blockIdx.x == 0);
    const size_t pair = (size_t)b * p.num_kv_heads + g;
    const float* w = p.weights + pair * p.stride;
    const int32_t* pos = p.positions + pair * p.stride;
    float* wo = p.weights_out + pair * p.stride;
    int32_t* po = p.positions_out + pair * p.stride;
    if (blockIdx.x == 0 && tid == 0) p.new_lens[b] = s.left;
    // this CTA's slice, in chunks that fit the registers
    const int slice = ((s.L + C - 1) / C + 31) / 32 * 32;
    const int lo = min(rank * slice, s.L), hi = min(lo + slice, s.L);
    if (s.left == s.L) {
        if (rank == 0 && tid == 0) p.num_moves[pair] = 0;
        const bool copy = p.weights_out != p.weights, move = p.positions_out != p.positions;
        for (int i = lo + tid; i < hi; i += kThreads) {
            if (copy) wo[i] = w[i];
            if (move || i >= s.known) po[i] = evict_position(s, pos, i);
        }
        return;
    }
    const int newest = (int)max((int64_t)s.seen - p.recent, (int64_t)INT32_MIN);
    uint32_t key[kEvictKeys];
    // rows of kThreads tokens that the chunk at c0 has
    auto rows_of = [&](int c0) { return min(kEvictKeys, (hi - c0 + kThreads - 1) / kThreads); };
    // positions, weights and images of tokens c0 + tid, + kThreads, ...; all
    // loads requested before the first is used
    int at[kEvictKeys];
    float x[kEvictKeys];
    auto load = [&](int c0) {
        const int n = rows_of(c0), known = min(hi, s.known), ahead = s.seen - s.L;
#pragma unroll
        for (int e = 0; e < kEvictKeys; ++e) {
            if (e >= n) break;
            const int i = c0 + e * kThreads + tid;
            at[e] = i < known ? pos[i] : i + ahead;
            x[e] = i < hi ? w[i] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < kEvictKeys; ++e) {
            if (e >= n) break;
            key[e] = at[e] < p.sinks || at[e] >= newest ? kProtected : weight_image(x[e]);
        }
    };
    auto barrier = [&] {
        if (C > 1) cluster_barrier();
        else __syncthreads();
    };
    const bool once = hi - lo <= kChunk;
    if (once) load(lo);
    __syncthreads();                            // histograms cleared
    // T, the image of the left-th largest, and how many of its equals stay
    uint32_t T = 0, want = s.left, inside = 0;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int c0 = lo; c0 < hi; c0 += kChunk) {
            if (!once) load(c0);
            const int n = rows_of(c0);
#pragma unroll
            for (int e = 0; e < kEvictKeys; ++e) {
                if (e >= n) break;
                if (c0 + e * kThreads + tid < hi && (pass == 0 || (key[e] ^ T) >> shift < 256u))
                    atomicAdd(&hist[pass][(key[e] >> shift) & 255u], 1u);
            }
        }
        barrier();
        if (C > 1) {                            // the cluster's sum
            if (tid < kEvictBins / 4) {
                uint4 sum = make_uint4(0u, 0u, 0u, 0u);
                for (int r = 0; r < C; ++r) {
                    const uint4 v = cluster_words(&hist[pass][4 * tid], r);
                    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                }
                *reinterpret_cast<uint4*>(&joint[pass][4 * tid]) = sum;
            }
            __syncthreads();
        }
        // one warp: bins from the top one down, eight to a lane
        if (warp == 0) {
            const uint4* low = reinterpret_cast<const uint4*>(&(C > 1 ? joint : hist)[pass][kEvictBins - 8 * (lane + 1)]);
            const uint4 v0 = low[0], v1 = low[1];
            const uint32_t bins[8] = {v1.w, v1.z, v1.y, v1.x, v0.w, v0.z, v0.y, v0.x};
            uint32_t sum = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += bins[k];
            uint32_t above = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, above, d);
                if (lane >= d) above += u;
            }
            const bool mine = above >= want && above - sum < want;
            above -= sum;
            int digit = 255 - 8 * lane;
            uint32_t in = bins[0];
#pragma unroll
            for (int k = 1; k < 8; ++k) {           // as long as the bin ends before the want-th
                const bool past = above + in < want && digit == 256 - 8 * lane - k;
                if (past) above += in, in = bins[k], --digit;
            }
            if (mine) found[pass] = make_int4(digit, (int)above, (int)in, 0);
        }
        __syncthreads();
        const int4 f = found[pass];
        T |= (uint32_t)f.x << shift;
        want -= f.y;
        inside = f.z;
        // the whole bin stays: its lower bits do not matter
        if (inside == want) break;
    }
    // where every equal stays, none needs its rank among them
    const bool ranked = inside != want;
    // the slices before this one: their equals, gaps and movers
    uint32_t equal = 0, n_gaps = 0, n_movers = 0, moves = 0;
    if (C > 1) {
        uint32_t n[4] = {0, 0, 0, 0};
        for (int c0 = lo; c0 < hi; c0 += kChunk) {
            if (!once) load(c0);
            const int held = rows_of(c0);
#pragma unroll
            for (int e = 0; e < kEvictKeys; ++e) {
                if (e >= held) break;
                const int i = c0 + e * kThreads + tid;
                const int past = i >= s.left ? 2 : 0;
                const bool gt = i < hi && key[e] > T, eq = i < hi && key[e] == T;
#pragma unroll
                for (int q = 0; q < 4; ++q) n[q] += (q & 2) == past && (q & 1 ? eq : gt);
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t t = __reduce_add_sync(0xffffffffu, n[q]);
            if (lane == 0) atomicAdd(&counts[q], t);
        }
        cluster_barrier();
        uint32_t seen_equal = 0;
        for (int r = 0; r < C; ++r) {
            const uint4 c = cluster_words(counts, r);
            const int r0 = min(r * slice, s.L), r1 = min(r0 + slice, s.L);
            const uint32_t below = max(0, min(r1, s.left) - r0);
            // equals stay from the lowest index on
            const uint32_t free = want > seen_equal ? want - seen_equal : 0u;
            const uint32_t eq_below = min(free, c.y), eq_past = min(free - eq_below, c.w);
            if (r < rank) equal += c.y + c.w, n_gaps += below - c.x - eq_below, n_movers += c.z + eq_past;
            moves += below - c.x - eq_below;
            seen_equal += c.y + c.w;
        }
    }
    // gaps below left and movers from left on, in order
    int32_t* gaps = p.moves + pair * 2 * p.moves_stride;
    int32_t* movers = gaps + p.moves_stride;
    for (int c0 = lo; c0 < hi; c0 += kChunk) {
        if (!once) load(c0);
        if (c0 > lo) __syncthreads();           // the previous chunk's reads of line
        const int held = rows_of(c0);
        uint32_t equals_before = 0;             // of this warp's rows, by lane
        if (ranked) {
            // rank among the equals: rows of kThreads tokens, warps, lanes
#pragma unroll
            for (int e = 0; e < kEvictKeys; ++e) {
                if (e >= held) break;
                const uint32_t eq = __ballot_sync(0xffffffffu, c0 + e * kThreads + tid < hi && key[e] == T);
                if (lane == 0) line[0][e * kWarps + warp] = __popc(eq);
            }
            __syncthreads();
            const RowPrefix<kWarps> ranks(line[0], held);
            equals_before = equal + ranks.before;
            equal += ranks.total;
        }
        uint32_t gap_bits = 0, mover_bits = 0;
#pragma unroll
        for (int e = 0; e < kEvictKeys; ++e) {
            if (e >= held) break;
            const int i = c0 + e * kThreads + tid;
            const bool in = i < hi, is_eq = in && key[e] == T;
            bool keep = in && key[e] >= T;
            if (ranked) {
                const uint32_t eq = __ballot_sync(0xffffffffu, is_eq);
                const uint32_t first = RowPrefix<kWarps>::at(equals_before, e);
                if (is_eq) keep = first + __popc(eq & ((1u << lane) - 1u)) < want;
            }
            const bool gap = in && i < s.left && !keep, mover = keep && i >= s.left;
            const uint32_t gap_mask = __ballot_sync(0xffffffffu, gap), mover_mask = __ballot_sync(0xffffffffu, mover);
            gap_bits |= (uint32_t)gap << e, mover_bits |= (uint32_t)mover << e;
            // both counts of a chunk fit 16 bits
            if (lane == 0) line[1][e * kWarps + warp] = __popc(gap_mask) | (__popc(mover_mask) << 16);
            if (keep && i < s.left) {
                if (p.weights_out != p.weights) wo[i] = x[e];
                if (p.positions_out != p.positions || i >= s.known) po[i] = at[e];
            }
        }
        __syncthreads();
        const RowPrefix<kWarps> counted(line[1], held);
#pragma unroll
        for (int e = 0; e < kEvictKeys; ++e) {
            if (e >= held) break;
            const int i = c0 + e * kThreads + tid;
            const uint32_t before = RowPrefix<kWarps>::at(counted.before, e);
            const uint32_t gap_mask = __ballot_sync(0xffffffffu, (gap_bits >> e) & 1u);
            const uint32_t mover_mask = __ballot_sync(0xffffffffu, (mover_bits >> e) & 1u);
            if ((gap_bits >> e) & 1u) {
                const int n = n_gaps + (before & 0xffffu) + __popc(gap_mask & ((1u << lane) - 1u));
                gaps[n] = i;
                if (n < kThreads) own_gaps[n] = i;
            }
            if ((mover_bits >> e) & 1u) {
                const int n = n_movers + (before >> 16) + __popc(mover_mask & ((1u << lane) - 1u));
                movers[n] = i;
                if (n < kThreads) own_movers[n] = i;
            }
        }
        n_gaps += counted.total & 0xffffu, n_movers += counted.total >> 16;
    }
    if (C == 1) moves = n_gaps;
    const bool own = (int64_t)moves <= (int64_t)p.own_moves * C;
    if (rank == 0 && tid == 0) p.num_moves[pair] = own ? 0 : moves;
    // the lists are complete; also no CTA leaves while another reads its shared memory
    barrier();
    if (!own) return;
    const int per = ((int)moves + C - 1) / C, n0 = min(rank * per, (int)moves), n1 = min(n0 + per, (int)moves);
    // a CTA of its own has the first of the lists in shared memory
    const bool here = C == 1 && (int)moves <= kThreads;
    for (int n = n0; n < n1; n += kThreads)
        move_rows<kThreads, kThreads>(p, s, b, g, pair, here ? own_gaps : gaps, here ? own_movers : movers, n,
                                      min(n + kThreads, n1), rows);
}

// 32 moves to 128 threads (17 us of 16 prompts' cut, 116 MB read and written,
// near the copy rate): with the select of then 29.5 us in all; 64 to 256 31.1,
// 128 to 512 33.6, 16 to 128 33.1.
constexpr int kMoveThreads = 128, kMoveBatch = 32;

// Grid (move batches, KV heads, sequences).  The count, the lists and the
// lengths are requested together; what lies past the count is not used.
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const __grid_constant__ EvictParams p) {
    __shared__ MoveRows<kMoveBatch> rows;
    __shared__ int32_t gaps[kMoveBatch], movers[kMoveBatch];
    grid_dependency_wait();
    allow_dependent_launch();
    const int g = blockIdx.y, b = blockIdx.z;
    const size_t pair = (size_t)b * p.num_kv_heads + g;
    const int n0 = blockIdx.x * kMoveBatch, total = p.num_moves[pair];
    const int32_t* lists = p.moves + pair * 2 * p.moves_stride + n0;
    for (int i = threadIdx.x; i < min(kMoveBatch, p.moves_stride - n0); i += kMoveThreads)
        gaps[i] = lists[i], movers[i] = lists[p.moves_stride + i];
    const EvictSeq s = evict_sequence(p, b, false);
    if (n0 >= total) return;
    __syncthreads();
    move_rows<kMoveThreads, kMoveBatch>(p, s, b, g, pair, gaps, movers, 0, min(kMoveBatch, total - n0), rows);
}

template <int kThreads>
cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t stream) {
    return launch_clusters(evict_select_kernel<kThreads>, dim3(p.cluster),
                           dim3(p.num_kv_heads * p.cluster, p.num_seqs), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_evict(const EvictParams& params, cudaStream_t stream) {
    EvictParams p = params;
    // What the tables can hold decides: 256 threads where that fits their
    // registers (four such CTAs share an SM; 64 x 8 rows of 1040 tokens 11.1
    // us, 128 threads of 16 images 13.8), else 1024, and a cluster that holds
    // the longest context in registers, up to the portable size (16 x 8 rows
    // of up to 8192 25.3 us with the moves in a graph, 28 called on cold caches).
    const int64_t longest = (int64_t)p.max_blocks_per_seq * p.block_size;
    const bool small = longest <= 256 * kEvictKeys;
    const int64_t ctas = (longest + 1024 * kEvictKeys - 1) / (1024 * kEvictKeys);
    p.cluster = small ? 1 : (int)(ctas < kEvictMaxCluster ? ctas : kEvictMaxCluster);
    // Rows that fill three quarters of the SMs' select CTAs move everything
    // themselves, those done early beside the others' selects (128 rows of up
    // to 8192, in a graph, 25.3 us, with the move kernel 27.5; 64 rows 22.6
    // against 19.2).
    const int64_t pairs = (int64_t)p.num_seqs * p.num_kv_heads;
    p.own_moves = !small && p.cluster == 1 && pairs >= 114 ? INT32_MAX : kEvictOwnMoves;
    cudaError_t e = small ? launch_evict_select<256>(p, stream) : launch_evict_select<1024>(p, stream);
    if (e != cudaSuccess || p.moves_stride <= (int64_t)p.own_moves * p.cluster) return e;
    const dim3 grid((p.moves_stride + kMoveBatch - 1) / kMoveBatch, p.num_kv_heads, p.num_seqs);
    return launch_with_pdl(evict_move_kernel, grid, dim3(kMoveThreads), 0, stream, p);
}

}  // namespace pa
