// Attention weights that a prefill chunk's queries give to the cached tokens,
// on the fifth-generation tensor cores (tcgen05, tensor-memory accumulators).
//
// Sequence b holds L tokens, the last C of which are new; the counted queries
// are the chunk's last W (window; all C without one), counted query i at
// position L - W + i seeing the tokens up to itself:
//   weights[b][g][j] (+)= sum over the group's heads h and the counted i with
//                         position >= j of softmax_j(scale q_ih . K_j)
// A column of the softmax matrix is wanted, and its rows' sums are known only
// at the end of the row, so Q K^T is formed twice, each time with the axis
// that is summed along the columns of tensor memory, where one thread owns a
// whole row of the tile and no exchange between lanes is needed:
//   pass 1: 128 query rows (tokens x heads of the group) in the lanes, key
//           tiles streamed: row maximum m (raised lazily, threshold 2^8) and
//           sum z of 2^(x - m), kept as lse = m + log2 z;
//   pass 2: 128 keys in the lanes, query tiles streamed: the sum over the
//           columns of 2^(x - lse), x = scale log2(e) q . K in fp32.
// Long rows are cut into chunks of key tiles (pass 1) and of query tiles
// (pass 2) so that there are many equal units of work; a small kernel each
// joins the chunks in a fixed order.  No atomics: results do not depend on
// the schedule.
//
// Both passes are one kernel with the operands exchanged.  A unit holds one
// resident tile (operand A) and streams others (operand B); one persistent
// CTA per SM walks its units, its rings running on from one unit to the next.
// Warps 1-3 load tiles with TMA (K through the block table in 16-token boxes,
// Q in one box of tokens x heads), warp 0 issues the MMAs into four
// 128-column buffers, and four groups of four warps take the finished tiles
// in turn.  Rows of Q past a sequence's chunk and K rows past its end may
// hold anything: they only reach their own lane or column, which is masked.
//
// Every mbarrier wait gives up after 1 s and flags PA_DEVERR_WAIT_TIMEOUT;
// the epilogue warps then run their remaining steps without waiting, and
// tensor memory is always released.
#include <algorithm>

#include "bounded_internal.h"
#include "decode_tile.cuh"
#include "tc_device.cuh"

namespace pa {

constexpr int kPwRows = 128;                   // lanes: rows of the resident tile
constexpr int kPwCols = 128;                   // columns: rows of a streamed tile
constexpr int kPwBufs = 4;                     // accumulators in tensor memory
constexpr int kPwProducers = 3;                // warps that load
constexpr int kPwGroups = 4;                   // epilogue groups of four warps, one per buffer
constexpr int kPwThreads = (1 + kPwProducers + 4 * kPwGroups) * 32;
constexpr int kPwJoinThreads = 256;

template <int D>
struct PwLayout {
    static constexpr int kHalf = kPwRows * 128;               // 64 dims of 128 rows
    static constexpr int kHalves = D / kBoxElems;
    static constexpr int kTile = kHalves * kHalf;
    static constexpr int kStages = 6;                         // of both rings
    static constexpr int kDynamicSmem = kStages * kTile + 1024;
};

struct PwSeq {
    int L, C, counted;             // context, chunk, counted queries
    int64_t q0;                    // row of the first counted query in q
    int n_qt, n_kt;                // query and key tiles
};

__device__ __forceinline__ void pw_sequence(const PrefillWeightsParams& p, int b, bool report,
                                            PwSeq& s) {
    int L = p.context_lens[b];
    const int64_t start = p.query_start[b];
    int64_t C = (int64_t)p.query_start[b + 1] - start;
    bool bad = false;
    if (L < 0 || L > p.max_context) bad = true, L = L < 0 ? 0 : p.max_context;
    if (C < 0 || C > L) bad = true, C = C < 0 ? 0 : L;
    if (start < 0 || start + C > p.num_tokens) bad = true, C = 0;
    s.L = L, s.C = (int)C;
    s.counted = p.window > 0 ? min(p.window, s.C) : s.C;
    if (s.counted > p.max_counted) bad = true, s.counted = p.max_counted;
    s.q0 = start + s.C - s.counted;
    s.n_qt = (s.counted + p.tile_tokens - 1) / p.tile_tokens;
    s.n_kt = (L + kPwCols - 1) / kPwCols;
    if (bad && report) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
}

// Key tiles that query tile qt sees, and the first query tile that sees any
// key of tile kt.
__device__ __forceinline__ int pw_key_tiles(const PrefillWeightsParams& p, const PwSeq& s, int qt) {
    const int last = min((qt + 1) * p.tile_tokens, s.counted) - 1;
    return (s.L - s.counted + last) / kPwCols + 1;
}

__device__ __forceinline__ int pw_first_query_tile(const PrefillWeightsParams& p, const PwSeq& s,
                                                   int kt) {
    return max(0, kt * kPwCols - (s.L - s.counted)) / p.tile_tokens;
}

// One unit: resident tile `a` of (b, g), streamed tiles [first, last).
struct PwUnit {
    int b, g, a, chunk, first, last;
};

// Walks the units u = blockIdx.x, + gridDim.x, ... in order (their number
// fits 31 bits: checked on the host).  All lanes of a warp walk together;
// the unit's fields are broadcast so that what depends on them is known to be
// uniform.
template <bool kStats>
struct PwWalk {
    int b = -1;
    unsigned u, base = 0, count = 0;
    PwSeq s;

    __device__ __forceinline__ PwWalk() : u(blockIdx.x) {}

    __device__ __forceinline__ bool next(const PrefillWeightsParams& p, PwUnit& U) {
        while (u >= base + count) {
            base += count;
            if (++b >= p.num_seqs) return false;
            pw_sequence(p, b, kStats && blockIdx.x == 0 && threadIdx.x == 0, s);
            count = kStats ? s.n_qt * ((s.n_kt + p.key_chunk - 1) / p.key_chunk)
                           : s.n_kt * max(1, (s.n_qt + p.query_chunk - 1) / p.query_chunk);
            count = __shfl_sync(0xffffffffu, count * p.num_kv_heads, 0);
        }
        const unsigned r = u - base, rest = r / (unsigned)p.num_kv_heads;
        u += gridDim.x;
        const unsigned tiles = kStats ? s.n_qt : s.n_kt;
        U.b = b;
        U.g = __shfl_sync(0xffffffffu, (int)(r - rest * (unsigned)p.num_kv_heads), 0);
        U.chunk = __shfl_sync(0xffffffffu, (int)(rest / tiles), 0);
        U.a = __shfl_sync(0xffffffffu, (int)(rest % tiles), 0);
        if (kStats) {
            U.first = U.chunk * p.key_chunk;
            U.last = min(U.first + p.key_chunk, pw_key_tiles(p, s, U.a));
        } else {
            U.first = max(U.chunk * p.query_chunk, pw_first_query_tile(p, s, U.a));
            U.last = min((U.chunk + 1) * p.query_chunk, s.n_qt);
        }
        U.first = __shfl_sync(0xffffffffu, U.first, 0);
        U.last = __shfl_sync(0xffffffffu, U.last, 0);
        return true;
    }
};

__device__ __forceinline__ float sum8(const uint64_t (&ps)[4]) {
    float t[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) f32x2_unpack(ps[e], t[2 * e], t[2 * e + 1]);
    return ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
}

// (m, z) and another chunk's: the maximum, and the sum taken against it.
__device__ __forceinline__ void join_stats(float& m, float& z, float2 o) {
    const float n = fmaxf(m, o.x), ref = n == -INFINITY ? 0.f : n;
    z = z * ex2(m - ref) + o.y * ex2(o.x - ref);
    m = n;
}

// Pass 2: adds 2^(x - lse) over the tile's columns (of [lo, hi) with kMask);
// `neg_lse` in shared memory, `release` called once the tile is read.
template <bool kMask, typename Release>
__device__ __forceinline__ void column_sums(uint64_t (&ps)[4], uint32_t tile_addr, const float* neg_lse,
                                            uint64_t sl2, int lo, int hi, Release&& release) {
#pragma unroll
    for (int c = 0; c < kPwCols; c += 32) {
        uint32_t v[32];
        tmem_ld32(tile_addr + c, v);
        tmem_wait_ld();
        if (c == kPwCols - 32) release();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const float4 l = *reinterpret_cast<const float4*>(neg_lse + c + e);
            float a[4];
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sl2,
                                   f32x2_pack(l.x, l.y)), a[0], a[1]);
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), sl2,
                                   f32x2_pack(l.z, l.w)), a[2], a[3]);
            if (kMask) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[i] = c + e + i >= lo && c + e + i < hi ? a[i] : -INFINITY;
            }
            ps[(e >> 1) & 3] = f32x2_add(ps[(e >> 1) & 3], f32x2_pack(ex2(a[0]), ex2(a[1])));
            ps[((e >> 1) + 1) & 3] = f32x2_add(ps[((e >> 1) + 1) & 3], f32x2_pack(ex2(a[2]), ex2(a[3])));
        }
    }
}

template <typename T, int D, bool kStats>
__global__ void __launch_bounds__(kPwThreads, 1)
    prefill_weights_kernel(const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_q,
                           const __grid_constant__ PrefillWeightsParams p) {
    using Lay = PwLayout<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    // resident tiles wait for a whole unit, unless units are single steps
    constexpr int kA = kStats ? 2 : 3, kB = Lay::kStages - kA;
    __shared__ __align__(8) uint64_t a_full[kA], a_empty[kA], b_full[kB], b_empty[kB];
    __shared__ __align__(8) uint64_t s_full[kPwBufs], s_empty[kPwBufs];
    __shared__ uint32_t tmem_base;
    __shared__ __align__(16) float lse_s[kPwGroups][2][kPwCols];     // pass 2: [group][tile parity]
    __shared__ float2 other[2][kPwGroups - 1][kPwRows];              // the other groups' results
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int G = p.group;
    const int q_rows = p.tile_tokens * G;                    // rows of a query tile, <= 128
    // K tiles are loaded by every producer warp, Q tiles by the first
    constexpr int kALoaders = kStats ? 1 : kPwProducers, kBLoaders = kStats ? kPwProducers : 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kA; ++i) mbar_init(&a_full[i], kALoaders), mbar_init(&a_empty[i], 1);
        for (int i = 0; i < kB; ++i) mbar_init(&b_full[i], kBLoaders), mbar_init(&b_empty[i], 1);
        for (int i = 0; i < kPwBufs; ++i) mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], 4);
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(&tmem_base, kPwBufs * kPwCols);
    if (!kStats && q_rows < kPwCols) {
        // rows that no query box fills stay zero (their lse is +inf)
        for (int i = threadIdx.x; i < kB * Lay::kTile / 16; i += kPwThreads)
            reinterpret_cast<uint4*>(smem + kA * Lay::kTile)[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    grid_dependency_wait();
    allow_dependent_launch();

    if (warp >= 1 && warp <= kPwProducers) {
        // ------------------------------------------------------------------
        // producers: all lanes run along, one issues
        // ------------------------------------------------------------------
        const int who = warp - 1;
        if (lane == 0) prefetch_tensor_map(who == 0 ? &tmap_q : &tmap_k);
        // waits for stage n % stages to be free
        auto open = [&](uint64_t* empty, int stages, int n) -> bool {
            return n < stages || __all_sync(0xffffffffu, mbar_wait(&empty[n % stages], ((n / stages) - 1) & 1));
        };
        auto blocks_of = [&](const PwSeq& s, int b, int kt) {     // lane i: block of box i
            const int tok = kt * kPwCols + 16 * lane;
            if (lane >= 8 || tok >= s.L) return 0;
            const int blk = __ldg(p.block_tables + (size_t)b * p.max_blocks_per_seq + tok / p.block_size);
            if (blk < 0 || blk >= p.num_blocks) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
            return blk;
        };
        // this warp's boxes of a K tile: every kPwProducers-th
        auto load_k = [&](uint8_t* dst, uint64_t* full, uint64_t* empty, int stages, int n,
                          const PwSeq& s, const PwUnit& U, int kt, int blk) -> bool {
            if (!open(empty, stages, n)) return false;
            const int nbox = __shfl_sync(0xffffffffu, min(8, (s.L - kt * kPwCols + 15) / 16), 0);
            const int own = nbox > who ? (nbox - who + kPwProducers - 1) / kPwProducers : 0;
            uint64_t* bar = &full[n % stages];
            if (elect_one()) mbar_arrive_expect_tx(bar, (uint32_t)(own * Lay::kHalves * kBox16Bytes));
            __syncwarp();
            dst += (n % stages) * Lay::kTile;
#pragma unroll
            for (int i = 0; i < (8 + kPwProducers - 1) / kPwProducers; ++i) {
                const int box = who + i * kPwProducers;
                if (box >= nbox) break;
                const int pblk = __shfl_sync(0xffffffffu, blk, box);
                const int sub = (kt * kPwCols + 16 * box) % p.block_size;
                if (elect_one()) {
#pragma unroll
                    for (int h = 0; h < Lay::kHalves; ++h)
                        tma_load_4d(dst + h * Lay::kHalf + box * kBox16Bytes, &tmap_k, bar,
                                    h * kBoxElems, U.g, sub, pblk);
                }
                __syncwarp();
            }
            return true;
        };
        auto load_q = [&](uint8_t* dst, uint64_t* full, uint64_t* empty, int stages, int n,
                          const PwSeq& s, const PwUnit& U, int qt) -> bool {
            if (!open(empty, stages, n)) return false;
            uint64_t* bar = &full[n % stages];
            const int row = __shfl_sync(0xffffffffu, (int)(s.q0 + (int64_t)qt * p.tile_tokens), 0);
            dst += (n % stages) * Lay::kTile;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar, (uint32_t)(q_rows * Lay::kHalves * 128));
#pragma unroll
                for (int h = 0; h < Lay::kHalves; ++h)
                    tma_load_3d(dst + h * Lay::kHalf, &tmap_q, bar, h * kBoxElems, U.g * G, row);
            }
            __syncwarp();
            return true;
        };
        uint8_t* a_ring = smem;
        uint8_t* b_ring = smem + kA * Lay::kTile;
        PwWalk<kStats> walk;
        PwUnit U;
        int na = 0, nb = 0, at_b = -1, at_g = -1, at_qt = -1;
        bool ok = true;
        while (ok && walk.next(p, U)) {
            if (U.first >= U.last) continue;
            if constexpr (kStats) {
                int blk = blocks_of(walk.s, U.b, U.first);
                if (who == 0) ok = load_q(a_ring, a_full, a_empty, kA, na++, walk.s, U, U.a);
                for (int kt = U.first; ok && kt < U.last; ++kt) {
                    const int now = blk;                     // the next tile's blocks a step ahead
                    if (kt + 1 < U.last) blk = blocks_of(walk.s, U.b, kt + 1);
                    ok = load_k(b_ring, b_full, b_empty, kB, nb++, walk.s, U, kt, now);
                }
            } else {
                ok = load_k(a_ring, a_full, a_empty, kA, na++, walk.s, U, U.a,
                            blocks_of(walk.s, U.b, U.a));
                for (int qt = U.first; ok && who == 0 && qt < U.last; ++qt) {
                    if (U.b == at_b && U.g == at_g && qt == at_qt) continue;     // still there
                    at_b = U.b, at_g = U.g, at_qt = qt;
                    ok = load_q(b_ring, b_full, b_empty, kB, nb++, walk.s, U, qt);
                }
            }
        }
        if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    } else if (warp == 0) {
        // ------------------------------------------------------------------
        // MMA issuer: all lanes run along, one issues
        // ------------------------------------------------------------------
        constexpr uint32_t kId = idesc_f16(kPwRows, kPwCols, kBf16, false);
        const uint64_t a_ring = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t b_ring = smem_desc_sw128(smem_u32(smem) + kA * Lay::kTile, 16, 1024);
        PwWalk<kStats> walk;
        PwUnit U;
        int na = 0, nb = -1, step = 0, at_b = -1, at_g = -1, at_qt = -1;
        bool ok = true;
        auto wait = [&](uint64_t* bar, int phase) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, phase & 1));
        };
        while (ok && walk.next(p, U)) {
            if (U.first >= U.last) continue;
            wait(&a_full[na % kA], na / kA);
            for (int i = U.first; ok && i < U.last; ++i, ++step) {
                if (kStats || U.b != at_b || U.g != at_g || i != at_qt) {
                    // the previous streamed tile is free once the products so far are done
                    if (nb >= 0 && elect_one()) mma_commit(&b_empty[nb % kB]);
                    __syncwarp();
                    ++nb;
                    at_b = U.b, at_g = U.g, at_qt = i;
                    wait(&b_full[nb % kB], nb / kB);
                }
                if (step >= kPwBufs) wait(&s_empty[step % kPwBufs], step / kPwBufs - 1);
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t a = a_ring + (na % kA) * (Lay::kTile >> 4);
                const uint64_t b = b_ring + (nb % kB) * (Lay::kTile >> 4);
                const uint32_t d = tmem + kPwCols * (step % kPwBufs);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        constexpr int kHalf16 = Lay::kHalf >> 4;
                        const uint64_t off = (kk >> 2) * kHalf16 + (kk & 3) * 2;
                        mma_f16_ss(d, a + off, b + off, kId, kk > 0);
                    }
                    mma_commit(&s_full[step % kPwBufs]);
                }
                __syncwarp();
            }
            if (ok && elect_one()) mma_commit(&a_empty[na % kA]);
            __syncwarp();
            ++na;
        }
        if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    } else {
        // ------------------------------------------------------------------
        // epilogue: group w takes the steps w, w + 4, ... (buffer w); this
        // thread owns lane r of every tile
        // ------------------------------------------------------------------
        const int group = (warp >> 2) - 1;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t tile_addr = tmem + kPwCols * group + ((uint32_t)((warp & 3) * 32) << 16);
        const float sl = p.scale_log2;
        const uint64_t sl2 = f32x2_pack(sl, sl);
        bool failed = false;
        auto wait = [&](int n) {                // the group's n-th tile
            if (!failed && !__all_sync(0xffffffffu, mbar_wait(&s_full[group], n & 1))) failed = true;
            tc_fence_after_sync();
        };
        auto release = [&] {                    // the tile is in registers
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[group]);
        };
        PwWalk<kStats> walk;
        PwUnit U;
        int step = 0, units = 0, mine = 0;
        while (walk.next(p, U)) {
            const PwSeq& s = walk.s;
            const int steps = max(0, U.last - U.first);
            if (kStats && steps == 0) continue;
            const size_t pair = (size_t)U.b * p.num_kv_heads + U.g;
            const int key = U.a * kPwCols + r;
            // a unit of one step is its group's alone, others are joined by group 0
            const bool writer = steps == 1 ? (step & (kPwGroups - 1)) == group : group == 0;
            float before = 0.f;
            if (!kStats && writer && p.query_chunks == 1 && p.weights && key < s.L - s.C)
                before = p.weights[pair * p.weights_stride + key];
            float m = -INFINITY, z = 0.f;
            // first step of this unit that is the group's
            const int skip = (group - step) & (kPwGroups - 1);
            step += steps;
            if constexpr (kStats) {
                const int pos = min(s.L - s.counted + U.a * p.tile_tokens + r / G, s.L - 1);
                for (int kt = U.first + skip; kt < U.last; kt += kPwGroups) {
                    wait(mine++);
                    const int visible = pos - kt * kPwCols;           // keys 0 .. visible of the tile
                    const bool whole = __all_sync(0xffffffffu, visible >= kPwCols - 1);
#pragma unroll
                    for (int c = 0; c < kPwCols; c += 64) {
                        uint32_t v[64];
                        tmem_ld32(tile_addr + c, *reinterpret_cast<uint32_t(*)[32]>(v));
                        tmem_ld32(tile_addr + c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
                        tmem_wait_ld();
                        if (c == 64) release();
                        if (!whole) {
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                if (c + e > visible) v[e] = 0xff800000u;
                        }
                        float pm[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) pm[e] = __uint_as_float(v[e]);
#pragma unroll
                        for (int e = 4; e < 64; ++e) pm[e & 3] = fmaxf(pm[e & 3], __uint_as_float(v[e]));
                        const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])) * sl;
                        if (mx > m + kRescaleThresholdLog2) {         // also the first finite maximum
                            z *= ex2(m - mx);
                            m = mx;
                        }
                        const float ref = m == -INFINITY ? 0.f : m;   // nothing visible yet
                        const uint64_t neg2 = f32x2_pack(-ref, -ref);
                        uint64_t ps[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float a0, a1;
                            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])),
                                                   sl2, neg2), a0, a1);
                            ps[e & 3] = f32x2_add(ps[e & 3], f32x2_pack(ex2(a0), ex2(a1)));
                        }
                        z += sum8(ps);
                    }
                }
            } else {
                for (int qt = U.first + skip; qt < U.last; qt += kPwGroups) {
                    const float lse = p.lse[(pair * p.max_query_tiles + qt) * kPwCols + r];
                    float* ls = lse_s[group][mine & 1];
                    wait(mine++);
                    ls[r] = -lse;
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
                    const int tokens = min(p.tile_tokens, s.counted - qt * p.tile_tokens);
                    // columns that see this key: from `lo` on, up to the chunk's end
                    const int lo = (key - (s.L - s.counted + qt * p.tile_tokens)) * G, hi = tokens * G;
                    const bool whole = tokens == p.tile_tokens && __all_sync(0xffffffffu, lo <= 0);
                    uint64_t ps[4] = {0ull, 0ull, 0ull, 0ull};
                    if (whole) column_sums<false>(ps, tile_addr, ls, sl2, lo, hi, release);
                    else column_sums<true>(ps, tile_addr, ls, sl2, lo, hi, release);
                    z += sum8(ps);
                }
            }
            if (steps > 1) {
                if (group > 0) other[units & 1][group - 1][r] = make_float2(m, z);
                asm volatile("bar.sync 5, %0;" ::"n"(kPwGroups * 128) : "memory");
                if (group == 0) {
#pragma unroll
                    for (int i = 0; i < kPwGroups - 1; ++i) {
                        const float2 o = other[units & 1][i][r];
                        if (kStats) join_stats(m, z, o);
                        else z += o.y;
                    }
                }
                ++units;
            }
            if (!writer || failed) continue;
            if constexpr (kStats) {
                const int tokens = min(p.tile_tokens, s.counted - U.a * p.tile_tokens);
                const size_t at = (pair * p.max_query_tiles + U.a) * kPwRows + r;
                if (p.key_chunks == 1) p.lse[at] = r < tokens * G ? m + log2f(z) : INFINITY;
                else p.stats[(size_t)U.chunk * p.num_seqs * p.num_kv_heads * p.max_query_tiles * kPwRows + at] =
                    make_float2(m, z);
            } else if (key < s.L) {
                if (p.query_chunks == 1)
                    p.weights_out[pair * p.weights_stride + key] = before + z;
                else
                    p.columns[((size_t)U.chunk * p.num_seqs * p.num_kv_heads + pair) * p.columns_stride + key] = z;
            }
        }
        if (failed && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kPwBufs * kPwCols);
    }
}

// lse of every query row from its chunks' (m, z); +inf past the chunk.
__global__ void __launch_bounds__(kPwRows)
    prefill_stats_join_kernel(const __grid_constant__ PrefillWeightsParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int qt = blockIdx.x, g = blockIdx.y, b = blockIdx.z, r = threadIdx.x;
    PwSeq s;
    pw_sequence(p, b, false, s);
    if (qt >= s.n_qt) return;
    const size_t rows = (size_t)p.num_seqs * p.num_kv_heads * p.max_query_tiles * kPwRows;
    const size_t at = (((size_t)b * p.num_kv_heads + g) * p.max_query_tiles + qt) * kPwRows + r;
    const int chunks = (pw_key_tiles(p, s, qt) + p.key_chunk - 1) / p.key_chunk;
    float m = -INFINITY, z = 0.f;
    for (int c = 0; c < chunks; ++c) {
        join_stats(m, z, p.stats[c * rows + at]);
    }
    const int tokens = min(p.tile_tokens, s.counted - qt * p.tile_tokens);
    p.lse[at] = r < tokens * p.group ? m + log2f(z) : INFINITY;
}

// weights from the column sums of the query chunks.
__global__ void __launch_bounds__(kPwJoinThreads)
    prefill_columns_join_kernel(const __grid_constant__ PrefillWeightsParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int j = blockIdx.x * kPwJoinThreads + threadIdx.x, g = blockIdx.y, b = blockIdx.z;
    PwSeq s;
    pw_sequence(p, b, false, s);
    if (j >= s.L) return;
    const size_t pair = (size_t)b * p.num_kv_heads + g, pairs = (size_t)p.num_seqs * p.num_kv_heads;
    const size_t at = pair * p.weights_stride + j;
    float w = p.weights && j < s.L - s.C ? p.weights[at] : 0.f;
    const int first = pw_first_query_tile(p, s, j / kPwCols) / p.query_chunk;
    const int chunks = (s.n_qt + p.query_chunk - 1) / p.query_chunk;
    float sum = 0.f;
    for (int c = first; c < chunks; ++c) sum += p.columns[(c * pairs + pair) * p.columns_stride + j];
    p.weights_out[at] = w + sum;
}

size_t prefill_weights_plan(PrefillWeightsParams& p, void* workspace) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    p.tile_tokens = kPwRows / p.group;
    p.max_query_tiles = (p.max_counted + p.tile_tokens - 1) / p.tile_tokens;
    const int64_t key_tiles = ((int64_t)p.max_context + kPwCols - 1) / kPwCols;
    const int64_t pairs = (int64_t)p.num_seqs * p.num_kv_heads;
    // Pass 1 in chunks of so many key tiles that each SM gets some 16 units
    // (the batch taken at its bounds), but not below four tiles (a unit's
    // load of its queries) nor above 64; pass 2 in chunks of 16 query tiles.
    const int64_t share = pairs * p.max_query_tiles * key_tiles / (152 * 16);
    p.key_chunk = (int)std::min<int64_t>(64, std::max<int64_t>(4, share));
    p.key_chunks = (int)std::max<int64_t>(1, (key_tiles + p.key_chunk - 1) / p.key_chunk);
    p.query_chunk = 16;
    p.query_chunks = std::max(1, (p.max_query_tiles + p.query_chunk - 1) / p.query_chunk);
    p.columns_stride = (int)(key_tiles * kPwCols);
    const size_t rows = (size_t)pairs * p.max_query_tiles * kPwRows;
    char* base = static_cast<char*>(workspace);
    size_t off = 0;
    p.lse = reinterpret_cast<float*>(base);
    off += up(rows * sizeof(float) + 1);
    p.stats = reinterpret_cast<float2*>(base + off);
    if (p.key_chunks > 1) off += up(p.key_chunks * rows * sizeof(float2));
    p.columns = reinterpret_cast<float*>(base + off);
    if (p.query_chunks > 1) off += up((size_t)p.query_chunks * pairs * p.columns_stride * sizeof(float));
    return off;
}

template <typename T, int D>
cudaError_t launch_prefill_weights_t(const CUtensorMap& tmk, const CUtensorMap& tmq,
                                     const PrefillWeightsParams& p, cudaStream_t stream) {
    constexpr int smem = PwLayout<D>::kDynamicSmem;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(prefill_weights_kernel<T, D, true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(prefill_weights_kernel<T, D, false>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    const dim3 grid(sms), threads(kPwThreads);
    if (e == cudaSuccess && p.max_counted > 0) {
        e = launch_with_pdl(prefill_weights_kernel<T, D, true>, grid, threads, smem, stream, tmk, tmq, p);
        if (e == cudaSuccess && p.key_chunks > 1)
            e = launch_with_pdl(prefill_stats_join_kernel,
                                dim3(p.max_query_tiles, p.num_kv_heads, p.num_seqs), dim3(kPwRows), 0,
                                stream, p);
    }
    if (e == cudaSuccess)
        e = launch_with_pdl(prefill_weights_kernel<T, D, false>, grid, threads, smem, stream, tmk, tmq, p);
    if (e == cudaSuccess && p.query_chunks > 1)
        e = launch_with_pdl(prefill_columns_join_kernel,
                            dim3((p.max_context + kPwJoinThreads - 1) / kPwJoinThreads, p.num_kv_heads,
                                 p.num_seqs), dim3(kPwJoinThreads), 0, stream, p);
    return e;
}

cudaError_t launch_prefill_weights(int dtype, int head_dim, const CUtensorMap& tmk,
                                   const CUtensorMap& tmq, const PrefillWeightsParams& p,
                                   cudaStream_t stream) {
    if (dtype == PA_BF16)
        return head_dim == 64 ? launch_prefill_weights_t<__nv_bfloat16, 64>(tmk, tmq, p, stream)
                              : launch_prefill_weights_t<__nv_bfloat16, 128>(tmk, tmq, p, stream);
    return head_dim == 64 ? launch_prefill_weights_t<__half, 64>(tmk, tmq, p, stream)
                          : launch_prefill_weights_t<__half, 128>(tmk, tmq, p, stream);
}

}  // namespace pa
