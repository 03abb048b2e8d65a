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
// Both passes are one kernel with the operands exchanged.  A unit holds two
// resident tiles (operand A) and streams others (operand B) past both, so
// that a streamed tile is loaded once for two products; one persistent CTA
// per SM walks its units, its rings running on from one unit to the next.
// Pass 1 has three warps that load with TMA, one for each stage of the K ring
// (16-token boxes through the block table: a box costs its warp some 120
// cycles) and of the Q ring (one box of tokens x heads per 64 dims); pass 2,
// whose K tiles stay for a unit, has one warp for each ring.  Two warps issue
// the MMAs, one for each resident tile, into two 128-column buffers each: a
// single issuer spends 1,060 cycles on its waits and commits per tile, twice
// what the product takes.  Four groups of four warps take the finished tiles.
// Rows of Q past a sequence's chunk and K rows past its end may hold anything:
// they only reach their own lane or column, which is masked.
//
// Measured (chunks of 2048 and 1920 on contexts of 2048 and 16384, 32 heads
// over 8, D 128, bf16): 189 us for pass 1 and 199 for pass 2, 1.34 PFLOP/s over
// both, in a graph whose replays find part of K and Q in L2; called back to
// back on cold caches 412 to 420 us in all.  The tensor pipe is busy 62 % of the time, the exponentials' unit 64 %, issue
// slots 62 / 60 %: bound by how the four groups of epilogue warps overlap,
// whose instructions per score are few but for the exponential.
//
// Every mbarrier wait gives up after 1 s and flags PA_DEVERR_WAIT_TIMEOUT;
// the epilogue warps then run their remaining steps without waiting.  Loaders
// and issuers end only when their last copies and products have landed (or
// have not for 1 s), and tensor memory is always released.
#include <algorithm>

#include "prefill_weights.cuh"

namespace pa {

constexpr int kPwJoinThreads = 256;

// One unit of (b, g): resident tiles 2a and 2a + 1 (where there are two) and
// the streamed tiles [first, last).
struct PwUnit {
    int b, g, a, chunk, first, last;
};

// Walks the units u = blockIdx.x, + gridDim.x, ... in order (their number
// fits 31 bits: checked on the host), all lanes of a warp together.  Lane i
// holds the lengths and the unit count of sequence base_b + i, so that 32
// sequences cost one round of loads.  Pass 2 takes the sequences from the
// last on: their keys are those that pass 1 left in L2.
template <bool kStats>
struct PwWalk {
    unsigned u, base = 0;
    int base_b = -32;
    unsigned ends = 0;             // lane: units up to and with its sequence, from base on
    unsigned total = 0;
    PwSeq mine, s;

    __device__ __forceinline__ PwWalk() : u(blockIdx.x) {}

    __device__ __forceinline__ bool next(const PrefillWeightsParams& p, PwUnit& U) {
        const int lane = threadIdx.x & 31;
        while (u >= base + total) {
            base += total;
            base_b += 32;
            if (base_b >= p.num_seqs) return false;
            const int i = base_b + lane;
            unsigned count = 0;
            if (i < p.num_seqs) {
                pw_sequence(p, kStats ? i : p.num_seqs - 1 - i, (kStats || p.max_counted == 0) && blockIdx.x == 0 && threadIdx.x < 32, mine);
                count = kStats ? (mine.n_qt + 1) / 2 * ((mine.n_kt + p.key_chunk - 1) / p.key_chunk)
                               : (mine.n_kt + 1) / 2 * max(1, (mine.n_qt + p.query_chunk - 1) / p.query_chunk);
                count *= p.num_kv_heads;
            }
            ends = count;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned v = __shfl_up_sync(0xffffffffu, ends, d);
                if (lane >= d) ends += v;
            }
            total = __shfl_sync(0xffffffffu, ends, 31);
        }
        const int at = __ffs(__ballot_sync(0xffffffffu, u - base < ends)) - 1;
        const unsigned before = __shfl_sync(0xffffffffu, ends, max(at - 1, 0));
        const unsigned r = u - base - (at > 0 ? before : 0u), rest = r / (unsigned)p.num_kv_heads;
        u += gridDim.x;
        U.b = kStats ? base_b + at : p.num_seqs - 1 - (base_b + at);
        s.L = __shfl_sync(0xffffffffu, mine.L, at);
        s.C = __shfl_sync(0xffffffffu, mine.C, at);
        s.counted = __shfl_sync(0xffffffffu, mine.counted, at);
        s.q0 = __shfl_sync(0xffffffffu, mine.q0, at);
        s.n_qt = __shfl_sync(0xffffffffu, mine.n_qt, at);
        s.n_kt = __shfl_sync(0xffffffffu, mine.n_kt, at);
        U.g = r - rest * (unsigned)p.num_kv_heads;
        const unsigned tile_pairs = ((kStats ? s.n_qt : s.n_kt) + 1) / 2;
        U.chunk = rest / tile_pairs;
        U.a = rest - U.chunk * tile_pairs;
        if (kStats) {
            U.first = U.chunk * p.key_chunk;
            U.last = min(U.first + p.key_chunk, pw_key_tiles(p, s, min(2 * U.a + 1, s.n_qt - 1)));
        } else {
            U.first = max(U.chunk * p.query_chunk, pw_first_query_tile(p, s, 2 * U.a));
            U.last = min((U.chunk + 1) * p.query_chunk, s.n_qt);
        }
        return true;
    }

    __device__ __forceinline__ int residents(const PwUnit& U) const {
        return min(2, (kStats ? s.n_qt : s.n_kt) - 2 * U.a);
    }
};

// lse of row r of query tile qt from the tile's chunks (eight loads in
// flight); +inf past the sequence's queries.
__device__ __forceinline__ float joined_lse(const PrefillWeightsParams& p, const PwSeq& s, size_t pair,
                                            int qt, int r) {
    const size_t rows = (size_t)p.num_seqs * p.num_kv_heads * p.max_query_tiles * kPwRows;
    const float2* src = p.stats + (pair * p.max_query_tiles + qt) * kPwRows + r;
    // chunks of this tile: up to the last key tile that the pair it was resident in reaches
    const int seen = pw_key_tiles(p, s, min(qt | 1, s.n_qt - 1));
    const int chunks = (seen + p.key_chunk - 1) / p.key_chunk;
    float m = -INFINITY, z = 0.f;
    for (int c0 = 0; c0 < chunks; c0 += 8) {
        float2 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = c0 + i < chunks ? src[(c0 + i) * rows] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) join_stats(m, z, v[i]);
    }
    const int tokens = min(p.tile_tokens, s.counted - qt * p.tile_tokens);
    return r < tokens * p.group ? m + log2f(z) : INFINITY;
}

// Pass 1 loads a K tile per step, pass 2 two per unit: three loading warps and
// two.  (Six, sharing the boxes of a K stage, are no faster, and leave pass 2
// 80 registers a thread, where its column sums spill: 303 us against 222 then.)
__host__ __device__ constexpr int pw_loaders(bool stats) { return stats ? 3 : 2; }

template <typename T, int D, bool kStats>
__global__ void __launch_bounds__(pw_threads(pw_loaders(kStats)), 1)
    prefill_weights_kernel(const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_q,
                           const __grid_constant__ PrefillWeightsParams p) {
    using Lay = PwLayout<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    // resident tiles (a unit's, and the next's first), streamed tiles
    constexpr int kA = 3, kB = 3;
    static_assert(kA + kB == Lay::kStages, "the rings share the CTA's tiles");
    __shared__ __align__(8) uint64_t a_full[kA], a_empty[kA], b_full[kB], b_empty[kB];
    __shared__ __align__(8) uint64_t s_full[kPwBufs], s_empty[kPwBufs], done[2];
    __shared__ uint32_t tmem_base;
    __shared__ __align__(16) float4 lse_s[4 * kPwGroups][2][kPwCols / 4];   // pass 2: [warp][tile parity]
    __shared__ float2 other[2][2][kPwRows];                          // [join parity][resident tile]
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int G = p.group;
    const int q_rows = p.tile_tokens * G;                    // rows of a query tile, <= 128

    if (threadIdx.x == 0) {
        // a stage has one loader; a resident tile has one issuer, a streamed tile both
        for (int i = 0; i < kA; ++i) mbar_init(&a_full[i], 1), mbar_init(&a_empty[i], 1);
        for (int i = 0; i < kB; ++i) mbar_init(&b_full[i], 1), mbar_init(&b_empty[i], 2);
        for (int i = 0; i < kPwBufs; ++i) mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], 4);
        for (int i = 0; i < 2; ++i) mbar_init(&done[i], 1);
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(&tmem_base, kPwBufs * kPwCols);
    if (!kStats && q_rows < kPwCols) {
        // rows that no query box fills stay zero (their lse is +inf)
        for (int i = threadIdx.x; i < kB * Lay::kTile / 16; i += pw_threads(pw_loaders(kStats)))
            reinterpret_cast<uint4*>(smem + kA * Lay::kTile)[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    grid_dependency_wait();
    allow_dependent_launch();

    if (warp == 2 || warp == 3 || warp >= kPwLoadersAfter) {
        // ------------------------------------------------------------------
        // loaders; all lanes run along, one issues.  A loader keeps to its
        // stages so that every wait follows its wait for the stage's previous
        // phase: a parity says no more than that, and a loader that had not
        // waited for that phase would take the one before it for its own.
        // ------------------------------------------------------------------
        // Pass 1: warp w has stage w of either ring.  Pass 2: warp 0 has the Q
        // stages, warp 1 the K stages.
        const int who = warp < 4 ? warp - 2 : warp - kPwLoadersAfter + 2;
        auto mine_a = [&](int n) { return kStats ? n % kA == who : who == 1; };
        auto mine_b = [&](int n) { return kStats ? n % kB == who : who == 0; };
        if (lane == 0) prefetch_tensor_map(&tmap_q), prefetch_tensor_map(&tmap_k);
        // waits for stage n % stages to be free
        auto open = [&](uint64_t* empty, int stages, int n) -> bool {
            return n < stages || pw_wait(p, &empty[n % stages], n / stages - 1);
        };
        auto load_k = [&](uint8_t* dst, uint64_t* full, uint64_t* empty, int stages, int n,
                          const PwSeq& s, const PwUnit& U, int kt, int blk) -> bool {
            if (!open(empty, stages, n)) return false;
            pw_load_keys<D, 8>(&tmap_k, dst + (n % stages) * Lay::kTile, &full[n % stages], p, s, U.g, kt, blk, 0, 8, 1);
            return true;
        };
        auto load_q = [&](uint8_t* dst, uint64_t* full, uint64_t* empty, int stages, int n,
                          const PwSeq& s, const PwUnit& U, int qt) -> bool {
            if (!open(empty, stages, n)) return false;
            pw_load_queries<D>(&tmap_q, dst + (n % stages) * Lay::kTile, &full[n % stages], p, s, U.g, qt);
            return true;
        };
        uint8_t* a_ring = smem;
        uint8_t* b_ring = smem + kA * Lay::kTile;
        PwWalk<kStats> walk;
        PwUnit U;
        int na = 0, nb = 0, at_b = -1, at_g = -1, at_qt = -1;
        bool ok = true, held = false;
        static_assert(kA == 3 && kB == 3 && pw_loaders(true) == 3, "a loader for each stage");
        while (ok && !held && walk.next(p, U)) {
            // block ids of the current four key tiles and of the next four
            int quad = -2, blk = 0, blk_next = 0;
            auto to_tile = [&](int kt) {
                if ((kt >> 2) == quad) return;
                if ((kt >> 2) != quad + 1) blk_next = pw_blocks(p, walk.s, U.b, kt >> 2);
                quad = kt >> 2;
                const int ahead = pw_blocks(p, walk.s, U.b, quad + 1);
                blk = pw_checked(p, blk_next);
                blk_next = ahead;
            };
            if (U.first >= U.last) continue;
            for (int j = 0; ok && j < walk.residents(U); ++j) {
                if (!kStats) to_tile(2 * U.a + j);
                if (mine_a(na))
                    ok = kStats ? load_q(a_ring, a_full, a_empty, kA, na, walk.s, U, 2 * U.a + j)
                                : load_k(a_ring, a_full, a_empty, kA, na, walk.s, U, 2 * U.a + j, blk);
                na += ok;
            }
            for (int i = U.first; ok && i < U.last; ++i) {
                if (kStats) {
                    to_tile(i);
                } else {
                    if (U.b == at_b && U.g == at_g && i == at_qt) continue;     // still there
                    at_b = U.b, at_g = U.g, at_qt = i;
                }
                if (mine_b(nb) && pw_withheld(p, nb)) {
                    held = true;
                    break;
                }
                if (mine_b(nb))
                    ok = kStats ? load_k(b_ring, b_full, b_empty, kB, nb, walk.s, U, i, blk)
                                : load_q(b_ring, b_full, b_empty, kB, nb, walk.s, U, i);
                nb += ok;
            }
        }
        ok = pw_landed(p, a_full, kA, na, mine_a) && ok;
        ok = pw_landed(p, b_full, kB, nb, mine_b) && ok;
        if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    } else if (warp < 2) {
        // ------------------------------------------------------------------
        // MMA issuers, one per resident tile: all lanes run along, one issues
        // ------------------------------------------------------------------
        constexpr uint32_t kId = idesc_f16(kPwRows, kPwCols, kBf16, false);
        const uint64_t a_ring = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t b_ring = smem_desc_sw128(smem_u32(smem) + kA * Lay::kTile, 16, 1024);
        PwWalk<kStats> walk;
        PwUnit U;
        int na = 0, nb = -1, tiles = 0, at_b = -1, at_g = -1, at_qt = -1;
        int used[2] = {0, 0};                               // products so far in each buffer
        bool ok = true;
        auto wait = [&](uint64_t* bar, int phase) {
            ok = ok && pw_wait(p, bar, phase);
        };
        while (ok && walk.next(p, U)) {
            if (U.first >= U.last) continue;
            const int residents = walk.residents(U);
            const bool active = warp < residents;
            // both warps wait for every tile: no phase of a stage is passed over
            for (int j = 0; j < residents; ++j) wait(&a_full[(na + j) % kA], (na + j) / kA);
            const int stage = (na + warp) % kA;
            for (int i = U.first; ok && i < U.last; ++i, ++tiles) {
                if (kStats || U.b != at_b || U.g != at_g || i != at_qt) {
                    // the previous streamed tile is free once this warp's products are done
                    if (nb >= 0 && elect_one()) mma_commit(&b_empty[nb % kB]);
                    __syncwarp();
                    ++nb;
                    at_b = U.b, at_g = U.g, at_qt = i;
                    // also where this warp has no tile to multiply: it may not run ahead
                    wait(&b_full[nb % kB], nb / kB);
                }
                if (!active) continue;
                // the group of (resident tile, parity of the streamed tile) owns the buffer
                const int odd = tiles & 1, buf = warp + 2 * odd;
                const int n = odd ? used[1]++ : used[0]++;
                if (n > 0) wait(&s_empty[buf], n - 1);
                if (!ok) break;
                tc_fence_after_sync();
                pw_product<D>(tmem + kPwCols * buf, a_ring + stage * (Lay::kTile >> 4),
                              b_ring + (nb % kB) * (Lay::kTile >> 4), kId, &s_full[buf]);
            }
            if (ok && active && elect_one()) mma_commit(&a_empty[stage]);
            __syncwarp();
            na += residents;
        }
        ok = pw_products_done(p, &done[warp]) && ok;
        if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    } else {
        // ------------------------------------------------------------------
        // epilogue: group w takes the products of resident tile w % 2 with
        // the streamed tiles of parity w / 2 (buffer w); this thread owns
        // lane r of every tile
        // ------------------------------------------------------------------
        const int group = (warp >> 2) - 1, res = group & 1, parity = group >> 1;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t tile_addr = tmem + kPwCols * group + ((uint32_t)((warp & 3) * 32) << 16);
        const float sl = p.scale_log2;
        const uint64_t sl2 = f32x2_pack(sl, sl);
        bool failed = false;
        auto wait = [&](int n) {                // the group's n-th tile
            if (!failed && !pw_wait(p, &s_full[group], n)) failed = true;
            tc_fence_after_sync();
        };
        auto release = [&] {                    // the tile is in registers
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[group]);
        };
        PwWalk<kStats> walk;
        PwUnit U;
        int tiles = 0, mine = 0, joins = 0;
        while (walk.next(p, U)) {
            const PwSeq& s = walk.s;
            const int steps = max(0, U.last - U.first);
            if (kStats && steps == 0) continue;
            const int skip = (parity - tiles) & 1;           // to the group's first streamed tile
            tiles += steps;
            if (res >= walk.residents(U)) continue;
            const size_t pair = (size_t)U.b * p.num_kv_heads + U.g;
            const int tile = 2 * U.a + res, key = tile * kPwCols + r;
            // one streamed tile is its group's alone; two groups are joined by the first
            const bool writer = steps == 1 ? skip == 0 : parity == 0;
            float before = 0.f;
            if (!kStats && writer && p.query_chunks == 1 && p.weights && key < s.L - s.C)
                before = p.weights[pair * p.weights_stride + key];
            float m = -INFINITY, z = 0.f;
            if constexpr (kStats) {
                const int pos = min(s.L - s.counted + tile * p.tile_tokens + r / G, s.L - 1);
                for (int kt = U.first + skip; kt < U.last; kt += 2) {
                    wait(mine++);
                    const int visible = pos - kt * kPwCols;           // keys 0 .. visible of the tile
                    if (__all_sync(0xffffffffu, visible >= kPwCols - 1))
                        row_stats<false, false>(m, z, tile_addr, sl, sl2, visible, release);
                    else
                        row_stats<true, false>(m, z, tile_addr, sl, sl2, visible, release);
                }
            } else {
                // the streamed rows' -lse, a copy to each warp (no barrier of the
                // group), requested a tile ahead
                const float4* src = reinterpret_cast<const float4*>(
                    p.lse + (pair * p.max_query_tiles + U.first + skip) * kPwCols) + lane;
                float4 lse = U.first + skip < U.last ? *src : make_float4(0.f, 0.f, 0.f, 0.f);
                for (int qt = U.first + skip; qt < U.last; qt += 2) {
                    float4* ls4 = lse_s[warp - 4][mine & 1];
                    ls4[lane] = make_float4(-lse.x, -lse.y, -lse.z, -lse.w);
                    src += 2 * (kPwCols / 4);
                    if (qt + 2 < U.last) lse = *src;
                    __syncwarp();
                    const float* ls = reinterpret_cast<const float*>(ls4);
                    wait(mine++);
                    const int tokens = min(p.tile_tokens, s.counted - qt * p.tile_tokens);
                    // columns that see this key: from `lo` on, up to the chunk's end
                    const int lo = (key - (s.L - s.counted + qt * p.tile_tokens)) * G, hi = tokens * G;
                    if (tokens == p.tile_tokens && __all_sync(0xffffffffu, lo <= 0))
                        z += column_sums<false>(tile_addr, ls, sl2, lo, hi, release);
                    else
                        z += column_sums<true>(tile_addr, ls, sl2, lo, hi, release);
                }
            }
            if (steps > 1) {
                // two buffers: what a group writes was read before the barrier that it passed last
                float2* o = other[joins++ & 1][res];
                if (parity == 1) o[r] = make_float2(m, z);
                asm volatile("bar.sync %0, 256;" ::"r"(5 + res) : "memory");
                if (parity == 0) {
                    if (kStats) join_stats(m, z, o[r]);
                    else z += o[r].y;
                }
            }
            if (!writer || failed) continue;
            if constexpr (kStats) {
                const int tokens = min(p.tile_tokens, s.counted - tile * p.tile_tokens);
                const size_t at = (pair * p.max_query_tiles + tile) * kPwRows + r;
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
    const size_t pair = (size_t)b * p.num_kv_heads + g;
    p.lse[(pair * p.max_query_tiles + qt) * kPwRows + r] = joined_lse(p, s, pair, qt, r);
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
    // chunks whose queries reach the pair of key tiles that this key was resident in
    const int first = pw_first_query_tile(p, s, j / kPwCols & ~1) / p.query_chunk;
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
    if (p.max_query_tiles <= 1) return window_weights_plan(p, workspace);
    // Units of some sixteenth of an SM's share (the batch taken at its
    // bounds): pass 1 in chunks of 4 to 64 key tiles, pass 2 in chunks of 8
    // to 64 query tiles.
    const int64_t per_sm = 152 * 16;
    const int64_t share1 = pairs * ((p.max_query_tiles + 1) / 2) * key_tiles / per_sm;
    const int64_t share2 = pairs * ((key_tiles + 1) / 2) * p.max_query_tiles / per_sm;
    p.key_chunk = (int)std::min<int64_t>(64, std::max<int64_t>(4, share1));
    p.key_chunks = (int)std::max<int64_t>(1, (key_tiles + p.key_chunk - 1) / p.key_chunk);
    p.query_chunk = (int)std::min<int64_t>(64, std::max<int64_t>(8, share2));
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
    const dim3 grid(sms), threads1(pw_threads(pw_loaders(true))), threads2(pw_threads(pw_loaders(false)));
    if (e == cudaSuccess && p.max_counted > 0) {
        e = launch_with_pdl(prefill_weights_kernel<T, D, true>, grid, threads1, smem, stream, tmk, tmq, p);
        if (e == cudaSuccess && p.key_chunks > 1)
            e = launch_with_pdl(prefill_stats_join_kernel,
                                dim3(p.max_query_tiles, p.num_kv_heads, p.num_seqs), dim3(kPwRows), 0,
                                stream, p);
    }
    if (e == cudaSuccess)
        e = launch_with_pdl(prefill_weights_kernel<T, D, false>, grid, threads2, smem, stream, tmk, tmq, p);
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
