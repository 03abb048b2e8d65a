// Attention weights of a chunk's last queries where those of one KV head fit
// a single tile of 128 rows (tokens x heads of the group): the observation
// window of a prompt, or a short chunk (a few short contexts are
// prefill_short.cu's).  The mathematics and the two passes are those of
// prefill_weights.cu; here a query tile meets every key tile of its sequence
// once per pass, so that the key tiles are what streams and the batch is
// memory bound: K is read twice, Q next to never.
//
// The key tiles of all (sequence, KV head) rows, in order, are dealt out in
// equal contiguous ranges to one persistent CTA per SM.  A range meets few
// rows, so the walk is cheap and no SM waits for another's larger unit.  In
// pass 1 each CTA leaves one (maximum, sum) record per row it meets, in pass
// 2 it joins a row's records (the CTAs of a row follow from the tile counts)
// and writes the weights, walking the ranges backwards: the keys read last by
// pass 1 are then read first, from L2 where they still are.
//
// Four stages of key tiles and two of query tiles; four warps load a stage
// each, and two more help with half the boxes of two stages each; two warps
// issue the products, alternating tiles, and four groups of four warps take a
// finished tile in four each.  A stage, a buffer and whoever waits for them
// stay together (tile n: stage n % 4, issuer n % 2, group n % 4), so that
// every wait follows the wait for the phase before.
//
// Measured (32 queries of 4 heads on each of 16 x 8 rows of 2048 to 8192
// tokens, D 128, fp16): 60.4 us a call on cold caches.  Alone and cold the
// passes take 36.5 and 35.6 us, 175 MB each at 62 % of the DRAM peak, some 5 us
// of which pass before the first tile is there and where the CTAs end; pass 2
// overlaps that with the end of pass 1 (replays of a graph, part of K in L2:
// 54.8 us, and 58.6 where it does not).
#include <algorithm>

#include "prefill_weights.cuh"

namespace pa {

constexpr int kWkStages = 4;                   // key tiles in flight
constexpr int kWqStages = 2;                   // query tiles: a row's and the next's
constexpr int kWindowThreads = pw_threads(6);
constexpr int kMaxWindowCtas = 256;            // bounds the records of a row

// A run of key tiles [k0, k1) of one row, counted in the walk's direction;
// `begin`: the row's first tile in that count.
struct PwRun {
    int b, g, k0, k1;
    unsigned begin;
};

// Walks a CTA's range of the tiles, row by row; all lanes of a warp together.
// Backward, sequences, heads and tiles are counted from the last.
template <bool kBackward>
struct PwRuns {
    unsigned at = 0, end = 0, base = 0, total = 0, ends = 0;
    int base_b = 0;
    PwSeq mine, s;

    // The next 32 sequences' tiles: `ends` after each lane's, `total` in all.
    __device__ __forceinline__ void read(const PrefillWeightsParams& p, bool report) {
        const int lane = threadIdx.x & 31, i = base_b + lane;
        ends = 0;
        if (i < p.num_seqs) {
            pw_sequence<kBackward>(p, kBackward ? p.num_seqs - 1 - i : i, report, mine);
            ends = (unsigned)mine.n_kt * p.num_kv_heads;
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, ends, d);
            if (lane >= d) ends += v;
        }
        total = __shfl_sync(0xffffffffu, ends, 31);
    }
    // Key tiles of the batch (the count fits 31 bits: checked on the host),
    // left at the first sequences.
    __device__ __forceinline__ unsigned count(const PrefillWeightsParams& p, bool report) {
        unsigned n = 0;
        for (int b0 = 32; b0 < p.num_seqs; b0 += 32) {
            const int i = b0 + (int)(threadIdx.x & 31);
            PwSeq q;
            q.n_kt = 0;
            if (i < p.num_seqs) pw_sequence<kBackward>(p, kBackward ? p.num_seqs - 1 - i : i, report, q);
            n += (unsigned)q.n_kt * p.num_kv_heads;
        }
        read(p, report);
        return __reduce_add_sync(0xffffffffu, n) + total;
    }

    __device__ __forceinline__ bool next(const PrefillWeightsParams& p, PwRun& R) {
        if (at >= end) return false;
        while (at >= base + total) {
            base += total;
            base_b += 32;
            if (base_b >= p.num_seqs) return false;
            read(p, false);
        }
        const int who = __ffs(__ballot_sync(0xffffffffu, at - base < ends)) - 1;
        const unsigned before = __shfl_sync(0xffffffffu, ends, max(who - 1, 0));
        s.L = __shfl_sync(0xffffffffu, mine.L, who);
        s.C = __shfl_sync(0xffffffffu, mine.C, who);
        s.counted = __shfl_sync(0xffffffffu, mine.counted, who);
        s.q0 = __shfl_sync(0xffffffffu, mine.q0, who);
        s.n_qt = __shfl_sync(0xffffffffu, mine.n_qt, who);
        s.n_kt = __shfl_sync(0xffffffffu, mine.n_kt, who);
        const unsigned first = base + (who > 0 ? before : 0u), off = at - first;
        const unsigned row = off / (unsigned)s.n_kt;
        R.b = kBackward ? p.num_seqs - 1 - (base_b + who) : base_b + who;
        R.g = kBackward ? p.num_kv_heads - 1 - (int)row : (int)row;
        R.begin = first + row * s.n_kt;
        R.k0 = (int)(at - R.begin);
        R.k1 = (int)min((unsigned)s.n_kt, R.k0 + (end - at));
        at += R.k1 - R.k0;
        return true;
    }
};

template <typename T, int D, bool kStats>
__global__ void __launch_bounds__(kWindowThreads, 1)
    window_weights_kernel(const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_q,
                          const __grid_constant__ PrefillWeightsParams p) {
    using Lay = PwLayout<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    static_assert(kWkStages + kWqStages == Lay::kStages, "the rings share the CTA's tiles");
    __shared__ __align__(8) uint64_t k_full[kWkStages], k_empty[kWkStages], q_full[kWqStages], q_empty[kWqStages];
    __shared__ __align__(8) uint64_t s_full[kPwBufs], s_empty[kPwBufs], done[2];
    __shared__ uint32_t tmem_base;
    __shared__ __align__(16) float lse_s[kPwGroups][2][kPwCols];     // pass 2: [group][row parity]
    __shared__ float2 other[2][kPwGroups - 1][kPwRows];              // pass 1: [join parity][group]
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int G = p.group;
    const int q_rows = p.tile_tokens * G;                    // rows of a query tile, <= 128
    uint8_t* k_ring = smem;
    uint8_t* q_ring = smem + kWkStages * Lay::kTile;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWkStages; ++i) mbar_init(&k_full[i], 2), mbar_init(&k_empty[i], 1);
        for (int i = 0; i < kWqStages; ++i) mbar_init(&q_full[i], 1), mbar_init(&q_empty[i], 2);
        for (int i = 0; i < kPwBufs; ++i) mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], 4);
        for (int i = 0; i < 2; ++i) mbar_init(&done[i], 1);
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(&tmem_base, kPwBufs * kPwCols);
    if (!kStats && q_rows < kPwCols) {
        // rows that no query box fills stay zero (their lse is +inf)
        for (int i = threadIdx.x; i < kWqStages * Lay::kTile / 16; i += kWindowThreads)
            reinterpret_cast<uint4*>(q_ring)[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    // Pass 2 runs ahead of the end of pass 1 on whatever pass 1 does not write.
    // What came before pass 1 has ended, since pass 1 lets its dependents go
    // only after it has waited for that; lengths and tables are read from L2,
    // where it is.
    const bool ahead = !kStats && p.max_counted > 0;
    if (!ahead) grid_dependency_wait();
    allow_dependent_launch();
    PwRuns<!kStats> runs;
    const unsigned N = runs.count(p, (kStats || p.max_counted == 0) && blockIdx.x == 0 && warp == 0);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    // CTA c has the tiles [c N / ctas, (c + 1) N / ctas), one at least; CTAs
    // past the number of tiles have none
    const unsigned ctas = min((unsigned)gridDim.x, N);
    const bool idle = blockIdx.x >= ctas;
    if (!idle) {                                 // c N / ctas in 32 bits
        const unsigned whole = N / ctas, rest = N % ctas;
        runs.at = blockIdx.x * whole + blockIdx.x * rest / ctas;
        runs.end = (blockIdx.x + 1) * whole + (blockIdx.x + 1) * rest / ctas;
    }
    auto cta_of = [&](unsigned tile) { return (int)((((uint64_t)tile + 1) * ctas - 1) / N); };
    // tile of a run's place k
    auto tile_of = [](const PwSeq& s, int k) { return kStats ? k : s.n_kt - 1 - k; };
    PwRun R;

    if (warp == 2 || warp == 3 || warp >= kPwLoadersAfter) {
        // ------------------------------------------------------------------
        // loaders: 0 .. 3 have a stage each (4 boxes a tile; loader 0 also the
        // query tiles), 4 and 5 the other boxes of even and odd tiles
        // ------------------------------------------------------------------
        const int who = warp < 4 ? warp - 2 : warp - kPwLoadersAfter + 2;
        if (lane == 0) prefetch_tensor_map(&tmap_q), prefetch_tensor_map(&tmap_k);
        int n = 0, nq = 0;                                  // key and query tiles so far
        bool ok = true, held = false;
        while (ok && !held && runs.next(p, R)) {
            const PwSeq& s = runs.s;
            if (s.counted == 0) continue;
            if (who == 0) {
                const int st = nq % kWqStages;
                if (nq >= kWqStages) ok = pw_wait(p, &q_empty[st], nq / kWqStages - 1);
                if (!ok) break;
                pw_load_queries<D>(&tmap_q, q_ring + st * Lay::kTile, &q_full[st], p, s, R.g, 0);
            }
            ++nq;
            // block ids of the current four key tiles and of the next four
            constexpr int kAhead = kStats ? 1 : -1;
            int quad = -8, blk = 0, blk_next = 0;
            for (int k = R.k0; ok && k < R.k1; ++k, ++n) {
                const int kt = tile_of(s, k);
                if ((kt >> 2) != quad) {
                    if ((kt >> 2) != quad + kAhead) blk_next = pw_blocks<!kStats>(p, s, R.b, kt >> 2);
                    quad = kt >> 2;
                    const int after = pw_blocks<!kStats>(p, s, R.b, quad + kAhead);
                    blk = pw_checked(p, blk_next);
                    blk_next = after;
                }
                const int st = n % kWkStages;
                if (who != st && who != 4 + (n & 1)) continue;
                if (n >= kWkStages) ok = pw_wait(p, &k_empty[st], n / kWkStages - 1);
                held = pw_withheld(p, n);
                if (!ok || held) break;
                pw_load_keys<D, 4>(&tmap_k, k_ring + st * Lay::kTile, &k_full[st], p, s, R.g, kt, blk,
                                   who < 4 ? 0 : 4, who < 4 ? 4 : 8, 1);
            }
        }
        ok = pw_landed(p, k_full, kWkStages, n, [&](int st) { return who == st || who == 4 + (st & 1); }) && ok;
        ok = pw_landed(p, q_full, kWqStages, nq, [&](int) { return who == 0; }) && ok;
        if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    } else if (warp < 2) {
        // ------------------------------------------------------------------
        // MMA issuers: alternate tiles
        // ------------------------------------------------------------------
        constexpr uint32_t kId = idesc_f16(kPwRows, kPwCols, kBf16, false);
        const uint64_t dk = smem_desc_sw128(smem_u32(k_ring), 16, 1024);
        const uint64_t dq = smem_desc_sw128(smem_u32(q_ring), 16, 1024);
        int n = 0, nq = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, int phase) {
            ok = ok && pw_wait(p, bar, phase);
        };
        while (ok && runs.next(p, R)) {
            if (runs.s.counted == 0) continue;
            const int qs = nq % kWqStages;
            wait(&q_full[qs], nq / kWqStages);
            for (int k = R.k0; ok && k < R.k1; ++k, ++n) {
                if ((n & 1) != warp) continue;
                const int st = n % kWkStages;               // and accumulator
                wait(&k_full[st], n / kWkStages);
                if (n >= kWkStages) wait(&s_empty[st], n / kWkStages - 1);
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t key = dk + st * (Lay::kTile >> 4), query = dq + qs * (Lay::kTile >> 4);
                pw_product<D>(tmem + kPwCols * st, kStats ? query : key, kStats ? key : query, kId, &s_full[st]);
                if (elect_one()) mma_commit(&k_empty[st]);
                __syncwarp();
            }
            if (ok && elect_one()) mma_commit(&q_empty[qs]);
            __syncwarp();
            ++nq;
        }
        ok = pw_products_done(p, &done[warp]) && ok;
        if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    } else {
        // ------------------------------------------------------------------
        // epilogue: group w takes tiles w, w + 4, ... (buffer w); this thread
        // owns lane r of every tile
        // ------------------------------------------------------------------
        static_assert(kPwBufs == kWkStages && kPwGroups == kWkStages, "stage, buffer and group go together");
        const int group = (warp >> 2) - 1;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t tile_addr = tmem + kPwCols * group + ((uint32_t)((warp & 3) * 32) << 16);
        const float sl = p.scale_log2;
        const uint64_t sl2 = f32x2_pack(sl, sl);
        bool failed = false;
        auto wait = [&](int t) {                // the group's t-th tile
            if (!failed && !pw_wait(p, &s_full[group], t)) failed = true;
            tc_fence_after_sync();
        };
        auto release = [&] {                    // the tile is in registers
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[group]);
        };
        if (ahead) grid_dependency_wait();      // the records, and weights_out
        const int max_records = p.key_chunks;
        int n = 0, mine = 0, joins = 0, rows = 0;
        while (runs.next(p, R)) {
            const PwSeq& s = runs.s;
            const size_t pair = (size_t)R.b * p.num_kv_heads + R.g;
            const int count = R.k1 - R.k0;
            if (s.counted == 0) {
                // nothing is added: what was there is carried over
                if (!kStats) {
                    for (int k = R.k0 + group; k < R.k1; k += kPwGroups) {
                        const int key = tile_of(s, k) * kPwCols + r;
                        if (key >= s.L) continue;
                        const size_t at = pair * p.weights_stride + key;
                        p.weights_out[at] = p.weights && key < s.L - s.C ? p.weights[at] : 0.f;
                    }
                }
                continue;
            }
            const int skip = (group - n) & (kPwGroups - 1);      // to the group's first tile of the run
            n += count;
            const bool valid = r < s.counted * G;                // a row of the query tile
            if constexpr (kStats) {
                float m = -INFINITY, z = 0.f;
                const int pos = min(s.L - s.counted + r / G, s.L - 1);
                for (int k = R.k0 + skip; k < R.k1; k += kPwGroups) {
                    wait(mine++);
                    const int visible = pos - k * kPwCols;
                    if (__all_sync(0xffffffffu, visible >= kPwCols - 1))
                        row_stats<false, true>(m, z, tile_addr, sl, sl2, visible, release);
                    else
                        row_stats<true, true>(m, z, tile_addr, sl, sl2, visible, release);
                }
                // one tile is its group's alone, more are joined by the first group
                bool writer = group == 0;
                if (count == 1) {
                    writer = skip == 0;
                } else {
                    float2(*o)[kPwRows] = other[joins++ & 1];
                    if (group > 0) o[group - 1][r] = make_float2(m, z);
                    asm volatile("bar.sync 7, 512;" ::: "memory");
                    if (group == 0) {
#pragma unroll
                        for (int i = 0; i < kPwGroups - 1; ++i) join_stats(m, z, o[i][r]);
                    }
                }
                if (writer && valid && !failed)
                    p.stats[(pair * max_records + (blockIdx.x - cta_of(R.begin))) * kPwRows + r] = make_float2(m, z);
            } else {
                if (skip >= count) continue;
                // lse of row r from the records of the CTAs that met this row in pass 1
                const unsigned row = N - (R.begin + s.n_kt);     // its first tile, forward
                const int records = cta_of(row + s.n_kt - 1) - cta_of(row) + 1;
                float m = -INFINITY, z = 0.f;
                if (valid) {
                    const float2* src = p.stats + pair * max_records * kPwRows + r;
                    for (int i0 = 0; i0 < records; i0 += 4) {    // four loads in flight
                        float2 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = i0 + i < records ? src[(size_t)(i0 + i) * kPwRows] : make_float2(-INFINITY, 0.f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) join_stats(m, z, v[i]);
                    }
                }
                float* ls = lse_s[group][rows++ & 1];
                ls[r] = valid ? -(m + log2f(z)) : -INFINITY;
                asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
                for (int k = R.k0 + skip; k < R.k1; k += kPwGroups) {
                    const int key = tile_of(s, k) * kPwCols + r;
                    const size_t at = pair * p.weights_stride + key;
                    const float before = p.weights && key < s.L - s.C ? p.weights[at] : 0.f;
                    wait(mine++);
                    // columns that see this key: from `lo` on, up to the chunk's end
                    const int lo = (key - (s.L - s.counted)) * G, hi = s.counted * G;
                    float w;
                    if (s.counted == p.tile_tokens && __all_sync(0xffffffffu, lo <= 0))
                        w = column_sums<false>(tile_addr, ls, sl2, lo, hi, release);
                    else
                        w = column_sums<true>(tile_addr, ls, sl2, lo, hi, release);
                    if (key < s.L && !failed) p.weights_out[at] = before + w;
                }
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

// Records of a row: a CTA leaves at most one, and has at least one of its tiles.
size_t window_weights_plan(PrefillWeightsParams& p, void* workspace) {
    const int64_t key_tiles = ((int64_t)p.max_context + kPwCols - 1) / kPwCols;
    p.key_chunks = (int)std::max<int64_t>(1, std::min<int64_t>(key_tiles, kMaxWindowCtas));
    p.stats = static_cast<float2*>(workspace);
    const size_t bytes = (size_t)p.num_seqs * p.num_kv_heads * p.key_chunks * kPwRows * sizeof(float2);
    return (bytes + 256) & ~(size_t)255;
}

template <typename T, int D>
cudaError_t launch_window_weights_t(const CUtensorMap& tmk, const CUtensorMap& tmq,
                                    const PrefillWeightsParams& p, cudaStream_t stream) {
    constexpr int smem = PwLayout<D>::kDynamicSmem;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(window_weights_kernel<T, D, true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(window_weights_kernel<T, D, false>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // both passes deal the tiles out to the same number of CTAs
    const dim3 grid(std::min(sms, kMaxWindowCtas)), threads(kWindowThreads);
    if (p.max_counted > 0)
        e = launch_with_pdl(window_weights_kernel<T, D, true>, grid, threads, smem, stream, tmk, tmq, p);
    if (e == cudaSuccess)
        e = launch_with_pdl(window_weights_kernel<T, D, false>, grid, threads, smem, stream, tmk, tmq, p);
    return e;
}

cudaError_t launch_window_weights(int dtype, int head_dim, const CUtensorMap& tmk,
                                  const CUtensorMap& tmq, const PrefillWeightsParams& p,
                                  cudaStream_t stream) {
    if (dtype == PA_BF16)
        return head_dim == 64 ? launch_window_weights_t<__nv_bfloat16, 64>(tmk, tmq, p, stream)
                              : launch_window_weights_t<__nv_bfloat16, 128>(tmk, tmq, p, stream);
    return head_dim == 64 ? launch_window_weights_t<__half, 64>(tmk, tmq, p, stream)
                          : launch_window_weights_t<__half, 128>(tmk, tmq, p, stream);
}

}  // namespace pa
