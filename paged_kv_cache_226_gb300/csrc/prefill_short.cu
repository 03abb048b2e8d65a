// Attention weights of a chunk's last queries where those of one KV head fit
// a tile of 128 rows and the contexts are short: one launch that reads K once.
//
// A cluster serves one (sequence, KV head), and its CTAs hold all of the key
// tiles in shared memory, four each, so that both products of
// prefill_weights.cu can be formed without a second read: Q K^T with query
// rows in the tensor-memory lanes for the rows' maxima and sums, which the
// CTAs exchange through distributed shared memory, then K Q^T into the same
// tensor memory for the column sums.  Four warps own a key tile: they load
// its boxes, fold its rows, then its columns.  Bound by that chain (launch,
// tile, product, fold, exchange, product, fold): us against two launches of
// prefill_window.cu, 32 queries over 8 KV heads of 128 dims: one sequence of
// 120 tokens 5.4 (10.9), of 1000 7.3 (11.8), of 4096 8.9 (13.1); eight of 1000
// 9.3 (15.8); sixteen of 500 8.4 (16.0).  A second wave of CTAs starts when
// the first has ended, with nothing to overlap it, and so loses (eight of
// 4000 42 against 27, 64 of 1000 69 against 50).
#include <algorithm>

#include "prefill_weights.cuh"

namespace pa {

constexpr int kTiles = 4;                      // key tiles of a CTA, each with 128 columns of tensor memory
constexpr int kShortThreads = (4 * kTiles + 1) * 32;
constexpr int kShortMaxCluster = 8;            // the portable size
// A CTA takes most of its SM's shared memory whatever it uses: CTAs of a
// cluster wait for one another with their tensor memory allocated, so no two
// kernels that do may share an SM, where each could hold what the other's
// next CTA waits for.
constexpr int kShortSmem = 200 * 1024;

template <typename T, int D>
__global__ void __launch_bounds__(kShortThreads, 1)
    short_weights_kernel(const __grid_constant__ CUtensorMap tmap_k,
                         const __grid_constant__ CUtensorMap tmap_q,
                         const __grid_constant__ PrefillWeightsParams p, const int ranks) {
    using Lay = PwLayout<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kId = idesc_f16(kPwRows, kPwCols, kBf16, false);
    __shared__ __align__(8) uint64_t q_full, k_full[kTiles], s_full[kTiles], s_empty[kTiles], done;
    __shared__ uint32_t tmem_base;
    __shared__ float2 stats_s[kTiles][kPwRows];                  // per tile: a row's maximum and sum
    __shared__ float2 joined[kPwRows];                           // of the CTA's tiles
    __shared__ __align__(16) float neg_lse[kPwRows];
    extern __shared__ uint8_t smem_raw[];
    uint8_t* q_tile = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* k_tiles = q_tile + Lay::kTile;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int pair = blockIdx.x / ranks, rank = blockIdx.x % ranks;
    const int b = pair / p.num_kv_heads, g = pair % p.num_kv_heads;
    const int G = p.group, q_rows = p.tile_tokens * G;           // rows of the query box, <= 128

    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1), mbar_init(&done, 1);
        for (int i = 0; i < kTiles; ++i)
            mbar_init(&k_full[i], 4), mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], 4);
        fence_barrier_init();
    }
    if (warp == 4 * kTiles) {
        tmem_alloc(&tmem_base, kTiles * kPwCols);
        if (lane == 0) prefetch_tensor_map(&tmap_q), prefetch_tensor_map(&tmap_k);
    }
    if (q_rows < kPwCols) {
        // columns that the query box does not fill: their lse is +inf, their scores must be finite
        const int words = (kPwCols - q_rows) * 8;
        for (int i = threadIdx.x; i < words * Lay::kHalves; i += kShortThreads)
            *reinterpret_cast<uint4*>(q_tile + (i / words) * Lay::kHalf + q_rows * 128 + (i % words) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    grid_dependency_wait();
    PwSeq s;
    pw_sequence(p, b, threadIdx.x == 0 && rank == 0 && g == 0, s);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    allow_dependent_launch();                                    // with the tensor memory in hand
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    // this CTA's key tiles: rank, rank + ranks, ...; kTiles at most (max_context
    // <= ranks * kTiles tiles).  Lower ranks have no fewer, so those below
    // `active` have some.
    const int tiles = s.counted > 0 && rank < s.n_kt ? (s.n_kt - rank + ranks - 1) / ranks : 0;
    const int active = min(ranks, s.n_kt);
    bool ok = true;
    const int group = warp >> 2, r = (warp & 3) * 32 + lane;
    const bool epilogue = group < kTiles, works = epilogue && group < tiles;
    const int kt = rank + group * ranks;
    const bool valid = r < s.counted * G;                        // a row of the query tile
    const uint32_t tile_addr = tmem + kPwCols * group + ((uint32_t)((warp & 3) * 32) << 16);
    const float sl = p.scale_log2;
    const uint64_t sl2 = f32x2_pack(sl, sl);
    const size_t at = (size_t)pair * p.weights_stride + kt * kPwCols + r;
    float before = 0.f;
    auto wait = [&](uint64_t* bar, int phase) {
        ok = ok && pw_wait(p, bar, phase);
        tc_fence_after_sync();
    };
    auto release = [&] {                                         // the tile is in registers
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[group]);
    };

    if (!epilogue && tiles > 0) {
        pw_load_queries<D>(&tmap_q, q_tile, &q_full, p, s, g, 0);
        const uint64_t dq = smem_desc_sw128(smem_u32(q_tile), 16, 1024);
        const uint64_t dk = smem_desc_sw128(smem_u32(k_tiles), 16, 1024);
        wait(&q_full, 0);
        for (int i = 0; i < tiles; ++i) {
            wait(&k_full[i], 0);
            if (ok) pw_product<D>(tmem + kPwCols * i, dq, dk + i * (Lay::kTile >> 4), kId, &s_full[i]);
        }
        for (int i = 0; i < tiles; ++i) {
            wait(&s_empty[i], 0);
            if (ok) pw_product<D>(tmem + kPwCols * i, dk + i * (Lay::kTile >> 4), dq, kId, &s_full[i]);
        }
        ok = pw_products_done(p, &done) && ok;
    } else if (epilogue && tiles > 0) {
        float m = -INFINITY, z = 0.f;
        if (works) {
            const int blk = pw_checked(p, pw_blocks(p, s, b, kt >> 2));
            if (!pw_withheld(p, group))
                pw_load_keys<D, 2>(&tmap_k, k_tiles + group * Lay::kTile, &k_full[group], p, s, g, kt, blk, warp & 3, 8, 4);
            const int visible = min(s.L - s.counted + r / G, s.L - 1) - kt * kPwCols;
            if (p.weights && kt * kPwCols + r < s.L - s.C) before = p.weights[at];
            wait(&s_full[group], 0);
            if (__all_sync(0xffffffffu, visible >= kPwCols - 1))
                row_stats<false, true>(m, z, tile_addr, sl, sl2, visible, release);
            else
                row_stats<true, true>(m, z, tile_addr, sl, sl2, visible, release);
        }
        if (kTiles > 1) {
            if (group > 0) stats_s[group][r] = make_float2(m, z);
            asm volatile("bar.sync 1, %0;" ::"n"(128 * kTiles) : "memory");
        }
        if (group == 0) {
#pragma unroll
            for (int i = 1; i < kTiles; ++i) join_stats(m, z, stats_s[i][r]);
            joined[r] = make_float2(m, z);
            if (ranks == 1) neg_lse[r] = valid ? -(m + log2f(z)) : -INFINITY;
        }
    }
    if (ranks > 1) {
        __syncwarp();
        cluster_barrier();
        if (group == 0 && tiles > 0) {
            float m = -INFINITY, z = 0.f;
            float2 v[kShortMaxCluster];
#pragma unroll
            for (int i = 0; i < kShortMaxCluster; ++i)
                v[i] = i < active ? cluster_float2(&joined[r], i) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int i = 0; i < kShortMaxCluster; ++i) join_stats(m, z, v[i]);
            neg_lse[r] = valid ? -(m + log2f(z)) : -INFINITY;
        }
        __syncwarp();
        cluster_arrive();                                        // the others' rows are read
    }
    if (epilogue && tiles > 0) {
        asm volatile("bar.sync 1, %0;" ::"n"(128 * kTiles) : "memory");
        if (works) {
            const int key = kt * kPwCols + r;
            const int lo = (key - (s.L - s.counted)) * G, hi = s.counted * G;
            auto nothing = [] {};
            float w;
            wait(&s_full[group], 1);
            if (s.counted == p.tile_tokens && __all_sync(0xffffffffu, lo <= 0))
                w = column_sums<false>(tile_addr, neg_lse, sl2, lo, hi, nothing);
            else
                w = column_sums<true>(tile_addr, neg_lse, sl2, lo, hi, nothing);
            if (key < s.L && ok) p.weights_out[at] = before + w;
            ok = pw_wait(p, &k_full[group], 0) && ok;            // the copies have landed
        }
    } else if (epilogue && s.counted == 0) {
        // nothing is added: what was there is carried over
        const int key = kt * kPwCols + r;
        if (key < s.L) p.weights_out[at] = p.weights && key < s.L - s.C ? p.weights[at] : 0.f;
    }
    if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    if (ranks > 1) {
        __syncwarp();
        cluster_wait();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 4 * kTiles) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTiles * kPwCols);
    }
}

template <typename T, int D>
cudaError_t launch_short_weights_t(const CUtensorMap& tmk, const CUtensorMap& tmq,
                                   const PrefillWeightsParams& p, int ranks, cudaStream_t stream) {
    static_assert((1 + kTiles) * PwLayout<D>::kTile + 1024 <= kShortSmem, "the tiles fit");
    const cudaError_t e = cudaFuncSetAttribute(short_weights_kernel<T, D>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kShortSmem);
    if (e != cudaSuccess) return e;
    return launch_clusters(short_weights_kernel<T, D>, dim3(ranks),
                           dim3((unsigned)(p.num_seqs * p.num_kv_heads) * ranks), dim3(kShortThreads),
                           kShortSmem, stream, tmk, tmq, p, ranks);
}

// CTAs per (sequence, KV head), 0: not for this kernel.  Two key tiles a CTA
// while the batch fits one wave, else four (8 pairs of 2000 tokens: 8 CTAs
// each 7.6 us, 4 each 8.5; 128 pairs of 500: one each 8.4, two 15.5).  One
// wave is every SM for clusters of up to two; of larger ones fewer fit,
// since a cluster stays within a processing cluster of the GPU (36 of four
// run at once, 38 do not; 18 of six do, 16 of eight do not).
static int short_ranks(const PrefillWeightsParams& p, int sms) {
    const int64_t tiles = ((int64_t)p.max_context + kPwCols - 1) / kPwCols;
    const int64_t pairs = (int64_t)p.num_seqs * p.num_kv_heads;
    for (int per_cta : {kTiles / 2, kTiles}) {
        const int64_t ranks = (tiles + per_cta - 1) / per_cta;
        const int room = ranks <= 2 ? sms : ranks <= 4 ? sms * 9 / 10 : sms * 5 / 8;
        if (ranks <= kShortMaxCluster && pairs * ranks <= room) return (int)ranks;
    }
    return 0;
}

cudaError_t launch_short_weights(int dtype, int head_dim, const CUtensorMap& tmk,
                                 const CUtensorMap& tmq, const PrefillWeightsParams& p,
                                 cudaStream_t stream, bool* launched) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int ranks = e == cudaSuccess ? short_ranks(p, sms) : 0;
    *launched = ranks > 0;
    if (ranks == 0) return e;
    if (dtype == PA_BF16)
        return head_dim == 64 ? launch_short_weights_t<__nv_bfloat16, 64>(tmk, tmq, p, ranks, stream)
                              : launch_short_weights_t<__nv_bfloat16, 128>(tmk, tmq, p, ranks, stream);
    return head_dim == 64 ? launch_short_weights_t<__half, 64>(tmk, tmq, p, ranks, stream)
                          : launch_short_weights_t<__half, 128>(tmk, tmq, p, ranks, stream);
}

}  // namespace pa
