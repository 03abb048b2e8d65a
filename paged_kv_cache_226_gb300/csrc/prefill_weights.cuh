// What the two kernels of pa_prefill_weights share: the tile sizes, a
// sequence's bounds, and the folding of a finished tile's row into row
// statistics (pass 1) or column sums (pass 2).
#pragma once

#include "bounded_internal.h"
#include "decode_tile.cuh"
#include "tc_device.cuh"

namespace pa {

constexpr int kPwRows = 128;                   // lanes: rows of a resident tile
constexpr int kPwCols = 128;                   // columns: rows of a streamed tile
constexpr int kPwBufs = 4;                     // accumulators in tensor memory
constexpr int kPwGroups = 4;                   // epilogue groups of four warps, one per buffer
// Warps 0 and 1 issue MMAs, 2 and 3 load, 4 .. 19 are the epilogue's, and
// where more warps load, 20 and up do too.
constexpr int kPwLoadersAfter = 4 + 4 * kPwGroups;
__host__ __device__ constexpr int pw_threads(int loaders) {
    return (kPwLoadersAfter + loaders - 2) * 32;
}

template <int D>
struct PwLayout {
    static constexpr int kHalf = kPwRows * 128;               // 64 dims of 128 rows
    static constexpr int kHalves = D / kBoxElems;
    static constexpr int kTile = kHalves * kHalf;
    static constexpr int kStages = 6;                         // of a CTA's two rings
    static constexpr int kDynamicSmem = kStages * kTile + 1024;
};

// The wait limit of a kernel's barriers, and whether streamed tile n of this
// CTA is withheld from it (test builds only).
#ifdef PA_TEST_HOOKS
__device__ __forceinline__ uint64_t pw_wait_limit(const PrefillWeightsParams& p) { return p.test_wait_limit_ns; }
__device__ __forceinline__ bool pw_withheld(const PrefillWeightsParams& p, int n) {
    return (int)blockIdx.x == p.test_cta && n >= p.test_tile;
}
#else
__device__ __forceinline__ constexpr uint64_t pw_wait_limit(const PrefillWeightsParams&) { return kWaitLimitNs; }
__device__ __forceinline__ constexpr bool pw_withheld(const PrefillWeightsParams&, int) { return false; }
#endif

// mbar_wait for all lanes of a warp.
__device__ __forceinline__ bool pw_wait(const PrefillWeightsParams& p, uint64_t* bar, int phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, pw_wait_limit(p)));
}

// The end of a loader: tiles 0 .. n - 1 went to stages n % stages, this warp
// having issued those of the stages that mine() names.  The last of each has
// landed before the CTA's shared memory is given up, whatever became of those
// who wait for them.
template <typename Mine>
__device__ __forceinline__ bool pw_landed(const PrefillWeightsParams& p, uint64_t* full, int stages, int n,
                                          Mine&& mine) {
    bool ok = true;
    for (int st = 0; st < stages && st < n; ++st)
        if (mine(st)) ok = pw_wait(p, &full[st], (n - 1 - st) / stages) && ok;
    return ok;
}

// The end of an issuer: its products are done before tensor memory and their
// operands are given up.
__device__ __forceinline__ bool pw_products_done(const PrefillWeightsParams& p, uint64_t* bar) {
    if (elect_one()) mma_commit(bar);
    __syncwarp();
    return pw_wait(p, bar, 0);
}

struct PwSeq {
    int L, C, counted;             // context, chunk, counted queries
    int q0;                        // row of the first counted query in q
    int n_qt, n_kt;                // query and key tiles
};

// kL2: lengths (and block ids below) read past L1, by a kernel that runs ahead
// of the one before it (prefill_window.cu).
template <bool kL2 = false>
__device__ __forceinline__ void pw_sequence(const PrefillWeightsParams& p, int b, bool report,
                                            PwSeq& s) {
    auto at = [](const int32_t* x) { return kL2 ? __ldcg(x) : *x; };
    int L = at(p.context_lens + b);
    const int64_t start = at(p.query_start + b);
    int64_t C = (int64_t)at(p.query_start + b + 1) - start;
    bool bad = false;
    if (L < 0 || L > p.max_context) bad = true, L = L < 0 ? 0 : p.max_context;
    if (C < 0 || C > L) bad = true, C = C < 0 ? 0 : L;
    if (start < 0 || start + C > p.num_tokens) bad = true, C = 0;
    s.L = L, s.C = (int)C;
    s.counted = p.window > 0 ? min(p.window, s.C) : s.C;
    if (s.counted > p.max_counted) bad = true, s.counted = p.max_counted;
    s.q0 = (int)start + s.C - s.counted;
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

// Folds kCols scores of a row (those that are masked at -inf) into (m, z).
template <int kCols>
__device__ __forceinline__ void fold_scores(float& m, float& z, const uint32_t (&v)[kCols], float sl,
                                            uint64_t sl2) {
    float pm[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) pm[e] = __uint_as_float(v[e]);
#pragma unroll
    for (int e = 4; e < kCols - 4; e += 8) {          // two at a time: one instruction
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pm[i] = fmaxf(fmaxf(pm[i], __uint_as_float(v[e + i])), __uint_as_float(v[e + 4 + i]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) pm[i] = fmaxf(pm[i], __uint_as_float(v[kCols - 4 + i]));
    const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])) * sl;
    if (mx > m + kRescaleThresholdLog2) {             // also the first finite maximum
        z *= ex2(m - mx);
        m = mx;
    }
    const float ref = m == -INFINITY ? 0.f : m;       // nothing visible yet
    const uint64_t neg2 = f32x2_pack(-ref, -ref);
    uint64_t ps[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int e = 0; e < kCols / 2; ++e) {
        float a0, a1;
        f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sl2, neg2),
                     a0, a1);
        ps[e & 3] = f32x2_add(ps[e & 3], f32x2_pack(ex2(a0), ex2(a1)));
    }
    z += sum8(ps);
}

// Pass 1: folds a tile's row (keys up to `visible` with kMask) into (m, z).
// kAhead: 32 columns at a time, the next ones arriving meanwhile, where few
// tiles are in work at once (a window, in a graph: 57.1 us against 60.9);
// else 64 at once, which takes fewer instructions (large chunks: 190 against
// 193.5 us).
template <bool kMask, bool kAhead, typename Release>
__device__ __forceinline__ void row_stats(float& m, float& z, uint32_t tile_addr, float sl,
                                          uint64_t sl2, int visible, Release&& release) {
    if constexpr (kAhead) {
        uint32_t v[2][32];
        tmem_ld32(tile_addr, v[0]);
        tmem_wait_ld(v[0]);
#pragma unroll
        for (int c = 0; c < kPwCols / 32; ++c) {
            if (c < 3) tmem_ld32(tile_addr + 32 * (c + 1), v[(c + 1) & 1]);
            if (kMask) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (32 * c + e > visible) v[c & 1][e] = 0xff800000u;
            }
            fold_scores(m, z, v[c & 1], sl, sl2);
            if (c < 3) tmem_wait_ld(v[(c + 1) & 1]);
            if (c == 2) release();
        }
    } else {
#pragma unroll
        for (int c = 0; c < kPwCols; c += 64) {
            uint32_t v[64];
            tmem_ld32(tile_addr + c, *reinterpret_cast<uint32_t(*)[32]>(v));
            tmem_ld32(tile_addr + c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
            tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(v));
            tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(v + 32));
            if (c == 64) release();
            if (kMask) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (c + e > visible) v[e] = 0xff800000u;
            }
            fold_scores(m, z, v, sl, sl2);
        }
    }
}

// Pass 2: the sum of 2^(x - lse) over the tile's columns (of [lo, hi) with
// kMask); `neg_lse` in shared memory, `release` called once the tile is read.
template <bool kMask, typename Release>
__device__ __forceinline__ float column_sums(uint32_t tile_addr, const float* neg_lse, uint64_t sl2,
                                             int lo, int hi, Release&& release) {
    uint64_t ps[4] = {0ull, 0ull, 0ull, 0ull};
    uint32_t v[2][32];                       // the next 32 columns arrive while these are added
    tmem_ld32(tile_addr, v[0]);
    tmem_wait_ld(v[0]);
#pragma unroll
    for (int c = 0; c < kPwCols / 32; ++c) {
        if (c < 3) tmem_ld32(tile_addr + 32 * (c + 1), v[(c + 1) & 1]);
        const uint32_t(&x)[32] = v[c & 1];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const float4 l = *reinterpret_cast<const float4*>(neg_lse + 32 * c + e);
            float a[4];
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), sl2,
                                   f32x2_pack(l.x, l.y)), a[0], a[1]);
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), sl2,
                                   f32x2_pack(l.z, l.w)), a[2], a[3]);
            if (kMask) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[i] = 32 * c + e + i >= lo && 32 * c + e + i < hi ? a[i] : -INFINITY;
            }
            ps[(e >> 1) & 3] = f32x2_add(ps[(e >> 1) & 3], f32x2_pack(ex2(a[0]), ex2(a[1])));
            ps[((e >> 1) + 1) & 3] = f32x2_add(ps[((e >> 1) + 1) & 3], f32x2_pack(ex2(a[2]), ex2(a[3])));
        }
        if (c < 3) tmem_wait_ld(v[(c + 1) & 1]);
        if (c == 2) release();
    }
    return sum8(ps);
}

// Block ids of key tiles 4 q .. 4 q + 3: lane i has box i % 8 of tile i / 8.
// Requested here, looked at by pw_checked, so that two requests can be under way.
template <bool kL2 = false>
__device__ __forceinline__ int pw_blocks(const PrefillWeightsParams& p, const PwSeq& s, int b, int q) {
    const int tok = q * 4 * kPwCols + 16 * (threadIdx.x & 31);
    if (tok < 0 || tok >= s.L) return 0;
    const int32_t* at = p.block_tables + (size_t)b * p.max_blocks_per_seq + tok / p.block_size;
    return kL2 ? __ldcg(at) : __ldg(at);
}

__device__ __forceinline__ int pw_checked(const PrefillWeightsParams& p, int blk) {
    if (blk < 0 || blk >= p.num_blocks) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
    return blk;
}

// Boxes from, from + step, ... below `to` (kMost at most) of key tile kt (its tokens through the block table: `blk`
// as pw_checked gives it), announced on `bar` and issued; all lanes run along.
template <int D, int kMost>
__device__ __forceinline__ void pw_load_keys(const CUtensorMap* map, uint8_t* dst, uint64_t* bar,
                                             const PrefillWeightsParams& p, const PwSeq& s, int g,
                                             int kt, int blk, int from, int to, int step) {
    using Lay = PwLayout<D>;
    const int nbox = min(8, (s.L - kt * kPwCols + 15) / 16);
    const int own = max(0, (min(to, nbox) - from + step - 1) / step);
    if (elect_one()) mbar_arrive_expect_tx(bar, (uint32_t)(own * Lay::kHalves * kBox16Bytes));
    __syncwarp();
    const int sub_mask = p.block_size - 1;               // 16 or 32
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int box = from + i * step;
        if (i >= own) break;
        const int pblk = __shfl_sync(0xffffffffu, blk, (kt & 3) * 8 + box);
        if (elect_one()) {
#pragma unroll
            for (int h = 0; h < Lay::kHalves; ++h)
                tma_load_4d(dst + h * Lay::kHalf + box * kBox16Bytes, map, bar, h * kBoxElems, g,
                            (16 * box) & sub_mask, pblk);
        }
        __syncwarp();
    }
}

// Query tile qt of KV head g, in one box per 64 dims.
template <int D>
__device__ __forceinline__ void pw_load_queries(const CUtensorMap* map, uint8_t* dst, uint64_t* bar,
                                                const PrefillWeightsParams& p, const PwSeq& s, int g,
                                                int qt) {
    using Lay = PwLayout<D>;
    const int row = s.q0 + qt * p.tile_tokens;
    if (elect_one()) {
        mbar_arrive_expect_tx(bar, (uint32_t)(p.tile_tokens * p.group * Lay::kHalves * 128));
#pragma unroll
        for (int h = 0; h < Lay::kHalves; ++h)
            tma_load_3d(dst + h * Lay::kHalf, map, bar, h * kBoxElems, g * p.group, row);
    }
    __syncwarp();
}

// D(128 x 128) = A B^T over the head dim, A and B tiles given by their
// descriptors; issued by one lane, completion on `bar`.
template <int D>
__device__ __forceinline__ void pw_product(uint32_t acc, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint64_t* bar) {
    if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            constexpr int kHalf16 = PwLayout<D>::kHalf >> 4;
            const uint64_t off = (kk >> 2) * kHalf16 + (kk & 3) * 2;
            mma_f16_ss(acc, a + off, b + off, idesc, kk > 0);
        }
        mma_commit(bar);
    }
    __syncwarp();
}

}  // namespace pa
