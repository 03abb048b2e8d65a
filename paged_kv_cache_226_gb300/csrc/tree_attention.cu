// Attention of a tree of drafted tokens on the fifth-generation tensor cores:
// node i of a sequence's tree sees the sequence's context, its own ancestors
// and itself,
//   out = sum_j p_j V_j,   p = softmax_j(scale q . K_j),   j < base or
//   j - base on node i's line, base being the tokens before the tree.
//
// The rows of a (sequence, KV head) pair, its nodes times the G query heads
// that read the KV head, are cut into tiles of 128 rows (128 / G nodes), and
// its keys into tiles of 128.  A CTA has two slots, each with a query tile, a
// score tile S (probabilities P over it) and an output O in tensor memory, and
// four softmax warps, a thread per row.  Where a pair has two query tiles, each
// slot has one and every K / V tile serves both; where it has one, both slots
// have it and take the key tiles in turn.  So one slot's softmax runs beside
// the other's products either way, and K and V are read once for 256 rows.
// More rows than that go to CTAs side by side ("lanes") that walk the same
// keys at the same time, so that the second reads them from L2.
//
//   S = Q K^T           128 x 128 x D, operands in shared memory
//   P = 2^(S - m)       m a reference of the row's maximum, raised only when
//                       that grows by more than 2^8 (O is rescaled then); P
//                       goes back over S as two parts of the 16-bit type that
//                       together hold it to 2^-17 (bf16) or 2^-21 (fp16, whose
//                       reference stays 2^7 below the maximum so that small P
//                       are not lost below its range)
//   O += P V            128 x D x 128 for each part, P from tensor memory
//
// The key tiles of all pairs, in order, are dealt out to persistent CTAs in
// equal ranges, or, where contexts are short, whole pairs are.  A pair that
// more than one CTA meets leaves records (O, m, sum), joined by a second
// kernel.  What bounds it: K and V come once from HBM (512 B a token and KV
// head at D 128) and 256 rows cost 8 D operations a byte, 2/3 of the tensor
// cores' time at that rate; a row tile of its own costs a third.
//
// Warps: 0 loads K tiles and 2 V tiles, 1 issues S and 3 P V, 4 .. 7 are slot
// 0's softmax and 8 .. 11 slot 1's.  Every barrier's waits follow each other
// phase by phase: a tile's ring stage is its running number modulo the ring,
// and a slot's barriers count the slot's own tiles.
#include "decode_tile.cuh"
#include "tc_device.cuh"
#include "tree_device.cuh"

namespace pa {

constexpr int kTrRows = 128;
constexpr int kTrKeys = 128;
constexpr int kTrKStages = 3;
constexpr int kTrVStages = 2;
constexpr int kTrSlots = 2;
constexpr int kTrThreads = (4 + 4 * kTrSlots) * 32;
constexpr int kTrCtas = 152;                   // one per SM
constexpr int kTrMinTiles = 4;                 // key tiles of a CTA at least, where there are records
constexpr int kTrWholeTiles = 4;               // longest contexts, in tiles, whose pairs stay whole

template <int D>
struct TrLayout {
    static constexpr int kHalves = D / kBoxElems;
    static constexpr int kHalf = kTrRows * 128;               // 64 dims of 128 rows
    static constexpr int kTile = kHalves * kHalf;
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kTrSlots * kTile;
    static constexpr int kV = kK + kTrKStages * kTile;
    static constexpr int kRoom = kV + kTrVStages * kTile;
};

// Behind the tiles.
struct TrRoom {
    union {
        LineRoom lines;                        // a pair's, at its begin
        float2 ml[kTrSlots][kTrRows];          // the slots' statistics, at its end
    };
    uint64_t k_full[kTrKStages], k_empty[kTrKStages], v_full[kTrVStages], v_empty[kTrVStages];
    uint64_t q_full[kTrSlots], s_full[kTrSlots], p_full[kTrSlots], o_done[kTrSlots], done[2];
    uint32_t tmem;
};

template <int D>
constexpr int tr_smem() { return TrLayout<D>::kRoom + (int)sizeof(TrRoom); }
static_assert(tr_smem<128>() <= 232448, "shared memory over the per-CTA limit");

#ifdef PA_TEST_HOOKS
__device__ __forceinline__ uint64_t tr_wait_limit(const TreeParams& p) { return p.test_wait_limit_ns; }
__device__ __forceinline__ bool tr_withheld(const TreeParams& p, int n) {
    return (int)blockIdx.x == p.test_cta && n >= p.test_tile;
}
#else
__device__ __forceinline__ constexpr uint64_t tr_wait_limit(const TreeParams&) { return kWaitLimitNs; }
__device__ __forceinline__ constexpr bool tr_withheld(const TreeParams&, int) { return false; }
#endif

// mbar_wait for all lanes of a warp.
__device__ __forceinline__ bool tr_wait(const TreeParams& p, uint64_t* bar, int phase) {
    return __all_sync(0xffffffffu, mbar_wait(bar, phase & 1, tr_wait_limit(p)));
}

// A run of key tiles [k0, k1) of one pair of n tiles, the pair's first being
// number `begin` of all.
struct TrPiece {
    int b, g, k0, k1, n;
    unsigned begin;
    TreeSeq s;
};

// Walks a range of the batch's key tiles (or, with p.whole, of its pairs),
// pair by pair; all lanes of a warp together, which hold 32 sequences at a time.
struct TrWalk {
    unsigned at = 0, end = 0, base = 0, total = 0, ends = 0;
    int base_b = 0;
    TreeSeq mine;

    static __device__ __forceinline__ int tiles(const TreeSeq& s) {
        return s.C > 0 ? (s.L + kTrKeys - 1) / kTrKeys : 0;
    }
    static __device__ __forceinline__ unsigned weight(const TreeParams& p, const TreeSeq& s) {
        return (unsigned)(p.whole ? s.C > 0 : tiles(s)) * p.num_kv_heads;
    }
    __device__ __forceinline__ void read(const TreeParams& p, bool report) {
        const int lane = threadIdx.x & 31, b = base_b + lane;
        ends = 0;
        if (b < p.num_seqs) {
            mine = tree_sequence(p, b, report);
            ends = weight(p, mine);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, ends, d);
            if (lane >= d) ends += v;
        }
        total = __shfl_sync(0xffffffffu, ends, 31);
    }
    // All there is (31 bits: checked on the host), left at the first sequences.
    __device__ __forceinline__ unsigned count(const TreeParams& p, bool report) {
        unsigned n = 0;
        for (int b = 32 + (int)(threadIdx.x & 31); b < p.num_seqs; b += 32) n += weight(p, tree_sequence(p, b, report));
        read(p, report);
        return __reduce_add_sync(0xffffffffu, n) + total;
    }
    __device__ __forceinline__ bool next(const TreeParams& p, TrPiece& P) {
        if (at >= end) return false;
        while (at >= base + total) {
            base += total;
            base_b += 32;
            if (base_b >= p.num_seqs) return false;
            read(p, false);
        }
        const int who = __ffs(__ballot_sync(0xffffffffu, at - base < ends)) - 1;
        const unsigned before = __shfl_sync(0xffffffffu, ends, max(who - 1, 0));
        P.s.L = __shfl_sync(0xffffffffu, mine.L, who);
        P.s.C = __shfl_sync(0xffffffffu, mine.C, who);
        P.s.q0 = __shfl_sync(0xffffffffu, mine.q0, who);
        P.n = tiles(P.s);
        const unsigned first = base + (who > 0 ? before : 0u), off = at - first;
        const unsigned each = p.whole ? 1u : (unsigned)P.n, pair = off / each;
        P.b = base_b + who;
        P.g = (int)pair;
        P.begin = first + pair * each;
        if (p.whole) {
            P.k0 = 0, P.k1 = P.n;
            ++at;
        } else {
            P.k0 = (int)(at - P.begin);
            P.k1 = (int)min((unsigned)P.n, P.k0 + (end - at));
            at += P.k1 - P.k0;
        }
        return true;
    }
};

// How N tiles (or pairs) are dealt to the CTAs of a lane: CTA c has
// [c N / ctas, (c + 1) N / ctas).
struct TrDeal {
    unsigned N, ctas;
    __device__ __forceinline__ TrDeal(const TreeParams& p, unsigned n) : N(n) {
        ctas = p.whole ? min((unsigned)p.ctas, n) : min((unsigned)p.ctas, max(1u, n / kTrMinTiles));
    }
    __device__ __forceinline__ unsigned begin(unsigned c) const {       // in 32 bits
        const unsigned each = N / ctas, rest = N % ctas;
        return c * each + c * rest / ctas;
    }
    __device__ __forceinline__ unsigned cta_of(unsigned tile) const {
        return (unsigned)((((uint64_t)tile + 1) * ctas - 1) / N);
    }
};

// Rows of query tile t of a tree of C nodes.
__device__ __forceinline__ int tr_nodes_per_tile(int group) { return kTrRows / group; }

// The slots' use of a pair in this lane: query tiles 2 lane and 2 lane + 1.
__device__ __forceinline__ int tr_query_tiles(const TreeParams& p, int C, int lane) {
    const int per = tr_nodes_per_tile(p.group);
    return min(kTrSlots, (C + per - 1) / per - kTrSlots * lane);
}

// One operand of P V's first factor type: hi + lo parts of two probabilities.
template <typename M>
__device__ __forceinline__ void split_pair(float p0, float p1, uint32_t& hi, uint32_t& lo) {
    hi = M::pack(p0, p1);
    const float2 u = M::unpack(hi);
    float d0, d1;
    f32x2_unpack(f32x2_add(f32x2_pack(p0, p1), f32x2_pack(-u.x, -u.y)), d0, d1);
    lo = M::pack(d0, d1);
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ bool bar_or(int id, int threads, bool x) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(id), "r"(threads), "r"(x ? 1u : 0u) : "memory");
    return r != 0;
}

// Bits of 32 keys from `off` past the tree's base on: all of the context, of
// the tree those on the line.
__device__ __forceinline__ uint32_t seen_word(const TreeLine& line, int off) {
    if (off <= -32) return ~0u;
    if (off >= PA_TREE_NODES) return 0u;
    auto word = [&](int i) {
        return i < 0 ? ~0u : (i == 0 ? line.w[0] : (i == 1 ? line.w[1] : (i == 2 ? line.w[2] : (i == 3 ? line.w[3] : 0u))));
    };
    const int i = off >> 5;
    return __funnelshift_r(word(i), word(i + 1), off & 31);
}

// 16-bit elements that are not finite, at their sign bits.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    constexpr uint32_t kStep = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    return ((w & 0x7fff7fffu) + kStep) & 0x80008000u;
}

template <typename T, int D>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ TreeParams p) {
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    // how far below the maximum the reference is set, and the growth that sets it anew
    constexpr float kBelow = kBf16 ? 0.f : 7.f, kRaise = kBelow + kRescaleThresholdLog2;
    using Lay = TrLayout<D>;
    using M = Mma<T>;
    extern __shared__ __align__(1024) uint8_t smem[];        // the kernel has no other
    TrRoom& room = *reinterpret_cast<TrRoom*>(smem + Lay::kRoom);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int side = blockIdx.x % p.lanes;                   // the lane of CTAs
    const unsigned cta = blockIdx.x / p.lanes;
    const int G = p.group, per_tile = tr_nodes_per_tile(G);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kTrKStages; ++i) mbar_init(&room.k_full[i], 1), mbar_init(&room.k_empty[i], 1);
        for (int i = 0; i < kTrVStages; ++i) mbar_init(&room.v_full[i], 1), mbar_init(&room.v_empty[i], 1);
        for (int i = 0; i < kTrSlots; ++i) {
            mbar_init(&room.q_full[i], 4), mbar_init(&room.p_full[i], 4);
            mbar_init(&room.s_full[i], 1), mbar_init(&room.o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&room.done[i], 1);
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(&room.tmem, 512);
    grid_dependency_wait();
    allow_dependent_launch();
    TrWalk walk;
    const TrDeal deal(p, walk.count(p, blockIdx.x == 0 && warp == 0));
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, room.tmem, 0);
    if (cta < deal.ctas) walk.at = deal.begin(cta), walk.end = deal.begin(cta + 1);
    const unsigned range_begin = walk.at;
    TrPiece P;

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------------
        // loaders: K and V tiles, each at its own pace and on into the next
        // pair's; lane i has box i of eight
        // ------------------------------------------------------------------
        const CUtensorMap* map = warp == 0 ? &tmap_k : &tmap_v;
        uint64_t* full = warp == 0 ? room.k_full : room.v_full;
        uint64_t* empty = warp == 0 ? room.k_empty : room.v_empty;
        uint8_t* ring = smem + (warp == 0 ? Lay::kK : Lay::kV);
        const int stages = warp == 0 ? kTrKStages : kTrVStages;
        if (lane == 0) prefetch_tensor_map(map);
        int n = 0;
        bool ok = true, held = false;
        while (ok && !held && walk.next(p, P)) {
            if (tr_query_tiles(p, P.s.C, side) <= 0) continue;
            const int32_t* table = p.block_tables + (size_t)P.b * p.max_blocks_per_seq;
            // block ids: lane i has box i % 8 of tile i / 8 of four, the next
            // four tiles' requested while these are loaded
            auto ids = [&](int k) {
                const int tok = k * kTrKeys + 16 * lane;
                return tok < P.s.L ? __ldg(table + tok / p.block_size) : 0;
            };
            int blk = 0, ahead = ids(P.k0);
            for (int k = P.k0; ok && k < P.k1; ++k, ++n) {
                const int in = (k - P.k0) & 3;
                if (in == 0) {
                    blk = ahead;
                    ahead = ids(k + 4);
                    if (16 * lane + k * kTrKeys < min(P.s.L, P.k1 * kTrKeys) && (blk < 0 || blk >= p.num_blocks))
                        flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
                }
                const int st = n % stages;
                if (n >= stages) ok = tr_wait(p, &empty[st], n / stages - 1);
                held = tr_withheld(p, n);
                if (!ok || held) break;
                const int boxes = min(8, (P.s.L - k * kTrKeys + 15) / 16);
                if (elect_one()) mbar_arrive_expect_tx(&full[st], (uint32_t)(boxes * Lay::kHalves * kBox16Bytes));
                __syncwarp();
                const int id = __shfl_sync(0xffffffffu, blk, in * 8 + (lane & 7));
                if (lane < boxes) {
                    uint8_t* dst = ring + st * Lay::kTile + lane * kBox16Bytes;
#pragma unroll
                    for (int h = 0; h < Lay::kHalves; ++h)
                        tma_load_4d(dst + h * Lay::kHalf, map, &full[st], h * kBoxElems, P.g,
                                    (16 * lane) & (p.block_size - 1), id);
                }
                __syncwarp();
            }
        }
        // the last copies have landed before the CTA gives its memory up
        for (int st = 0; st < stages && st < n; ++st) ok = tr_wait(p, &full[st], (n - 1 - st) / stages) && ok;
        if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    } else if (warp == 1 || warp == 3) {
        // ------------------------------------------------------------------
        // issuers: S (warp 1) and P V (warp 3), tile by tile and slot by slot.
        // A slot's S overwrites its P, so it waits for the P V before.
        // ------------------------------------------------------------------
        constexpr uint32_t kIdS = idesc_f16(kTrRows, kTrKeys, kBf16, false);
        constexpr uint32_t kIdPV = idesc_f16(kTrRows, D, kBf16, true);
        const bool scores = warp == 1;
        const uint64_t dq = smem_desc_sw128(smem_u32(smem + Lay::kQ), 16, 1024);
        const uint64_t dk = smem_desc_sw128(smem_u32(smem + Lay::kK), 16, 1024);
        const uint64_t dv = smem_desc_sw128(smem_u32(smem + Lay::kV), Lay::kHalf, 1024);
        int n = 0, tiles[kTrSlots] = {0, 0}, queries[kTrSlots] = {0, 0};
        bool ok = true;
        auto wait = [&](uint64_t* bar, int phase) { ok = ok && tr_wait(p, bar, phase); };
        while (ok && walk.next(p, P)) {
            const int query_tiles = tr_query_tiles(p, P.s.C, side);
            if (query_tiles <= 0) continue;
            const bool share = query_tiles == kTrSlots;
            for (int k = P.k0; ok && k < P.k1; ++k, ++n) {
                const int ks = n % kTrKStages, vs = n % kTrVStages;
#pragma unroll
                for (int slot = 0; slot < kTrSlots; ++slot) {
                    if (!share && ((k - P.k0) & 1) != slot) continue;
                    const bool first = share ? k == P.k0 : k - P.k0 == slot;
                    const bool last = !share || slot == kTrSlots - 1;          // user of this tile
                    const int t = tiles[slot]++;
                    if (scores) {
                        if (first) wait(&room.q_full[slot], queries[slot]++);
                        wait(&room.k_full[ks], n / kTrKStages);
                        if (t > 0) wait(&room.o_done[slot], t - 1);
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t off = (kk >> 2) * (Lay::kHalf >> 4) + (kk & 3) * 2;
                                mma_f16_ss(tmem + kTrKeys * slot, dq + slot * (Lay::kTile >> 4) + off,
                                           dk + ks * (Lay::kTile >> 4) + off, kIdS, kk > 0);
                            }
                            mma_commit(&room.s_full[slot]);
                            if (last) mma_commit(&room.k_empty[ks]);
                        }
                        __syncwarp();
                    } else {
                        wait(&room.p_full[slot], t);
                        wait(&room.v_full[vs], n / kTrVStages);
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (elect_one()) {
                            // keys 32 c .. 32 c + 31: hi parts in columns 32 c ..
                            // 32 c + 15, lo parts in the next sixteen
#pragma unroll
                            for (int kk = 0; kk < kTrKeys / 16; ++kk) {
#pragma unroll
                                for (int part = 0; part < 2; ++part)
                                    mma_f16_ts(tmem + 2 * kTrKeys + D * slot,
                                               tmem + kTrKeys * slot + 32 * (kk >> 1) + 8 * (kk & 1) + 16 * part,
                                               dv + vs * (Lay::kTile >> 4) + kk * (16 * 128 >> 4), kIdPV,
                                               !first || kk > 0 || part > 0);
                            }
                            mma_commit(&room.o_done[slot]);
                            if (last) mma_commit(&room.v_empty[vs]);
                        }
                        __syncwarp();
                    }
                }
            }
        }
        // the products are done before tensor memory and operands are given up
        if (elect_one()) mma_commit(&room.done[warp >> 1]);
        __syncwarp();
        ok = tr_wait(p, &room.done[warp >> 1], 0) && ok;
        if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    } else {
        // ------------------------------------------------------------------
        // softmax and epilogue: this thread owns row r of its slot's tiles
        // ------------------------------------------------------------------
        const int slot = (warp >> 2) - 1;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes_at = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + kTrKeys * slot + lanes_at;
        const uint32_t tO = tmem + 2 * kTrKeys + lanes_at;         // slot 0's, slot 1's D columns on
        const int barrier = 1 + slot, both = 3;                    // named barriers
        const float sl = p.scale_log2;
        const uint64_t sl2 = f32x2_pack(sl, sl);
        bool failed = false;                  // a wait ran out: finish the loops without waiting
        auto wait = [&](uint64_t* bar, int phase) {
            if (!failed && !tr_wait(p, bar, phase)) failed = true;
        };
        int n = 0, t = 0;                     // tiles of the CTA and of the slot so far
        while (walk.next(p, P)) {
            const int query_tiles = tr_query_tiles(p, P.s.C, side);
            if (query_tiles <= 0) continue;
            const bool share = query_tiles == kTrSlots;
            const int base = P.s.L - P.s.C;
            const bool tree = P.k1 * kTrKeys > base;               // the piece has some of the tree
            const int in_tile = r / G;
            const int node = (kTrSlots * side + (share ? slot : 0)) * per_tile + in_tile;
            const bool valid = in_tile < per_tile && node < P.s.C;
            const bool live = __any_sync(0xffffffffu, valid);      // a warp without rows only keeps step
            const int64_t row = (int64_t)(P.s.q0 + node) * p.num_q_heads + P.g * G + (r - in_tile * G);
            const int count = P.k1 - P.k0;
            const int own = share ? count : (count + 1 - slot) / 2;
            // this row of Q (zero where there is none), laid out like a K tile
            if (own > 0) {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + row * D);
                uint8_t* dst = smem + Lay::kQ + slot * Lay::kTile;
#pragma unroll
                for (int c0 = 0; c0 < D / 8; c0 += 8) {
                    uint4 v[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = valid ? __ldg(src + c0 + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4*>(dst + (c0 >> 3) * Lay::kHalf + r * 128 + ((c ^ (r & 7)) << 4)) = v[c];
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&room.q_full[slot]);
            }
            TreeLine line{};
            if (tree) {
                // the tree's lines, made by slot 0 for both; the next pair's
                // come after another barrier that both slots meet
                if (slot == 0) {
                    const int up = r < P.s.C ? tree_parent(p.parents, P.s.q0, r, p.err) : -1;
                    tree_line(room.lines, r, P.s.C, up, [&](bool more) { return bar_or(barrier, kTrRows, more); });
                }
                bar_sync(both, 2 * kTrRows);
                if (valid) {
                    const uint4 w = room.lines.line[node];
                    line = TreeLine{{w.x, w.y, w.z, w.w}};
                }
            }
            float m = -INFINITY, l = 0.f;
            bool bad = false;                 // V of the tree has elements that are not finite
            for (int k = P.k0, j = 0; k < P.k1; ++k, ++n) {
                if (!share && ((k - P.k0) & 1) != slot) continue;
                const int key0 = k * kTrKeys, vs = n % kTrVStages;
                const bool masked = key0 + kTrKeys > base;
                if (masked) {
                    // V rows past the context may hold anything: clear them.
                    // Of the tree's, elements that are not finite are cleared
                    // too, since the tensor cores would carry them into rows
                    // that do not see them; rows that do get them back below.
                    const bool mine = !share || slot == 0;
                    bool odd = false;
                    if (mine) {
                        wait(&room.v_full[vs], n / kTrVStages);
                        uint8_t* vd = smem + Lay::kV + vs * Lay::kTile + r * 128;
                        const int key = key0 + r;
                        if (key >= P.s.L) {
#pragma unroll
                            for (int c = 0; c < D / 8; ++c)
                                *reinterpret_cast<uint4*>(vd + (c >> 3) * Lay::kHalf + ((c & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                        } else if (key >= base) {
                            uint32_t any = 0u;
#pragma unroll
                            for (int c = 0; c < D / 8; ++c) {
                                const uint4 w = *reinterpret_cast<const uint4*>(vd + (c >> 3) * Lay::kHalf + ((c & 7) << 4));
                                any |= not_finite<T>(w.x) | not_finite<T>(w.y) | not_finite<T>(w.z) | not_finite<T>(w.w);
                            }
                            if (any != 0u) {
                                odd = true;
                                for (int c = 0; c < D / 2; ++c) {
                                    uint32_t* w = reinterpret_cast<uint32_t*>(vd + (c >> 5) * Lay::kHalf) + (c & 31);
                                    const uint32_t x = not_finite<T>(*w);
                                    *w &= ~(((x >> 15) & 0x00010001u) * 0xffffu);
                                }
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    bad |= share ? bar_or(both, 2 * kTrRows, odd) : bar_or(barrier, kTrRows, odd);
                }
                wait(&room.s_full[slot], t);
                tc_fence_after_sync();
                if (live) {
                    uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) seen[c] = seen_word(line, key0 + 32 * c - base);
                    }
                    auto hide = [&](uint32_t(&v)[32], int c) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = (seen[c] >> e) & 1u ? v[e] : 0xff800000u;
                    };
                    // the row's maximum on the raw scores (the scale is positive)
                    float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    uint32_t v[2][32];
                    tmem_ld32(tS, v[0]);
                    tmem_wait_ld(v[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t(&x)[32] = v[c & 1];
                        if (c < 3) tmem_ld32(tS + 32 * (c + 1), v[(c + 1) & 1]);
                        if (masked) hide(x, c);
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                pm[i] = fmaxf(fmaxf(pm[i], __uint_as_float(x[e + i])), __uint_as_float(x[e + 4 + i]));
                        }
                        if (c < 3) tmem_wait_ld(v[(c + 1) & 1]);
                    }
                    const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])) * sl;
                    const bool raise = mx > m + kRaise;            // the first finite maximum, too
                    const float m_new = raise ? mx - kBelow : m;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? ex2(m - m_new) : 1.f;
                        l *= f;
                        if (j > 0) {                               // the P V before is done: S waited for it
                            wait(&room.o_done[slot], t - 1);
                            tc_fence_after_sync();
#pragma unroll
                            for (int c = 0; c < D / 32; ++c) {
                                tmem_ld32(tO + D * slot + 32 * c, v[0]);
                                tmem_wait_ld(v[0]);
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[0][e] = __float_as_uint(__uint_as_float(v[0][e]) * f);
                                tmem_st32(tO + D * slot + 32 * c, v[0]);
                            }
                        }
                        m = m_new;
                    }
                    const float ref = m == -INFINITY ? 0.f : m;    // nothing seen yet
                    const uint64_t neg2 = f32x2_pack(-ref, -ref);
                    uint64_t ps[4] = {0ull, 0ull, 0ull, 0ull};
                    tmem_ld32(tS, v[0]);
                    tmem_wait_ld(v[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t(&x)[32] = v[c & 1];
                        if (c < 3) tmem_ld32(tS + 32 * (c + 1), v[(c + 1) & 1]);
                        if (masked) hide(x, c);
                        uint32_t parts[32];                        // hi, then lo
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float a0, a1;
                            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                                                   sl2, neg2), a0, a1);
                            const float p0 = ex2(a0), p1 = ex2(a1);
                            ps[i & 3] = f32x2_add(ps[i & 3], f32x2_pack(p0, p1));
                            split_pair<M>(p0, p1, parts[i], parts[16 + i]);
                        }
                        if (c < 3) tmem_wait_ld(v[(c + 1) & 1]);
                        tmem_st32(tS + 32 * c, parts);
                    }
                    float q8[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f32x2_unpack(ps[e], q8[2 * e], q8[2 * e + 1]);
                    l += ((q8[0] + q8[1]) + (q8[2] + q8[3])) + ((q8[4] + q8[5]) + (q8[6] + q8[7]));
                    tmem_wait_st();
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&room.p_full[slot]);
                ++t, ++j;
            }
            // ---- the pair's (or piece's) end --------------------------------
            if (own > 0) wait(&room.o_done[slot], t - 1);
            tc_fence_after_sync();
            const bool full = count == P.n;
            const int64_t rec = (((int64_t)cta * p.lanes + side) * 2 + (P.begin < range_begin ? 0 : 1)) * kTrSlots +
                                (share ? slot : 0);
            float w0 = 1.f, w1 = 0.f, M_ = m;
            if (!share) {
                // both slots have this row: joined, a half of the dims each
                bar_sync(both, 2 * kTrRows);                       // the lines are not read any more
                room.ml[slot][r] = make_float2(m, l);
                tc_fence_before_sync();
                bad = bar_or(both, 2 * kTrRows, bad);
                tc_fence_after_sync();
                const float2 a = room.ml[0][r], b = room.ml[1][r];
                M_ = fmaxf(a.x, b.x);
                const float ref = M_ == -INFINITY ? 0.f : M_;
                w0 = ex2(a.x - ref), w1 = ex2(b.x - ref);
                l = a.y * w0 + b.y * w1;
            } else if (slot == 1) {
                w0 = 0.f, w1 = 1.f;
            }
            const int from = share ? 0 : slot * (D / 2), to = share ? D : from + D / 2;
            const float norm = full ? 1.f / l : 1.f;
            const bool use0 = !share || slot == 0, use1 = share ? slot == 1 : count > 1;
            w0 *= norm, w1 *= norm;
#pragma unroll 1
            for (int d = from; live && d < to; d += 32) {
                uint32_t v[2][32];
                if (use0) tmem_ld32(tO + d, v[0]);
                if (use1) tmem_ld32(tO + D + d, v[1]);
                tmem_wait_ld(v[0]);
                tmem_wait_ld(v[1]);
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] = (use0 ? __uint_as_float(v[0][e]) * w0 : 0.f) + (use1 ? __uint_as_float(v[1][e]) * w1 : 0.f);
                if (bad && valid) {
                    // what was taken out of V, for a row that sees it: the sums
                    // are what adding it gives
                    for (int i = 0; i < P.s.C; ++i) {
                        const int key = base + i;
                        if (!line.has(i) || key < P.k0 * kTrKeys || key >= P.k1 * kTrKeys) continue;
                        const int blk = p.block_tables[(size_t)P.b * p.max_blocks_per_seq + key / p.block_size];
                        if (blk < 0 || blk >= p.num_blocks) continue;
                        const T* src = static_cast<const T*>(p.v_cache) +
                                       (((int64_t)blk * p.block_size + key % p.block_size) * p.num_kv_heads + P.g) * D + d;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = (float)src[e];
                            if (!isfinite(x)) o[e] += x;
                        }
                    }
                }
                __syncwarp();
                if (!valid || failed) {
                } else if (full) {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * D + d);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        dst[q] = make_uint4(M::pack(o[8 * q], o[8 * q + 1]), M::pack(o[8 * q + 2], o[8 * q + 3]),
                                            M::pack(o[8 * q + 4], o[8 * q + 5]), M::pack(o[8 * q + 6], o[8 * q + 7]));
                } else {
                    float4* dst = reinterpret_cast<float4*>(p.rec_o + (rec * kTrRows + r) * D + d);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                }
                __syncwarp();
            }
            if (!full && valid && !failed && (share || slot == 0)) p.rec_ml[rec * kTrRows + r] = make_float2(M_, l);
            // O of both slots is read, and the statistics: the next pair may begin
            tc_fence_before_sync();
            if (!share) bar_sync(both, 2 * kTrRows);
        }
        if (failed && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
    }

    // every role is done with tensor memory
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the records of the pairs that more than one CTA met: a warp per row,
// D / 32 dims a lane.
constexpr int kTrMergeThreads = 256;
constexpr int kTrMergeRows = 32;               // of a CTA

template <typename T, int D>
__global__ void __launch_bounds__(kTrMergeThreads)
    tree_merge_kernel(const __grid_constant__ TreeParams p) {
    constexpr int kDims = D / 32;
    grid_dependency_wait();
    allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / p.num_kv_heads, g = blockIdx.x % p.num_kv_heads;
    const int tile = blockIdx.y / (kTrRows / kTrMergeRows), r0 = blockIdx.y % (kTrRows / kTrMergeRows) * kTrMergeRows;
    const TreeSeq s = tree_sequence(p, b, false);
    const int G = p.group, per_tile = tr_nodes_per_tile(G);
    if (tile * per_tile >= s.C || r0 >= min(per_tile, s.C - tile * per_tile) * G) return;
    // tiles in all, and before this sequence
    unsigned all = 0, before = 0;
    for (int i = lane; i < p.num_seqs; i += 32) {
        const unsigned w = TrWalk::weight(p, tree_sequence(p, i, false));
        all += w;
        if (i < b) before += w;
    }
    const TrDeal deal(p, __reduce_add_sync(0xffffffffu, all));
    const unsigned tiles = TrWalk::tiles(s), begin = __reduce_add_sync(0xffffffffu, before) + g * tiles;
    const unsigned c0 = deal.cta_of(begin), c1 = deal.cta_of(begin + tiles - 1);
    if (c0 == c1) return;                      // written by that CTA
    const int side = tile / kTrSlots;
    const int query_tiles = tr_query_tiles(p, s.C, side);
    const int slot = query_tiles == kTrSlots ? tile % kTrSlots : 0;
    for (int r = r0 + warp; r < r0 + kTrMergeRows; r += kTrMergeThreads / 32) {
        const int in_tile = r / G, node = tile * per_tile + in_tile;
        if (in_tile >= per_tile || node >= s.C) break;
        float m = -INFINITY, l = 0.f, o[kDims] = {};
        constexpr int kAhead = 4;
        for (unsigned c = c0; c <= c1; c += kAhead) {
            float2 ml[kAhead];
            float v[kAhead][kDims];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                ml[i] = make_float2(-INFINITY, 0.f);
                if (c + i > c1) continue;
                const int64_t rec = (((int64_t)(c + i) * p.lanes + side) * 2 + (begin < deal.begin(c + i) ? 0 : 1)) * kTrSlots + slot;
                ml[i] = p.rec_ml[rec * kTrRows + r];
                const float* src = p.rec_o + (rec * kTrRows + r) * D + kDims * lane;
                if constexpr (kDims == 4) {
                    const float4 x = *reinterpret_cast<const float4*>(src);
                    v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2*>(src);
                    v[i][0] = x.x, v[i][1] = x.y;
                }
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) top = fmaxf(top, ml[i].x);
            const float ref = top == -INFINITY ? 0.f : top, f = ex2(m - ref);
            m = top;
            l *= f;
#pragma unroll
            for (int k = 0; k < kDims; ++k) o[k] *= f;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (c + i > c1) continue;
                const float w = ex2(ml[i].x - ref);
                l += w * ml[i].y;
#pragma unroll
                for (int k = 0; k < kDims; ++k) o[k] += w * v[i][k];
            }
        }
        const float norm = 1.f / l;
        T* dst = static_cast<T*>(p.out) + ((int64_t)(s.q0 + node) * p.num_q_heads + g * G + (r - in_tile * G)) * D + kDims * lane;
        using M = Mma<T>;
        if constexpr (kDims == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(M::pack(o[0] * norm, o[1] * norm), M::pack(o[2] * norm, o[3] * norm));
        else
            *reinterpret_cast<uint32_t*>(dst) = M::pack(o[0] * norm, o[1] * norm);
    }
}

size_t tree_plan(TreeParams& p, int head_dim, void* workspace) {
    const int per_tile = kTrRows / p.group;
    const int query_tiles = (p.max_query + per_tile - 1) / per_tile;
    const int64_t pairs = (int64_t)p.num_seqs * p.num_kv_heads;
    const int tiles = (p.max_context + kTrKeys - 1) / kTrKeys;
    p.lanes = query_tiles > kTrSlots ? (query_tiles + kTrSlots - 1) / kTrSlots : 1;
    p.whole = tiles <= kTrWholeTiles;
    const int64_t most = p.whole ? pairs : (pairs * tiles + kTrMinTiles - 1) / kTrMinTiles;
    p.ctas = (int)(most < kTrCtas / p.lanes ? (most > 0 ? most : 1) : kTrCtas / p.lanes);
    const size_t rows = p.whole ? 0 : (size_t)p.ctas * p.lanes * 2 * kTrSlots * kTrRows;
    p.rec_o = static_cast<float*>(workspace);
    p.rec_ml = reinterpret_cast<float2*>(p.rec_o + rows * head_dim);
    return rows * (head_dim * sizeof(float) + sizeof(float2)) + 16;
}

cudaError_t launch_tree_codes(int dtype, const TreeParams& p, cudaStream_t stream);

template <typename T, int D>
cudaError_t launch_tree_t(const CUtensorMap& tmk, const CUtensorMap& tmv, const TreeParams& p, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(tree_attention_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         tr_smem<D>());
    if (e != cudaSuccess) return e;
    e = launch_with_pdl(tree_attention_kernel<T, D>, dim3((unsigned)(p.ctas * p.lanes)), dim3(kTrThreads), tr_smem<D>(),
                        stream, tmk, tmv, p);
    if (e != cudaSuccess || p.whole) return e;
    const int per_tile = kTrRows / p.group, query_tiles = (p.max_query + per_tile - 1) / per_tile;
    return launch_with_pdl(tree_merge_kernel<T, D>,
                           dim3((unsigned)(p.num_seqs * p.num_kv_heads), (unsigned)(query_tiles * (kTrRows / kTrMergeRows))),
                           dim3(kTrMergeThreads), 0, stream, p);
}

cudaError_t launch_tree_attention(int dtype, int head_dim, bool fp8, const CUtensorMap& tmk,
                                  const CUtensorMap& tmv, const TreeParams& p, cudaStream_t stream) {
    const bool bf16 = dtype == PA_BF16;
    if (fp8) return launch_tree_codes(dtype, p, stream);
    if (head_dim == 64) return bf16 ? launch_tree_t<__nv_bfloat16, 64>(tmk, tmv, p, stream)
                                    : launch_tree_t<__half, 64>(tmk, tmv, p, stream);
    return bf16 ? launch_tree_t<__nv_bfloat16, 128>(tmk, tmv, p, stream)
                : launch_tree_t<__half, 128>(tmk, tmv, p, stream);
}

}  // namespace pa
