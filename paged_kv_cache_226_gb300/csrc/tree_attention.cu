// Attention of a tree of drafted tokens on the fifth-generation tensor cores:
// node i of a sequence's tree sees the sequence's context, its own ancestors
// and itself,
//   out = sum_j p_j V_j,   p = softmax_j(scale q . K_j),   j < base or
//   j - base on node i's line, base being the tokens before the tree.
//
// The rows of a (sequence, KV head) pair, its nodes times the G query heads
// that read the KV head, are cut into tiles of 128 rows (128 / G nodes), and
// its keys into tiles of 64.  A CTA has two slots, each with a query tile, two
// score tiles S (probabilities P over them) and an output O in tensor memory,
// and four softmax warps, a thread per row.  Where a pair has two query tiles,
// each slot has one and every K / V tile serves both; where it has one, both
// slots take its key tiles in turn, or, where those are few, one slot takes
// them all and the other the next pair's.  So one slot's softmax runs beside
// the other's products, and K and V are read once for 256 rows.  More rows
// than that go to CTAs side by side that walk the same keys at the same time,
// so that the second reads them from L2.
//
//   S = Q K^T           128 x 64 x D, operands in shared memory
//   P = 2^(S - m)       m a reference of the row's maximum, raised only when
//                       that grows by more than 2^8 (O is rescaled then); P
//                       goes back over S as two parts of the 16-bit type that
//                       together hold it to 2^-15 (bf16) or 2^-22 (fp16, whose
//                       reference stays 2^7 below the maximum so that small P
//                       are not lost below its range)
//   O += P V            128 x D x 64 for each part, P from tensor memory, cut off
//                       toward zero for 128 key tiles, then added by rounding.  A
//                       third part of P (2^-22 in bf16 too) would be a third more
//                       products, which is what bounds wide and long batches
//
// A tile passes from products to softmax, to products and back in some 1900
// cycles beside the work itself, so a slot needs two tiles under way: with one
// S of 128 keys per slot 8 heads x 4 sequences of 32k to 50k tokens at 240 rows
// took 190 us, with one of 64 keys 227, with two of 64 keys 186 (now 163).
// Rows that leave half of the tile empty stay so: twice the same 64 rows, the
// lower with one part of P and the upper with the other, take half of the P V
// products, but put softmax warps beside the issuers (32 sequences over an
// E4M3 cache below 95 us, 85 without).
//
// The CTAs side by side, one for each 256 rows and KV head (or so many KV
// heads as divide the SMs well), make a lane.  The key tiles of all sequences,
// in order, are dealt out to the lanes in equal ranges, or, where contexts are
// short, whole pairs are.  KV heads walk along together because their rows are
// neighbours in memory (4 x 32k to 50k tokens, 8 heads, without the products
// 122 us, with a range of its own for each head 130).  A pair that more than
// one lane meets leaves records (O, m, sum), joined by a second kernel.
//
// What bounds it: K and V come once from HBM, 512 B a token and KV head at
// D 128 in 16 bits, and the products cost 6 D operations (P in two parts) for
// each row and token: to some 190 rows a KV head the bytes are the longer,
// above them the products.  Measured back to back, 40 calls at a time, and for
// seconds on end, where the power limit lowers the clock under dense products:
//   64 x 128 .. 2048 tokens, 64 rows, 8 KV heads    60.7, 61 us    301 MB, 5.0 TB/s
//   16 x 2k .. 8k, 512 rows                          167, 190 us   tensor pipe 78 %
//   4 x 32k .. 50k, 240 rows                         163, 186 us   tensor pipe 80 %
//   32 x 4096, E4M3, 64 rows                          81, 83 us    277 MB, 3.4 TB/s
//   the first over E4M3, fp16 and bf16              73.3, 79.5 us  159 MB, 2.0 TB/s
// Of the first some 8 us pass until the first scores are there and 4 between
// the last output and the join's end; its loads alone took 49.  The fourth has
// 56 % of the tensor pipe and 45 % of the issue slots: without its softmax 69,
// when it took 85.
//
// An E4M3 cache's codes are brought to the 16-bit type (exactly) by four
// warps between the loaders' ring and the operands'.  Eight warps, each with
// half a tile, were within 2 % either way for the first case over E4M3.
//
// Warps: 0 loads K tiles and 2 V tiles, 1 and 3 issue the slots' S, 14 and 15
// their P V, 4 .. 7 are slot 0's softmax and 8 .. 11 slot 1's, 12 makes the
// trees' lines, 16 .. 19 convert codes.  An issuer takes some 1200 cycles for a
// tile's S beside these warps, so one for both slots would hold them up, and
// which scheduler it shares with whom counts (S of both slots by 2 and 3, or
// P V by 12 and 13: 160 to 165 us for the third case, then 156).  A barrier's parity
// tells a phase from the one before it alone, so whoever waits for a phase has
// seen that the one before is over: by waiting for every phase in turn, or as
// the comments at the waits say.
#include "decode_tile.cuh"
#include "tc_device.cuh"
#include "tree_device.cuh"

namespace pa {

constexpr int kTrRows = 128;
constexpr int kTrKeys = kTreeKeys;
constexpr int kTrSlots = 2;
constexpr int kTrQStages = 2;
constexpr int kTrSoftmaxWarps = 4 * kTrSlots;
constexpr int kTrLineWarp = 4 + kTrSoftmaxWarps;
constexpr int kTrValueWarp = kTrLineWarp + 2;  // issuers of P V
constexpr int kTrConvertWarp = kTrValueWarp + kTrSlots;
constexpr int kTrConverters = 4;               // E4M3 only
__host__ __device__ constexpr int tr_threads(bool fp8) { return (kTrConvertWarp + (fp8 ? kTrConverters : 0)) * 32; }
// Registers: 512 threads are launched with 128 each (640 with 96); the softmax
// warps take over what the others give up.
constexpr int kTrControlRegs = 72;
__host__ __device__ constexpr int tr_softmax_regs(bool fp8) { return fp8 ? 128 : 184; }
static_assert(256 * tr_softmax_regs(false) + 256 * kTrControlRegs <= 512 * 128 &&
              256 * tr_softmax_regs(true) + 384 * kTrControlRegs <= 640 * 96, "registers of the CTA");
constexpr int kTrCtas = 152;                   // one per SM
// A lane's range weighs that much at least, so that not every lane has a record
// of the same few tiles (one KV head, 50,000 tokens: 4 took 51 us, 6 33, 8 28).
constexpr int kTrMinTiles = 8;
// The longest contexts, in tiles, whose pairs stay whole: no records, but uneven
// lanes (16 x 300 .. 512 tokens: whole 12.4 us, dealt out 18.1; 64 x up to 1000:
// whole 52.8 us, dealt out 46.0; up to 2048: 91 and 61).  Where most lanes have
// a pair each and none has two, longer ones do too (16 x 800 .. 1000 tokens:
// whole 18.7 us, dealt out 22.9; 20 pairs on the 19 lanes 30.0 and 25.1, one
// pair of 760 tokens 19.9 and 17.8).
constexpr int kTrWholeTiles = 8, kTrWholeTilesAlone = 16;
// What a pair weighs beside its tiles (64 x 128 .. 2048 tokens: 2 took 77 us,
// 4 73; 3 and 6 within 1 % of 4).
constexpr int kTrPairWeight = kTreePairWeight;
// The longest piece that one slot takes alone, while the other takes the next:
// joining costs two barriers of the CTA.
constexpr int kTrSoloTiles = 2;
// Tiles of a slot whose products add up in tensor memory.  The tensor cores cut
// each sum off toward zero, eight times a tile, which takes some 4e-7 of O a
// tile (0.4 % after 10,000); after so many tiles O is added, rounded, to what
// the softmax warps hold in the workspace and begins anew, so that it loses
// 5e-5, a fifth of fp16's smallest rounding error, however long the context.
// 4 x 32k to 50k tokens, some 135 tiles a CTA, in long runs: 64 190 us, 128
// 186, 256 184, as without.
constexpr int kTrRun = 128;
static_assert(kTrRun >= kTrWholeTilesAlone, "whole pairs have no workspace");

// Shared memory: query tiles, operand tiles, codes.
template <int D, bool kFp8>
struct TrLayout {
    static constexpr int kKStages = kFp8 ? 3 : 5, kVStages = kFp8 ? 3 : 5;
    static constexpr int kCodeStages = kFp8 ? 4 : 0;          // of K and of V each
    // barriers that say an operand stage is free again: over E4M3 two a stage,
    // for every other use (the converters' comment says why)
    static constexpr int kKEmpties = kFp8 ? 2 * kKStages : kKStages, kVEmpties = kFp8 ? 2 * kVStages : kVStages;
    static constexpr int kHalves = D / kBoxElems;
    static constexpr int kHalf = kTrKeys * 128;               // 64 dims of 64 rows
    static constexpr int kTile = kHalves * kHalf;
    static constexpr int kCodes = kTrKeys * 128;              // 128 codes of 64 rows
    static constexpr int kQHalf = kTrRows * 128, kQTile = kHalves * kQHalf;
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kTrQStages * kQTile;
    static constexpr int kV = kK + kKStages * kTile;
    static constexpr int kKCodes = kV + kVStages * kTile;
    static constexpr int kVCodes = kKCodes + kCodeStages * kCodes;
    static constexpr int kRoom = kVCodes + kCodeStages * kCodes;
};

// Tensor memory: a slot's two S, a slot's O.
constexpr int kTrS = 0, kTrO = 2 * kTrSlots * kTrKeys;

// Behind the tiles.
struct TrRoom {
    union {
        uint4 line[PA_TREE_NODES];             // a piece's lines, until they are read
        float2 ml[kTrSlots][kTrRows];          // the slots' statistics, at a joined piece's end
    };
    uint64_t k_full[5], k_empty[6], v_full[5], v_empty[6];
    uint64_t kc_full[4], kc_empty[4], vc_full[4], vc_empty[4];
    uint64_t q_full[kTrQStages], q_empty[kTrQStages], lines_full, lines_empty;
    uint64_t s_full[kTrSlots][2], p_full[kTrSlots][2], o_done[kTrSlots][2], v_there[kTrSlots], done[2 * kTrSlots];
    uint32_t tmem;
};

template <int D, bool kFp8>
constexpr int tr_smem() { return TrLayout<D, kFp8>::kRoom + (int)sizeof(TrRoom); }
static_assert(tr_smem<128, false>() <= 232448 && tr_smem<128, true>() <= 232448 && tr_smem<64, false>() <= 232448,
              "shared memory over the per-CTA limit");

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

// A ring's stage and lap, tile by tile.
template <int kStages>
struct TrRing {
    int at = 0, lap = 0;
    __device__ __forceinline__ void step() {
        if (++at == kStages) at = 0, ++lap;
    }
};

// A run of key tiles [k0, k1) of one pair of n tiles.
struct TrPiece {
    int b, g, k0, k1, n;
    int query;                     // query tiles of this CTA
    TreeSeq s;
    bool share;                    // each slot has a query tile, and all key tiles
    bool alone;                    // the slots do not join: shared, or few tiles
    int owner;                     // the slot of those few

    // The slot that takes key tile k where it is not both.
    __device__ __forceinline__ int slot_of(int k) const { return alone ? owner : (k - k0) & 1; }
    __device__ __forceinline__ bool has(int slot, int k) const { return share || slot_of(k) == slot; }
    // A slot's tiles.
    __device__ __forceinline__ int own(int slot) const {
        return share ? k1 - k0 : (alone ? (owner == slot ? k1 - k0 : 0) : (k1 - k0 + 1 - slot) / 2);
    }
    __device__ __forceinline__ int query_tiles() const { return share ? 2 : 1; }
    __device__ __forceinline__ bool rows(int slot) const { return slot < query; }
    // Whether key tile k has tokens of the tree, or ends behind it.
    __device__ __forceinline__ bool masked(int k) const { return (k + 1) * kTrKeys > s.L - s.C; }
    // The slot whose softmax warps clear V of such a tile.
    __device__ __forceinline__ bool clears(int slot) const { return !share || slot == 0; }
};

// Nodes of a query tile.
__device__ __forceinline__ int tr_nodes_per_tile(int group) { return kTrRows / group; }

// Walks a range of the batch's key tiles (or, with p.whole, of its pairs),
// pair by pair; all lanes of a warp together, which hold 32 sequences at a
// time.  A pair weighs its tiles and kTrPairWeight, which come first.
template <bool kL2 = false>
struct TrWalk {
    unsigned at = 0, end = 0, base = 0, total = 0, ends = 0;
    int base_b = 0, turn = 0;
    TreeSeq mine;

    static __device__ __forceinline__ int tiles(const TreeSeq& s) {
        return s.C > 0 ? (s.L + kTrKeys - 1) / kTrKeys : 0;
    }
    static __device__ __forceinline__ unsigned each(const TreeParams& p, const TreeSeq& s) {
        return s.C > 0 ? (p.whole ? 1u : (unsigned)(tiles(s) + kTrPairWeight)) : 0u;
    }
    static __device__ __forceinline__ unsigned weight(const TreeParams& p, const TreeSeq& s) {
        return each(p, s) * (p.num_kv_heads / p.heads);
    }
    __device__ __forceinline__ void read(const TreeParams& p, bool report) {
        const int lane = threadIdx.x & 31, b = base_b + lane;
        ends = 0;
        if (b < p.num_seqs) {
            mine = tree_sequence<kL2>(p, b, report);
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
        const int b1 = 32 + (int)(threadIdx.x & 31);
        TreeSeq next;
        next.C = 0;
        if (b1 < p.num_seqs) next = tree_sequence<kL2>(p, b1, report);       // under way beside the first
        read(p, report);
        unsigned n = weight(p, next);
        for (int b = b1 + 32; b < p.num_seqs; b += 32) n += weight(p, tree_sequence<kL2>(p, b, report));
        return __reduce_add_sync(0xffffffffu, n) + total;
    }
    // The pair at `at`, for query tiles `side` and KV heads head, head + p.heads,
    // ..., its first weight and all of it; its rows and slots of this CTA.
    __device__ __forceinline__ bool find(const TreeParams& p, int side, int head, TrPiece& P, unsigned& begin,
                                         unsigned& one) {
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
        one = each(p, P.s);
        const unsigned first = base + (who > 0 ? before : 0u), pair = (at - first) / one;
        begin = first + pair * one;
        P.b = base_b + who;
        P.g = head + (int)pair * p.heads;
        const int per = tr_nodes_per_tile(p.group);              // query tiles 2 side and 2 side + 1
        P.query = min((P.s.C + per - 1) / per - kTrSlots * side, kTrSlots);
        P.share = P.query == kTrSlots;
        return true;
    }
    // The next piece with work for that CTA.
    __device__ __forceinline__ bool next(const TreeParams& p, int side, int head, TrPiece& P) {
        while (at < end) {
            unsigned begin, one;
            if (!find(p, side, head, P, begin, one)) return false;
            if (p.whole) {
                P.k0 = 0, P.k1 = P.n;
                ++at;
            } else {
                const unsigned in = at - begin, stop = min(one, in + (end - at));
                P.k0 = max((int)in - kTrPairWeight, 0);
                P.k1 = (int)stop - kTrPairWeight;
                at += stop - in;
                if (P.k1 <= P.k0) continue;
            }
            if (P.query <= 0) continue;
            P.alone = P.share || P.k1 - P.k0 <= kTrSoloTiles;
            P.owner = turn;
            if (P.alone && !P.share) turn ^= 1;
            return true;
        }
        return false;
    }
};

// How weight N is dealt to the lanes: lane c has [c N / ctas, (c + 1) N / ctas).
struct TrDeal {
    unsigned N, ctas;
    __device__ __forceinline__ TrDeal(const TreeParams& p, unsigned n) : N(n) {
        ctas = p.whole ? min((unsigned)p.ctas, n) : min((unsigned)p.ctas, max(1u, n / kTrMinTiles));
    }
    __device__ __forceinline__ unsigned begin(unsigned c) const {       // in 32 bits
        const unsigned each = N / ctas, rest = N % ctas;
        return c * each + c * rest / ctas;
    }
    __device__ __forceinline__ unsigned cta_of(unsigned at) const {
        return (unsigned)((((uint64_t)at + 1) * ctas - 1) / N);
    }
};

// Two probabilities as hi + lo parts of the 16-bit type.  A bf16 hi is p cut to
// its upper half, so that lo does not wait for a conversion; for fp16 the
// rounded one is the quicker.
template <typename T>
__device__ __forceinline__ void split_pair(float p0, float p1, uint32_t& hi, uint32_t& lo) {
    using M = Mma<T>;
    float2 h;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        hi = prmt(__float_as_uint(p0), __float_as_uint(p1), 0x7632u);
        h.x = __uint_as_float(__float_as_uint(p0) & 0xffff0000u), h.y = __uint_as_float(__float_as_uint(p1) & 0xffff0000u);
    } else {
        hi = M::pack(p0, p1);
        h = M::unpack(hi);
    }
    float d0, d1;
    f32x2_unpack(f32x2_fma(f32x2_pack(h.x, h.y), f32x2_pack(-1.f, -1.f), f32x2_pack(p0, p1)), d0, d1);
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

// The lines of a tree's C nodes, a warp making them: lane i has nodes i, i +
// 32, ... and their masks.  Masks and parents double their reach in every
// round, as in tree_line.
__device__ __forceinline__ void warp_lines(uint32_t (&w)[kLineWords][kLineWords], int (&up)[kLineWords], int C) {
    const int lane = threadIdx.x & 31, sets = (C + 31) / 32;
#pragma unroll
    for (int i = 0; i < kLineWords; ++i) {
#pragma unroll
        for (int k = 0; k < kLineWords; ++k) w[i][k] = i == k && lane + 32 * i < C ? 1u << lane : 0u;
    }
    for (;;) {
        bool more = false;
#pragma unroll
        for (int i = 0; i < kLineWords; ++i) more |= up[i] >= 0;
        if (!__any_sync(0xffffffffu, more)) return;
        uint32_t add[kLineWords][kLineWords];
        int to[kLineWords];
#pragma unroll
        for (int i = 0; i < kLineWords; ++i) {
            to[i] = -1;
#pragma unroll
            for (int k = 0; k < kLineWords; ++k) add[i][k] = 0u;
            if (i >= sets) continue;
#pragma unroll
            for (int set = 0; set <= i; ++set) {             // parents stand before their nodes
                const bool here = up[i] >= 0 && (up[i] >> 5) == set;
                const int from = up[i] & 31;
#pragma unroll
                for (int k = 0; k <= set; ++k) {
                    const uint32_t x = __shfl_sync(0xffffffffu, w[set][k], from);
                    if (here) add[i][k] = x;
                }
                const int x = __shfl_sync(0xffffffffu, up[set], from);
                if (here) to[i] = x;
            }
        }
#pragma unroll
        for (int i = 0; i < kLineWords; ++i) {
            up[i] = to[i];
#pragma unroll
            for (int k = 0; k < kLineWords; ++k) w[i][k] |= add[i][k];
        }
    }
}

// By the four warps of a group together, in a branch of their own: what follows
// a join of branches would be held to the smaller count.
__device__ __forceinline__ void control_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTrControlRegs));
}

template <int kRegs>
__device__ __forceinline__ void softmax_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <typename T, int D, bool kFp8>
__global__ void __launch_bounds__(tr_threads(kFp8), 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ CUtensorMap tmap_q,
                          const __grid_constant__ TreeParams p) {
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    // how far below the maximum the reference is set, and the growth that sets it anew
    constexpr float kBelow = kBf16 ? 0.f : 7.f, kRaise = kBelow + kRescaleThresholdLog2;
    using Lay = TrLayout<D, kFp8>;
    using M = Mma<T>;
    extern __shared__ __align__(1024) uint8_t smem[];        // the kernel has no other
    TrRoom& room = *reinterpret_cast<TrRoom*>(smem + Lay::kRoom);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // CTA of the lane, and lane
    const int head = blockIdx.x % p.heads, side = blockIdx.x / p.heads % p.sides;
    const unsigned cta = blockIdx.x / p.heads / p.sides;
    const int G = p.group, per_tile = tr_nodes_per_tile(G);

    if (threadIdx.x == 0) {
        for (int i = 0; i < Lay::kKStages; ++i) mbar_init(&room.k_full[i], 1);
        for (int i = 0; i < Lay::kVStages; ++i) mbar_init(&room.v_full[i], 1);
        for (int i = 0; i < Lay::kKEmpties; ++i) mbar_init(&room.k_empty[i], kTrSlots);
        for (int i = 0; i < Lay::kVEmpties; ++i) mbar_init(&room.v_empty[i], kTrSlots);
        for (int i = 0; i < Lay::kCodeStages; ++i) {
            mbar_init(&room.kc_full[i], 1), mbar_init(&room.kc_empty[i], 1);
            mbar_init(&room.vc_full[i], 1), mbar_init(&room.vc_empty[i], 1);
        }
        for (int i = 0; i < kTrQStages; ++i) mbar_init(&room.q_full[i], 1), mbar_init(&room.q_empty[i], kTrSlots);
        mbar_init(&room.lines_full, 1), mbar_init(&room.lines_empty, kTrSoftmaxWarps);
        for (int i = 0; i < kTrSlots; ++i) {
            mbar_init(&room.v_there[i], 1);
            for (int j = 0; j < 2; ++j)
                mbar_init(&room.s_full[i][j], 1), mbar_init(&room.p_full[i][j], 4), mbar_init(&room.o_done[i][j], 1);
        }
        for (int i = 0; i < 2 * kTrSlots; ++i) mbar_init(&room.done[i], 1);
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(&room.tmem, 512);
    if (threadIdx.x == 64) prefetch_tensor_map(&tmap_q), prefetch_tensor_map(&tmap_k), prefetch_tensor_map(&tmap_v);
    grid_dependency_wait();
    allow_dependent_launch();
    TrWalk<> walk;
    const TrDeal deal(p, walk.count(p, blockIdx.x == 0 && warp == 0));
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, room.tmem, 0);
    if (cta < deal.ctas) walk.at = deal.begin(cta), walk.end = deal.begin(cta + 1);
    TrPiece P;

    if (warp < 4) {
        control_registers();
        if (warp == 0 || warp == 2) {
            // --------------------------------------------------------------
            // loaders: K (and query) tiles and V tiles, each at its own pace
            // and on into the next pair's; lane i has box i % 4, dims 64 (i / 4) on
            // --------------------------------------------------------------
            auto load = [&](auto kind) {
                constexpr bool keys = decltype(kind)::value;
                constexpr int kStages = kFp8 ? Lay::kCodeStages : (keys ? Lay::kKStages : Lay::kVStages);
                constexpr int kStage = kFp8 ? Lay::kCodes : Lay::kTile, kBoxes = kFp8 ? 1 : Lay::kHalves;
                const CUtensorMap* map = keys ? &tmap_k : &tmap_v;
                uint64_t* full = kFp8 ? (keys ? room.kc_full : room.vc_full) : (keys ? room.k_full : room.v_full);
                uint64_t* empty = kFp8 ? (keys ? room.kc_empty : room.vc_empty) : (keys ? room.k_empty : room.v_empty);
                uint8_t* ring = smem + (kFp8 ? (keys ? Lay::kKCodes : Lay::kVCodes) : (keys ? Lay::kK : Lay::kV));
                const int block_shift = p.block_size == 16 ? 4 : 5;
                const int box = lane & 3, dims = lane >> 2, sub = (16 * box) & (p.block_size - 1);
                uint8_t* dst = ring + dims * Lay::kHalf + box * kBox16Bytes;
                int n = 0;
                TrRing<kStages> at;
                TrRing<kTrQStages> q;
                bool ok = true, held = false;

                while (ok && !held && walk.next(p, side, head, P)) {
                    const int32_t* table = p.block_tables + (size_t)P.b * p.max_blocks_per_seq;
                    // block ids: lane i has box i % 4 of tile i / 4 of eight, the
                    // next eight tiles' requested while these are loaded
                    auto ids = [&](int k) {
                        const int tok = k * kTrKeys + 16 * lane;
                        return tok < P.s.L ? __ldg(table + (tok >> block_shift)) : 0;
                    };
                    int blk = 0, ahead = ids(P.k0);
                    // the piece's query tiles come before its keys
                    for (int i = 0; keys && ok && i < P.query_tiles(); ++i, q.step()) {
                        if (q.lap > 0) ok = tr_wait(p, &room.q_empty[q.at], q.lap - 1);
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&room.q_full[q.at], (uint32_t)(per_tile * G * Lay::kHalves * 128));
#pragma unroll
                            for (int h = 0; h < Lay::kHalves; ++h)
                                tma_load_3d(smem + Lay::kQ + q.at * Lay::kQTile + h * Lay::kQHalf, &tmap_q, &room.q_full[q.at],
                                            h * kBoxElems, P.g * G, P.s.q0 + (kTrSlots * side + i) * per_tile);
                        }
                        __syncwarp();
                    }
                    for (int k = P.k0; ok && k < P.k1; ++k, ++n, at.step()) {
                        const int in = (k - P.k0) & 7;
                        if (in == 0) {
                            blk = ahead;
                            ahead = ids(k + 8);
                            if (16 * lane + k * kTrKeys < min(P.s.L, P.k1 * kTrKeys) && (blk < 0 || blk >= p.num_blocks))
                                flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
                        }
                        if (at.lap > 0) ok = tr_wait(p, &empty[at.at], at.lap - 1);
                        held = tr_withheld(p, n);
                        if (!ok || held) break;
                        const int boxes = min(4, (P.s.L - k * kTrKeys + 15) / 16);
                        if (elect_one()) mbar_arrive_expect_tx(&full[at.at], (uint32_t)(boxes * kBoxes * kBox16Bytes));
                        __syncwarp();
                        const int id = __shfl_sync(0xffffffffu, blk, in * 4 + box);
                        if (dims < kBoxes && box < boxes)
                            tma_load_4d(dst + at.at * kStage, map, &full[at.at], dims * kBoxElems, P.g, sub, id);
                        __syncwarp();
                    }
                }
                // the last copies have landed before the CTA gives its memory up:
                // the stages of this lap, then the others of the lap before
                for (int st = 0; st < kStages; ++st) {
                    const int lap = st < at.at ? at.lap : at.lap - 1;
                    if (lap >= 0) ok = tr_wait(p, &full[st], lap) && ok;
                }
                for (int st = 0; keys && st < kTrQStages; ++st) {
                    const int lap = st < q.at ? q.lap : q.lap - 1;
                    if (lap >= 0) ok = tr_wait(p, &room.q_full[st], lap) && ok;
                }
                if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
            };
            if (warp == 0)
                load(std::true_type());
            else
                load(std::false_type());
        } else {
            // --------------------------------------------------------------
            // issuers of S: S overwrites the P of two tiles before, so it
            // waits for that P V.  Both see every stage full before they give
            // it back, whether it is theirs or not, so neither can give back
            // the next tile in its place.
            // --------------------------------------------------------------
            constexpr uint32_t kId = idesc_f16(kTrRows, kTrKeys, kBf16, false);
            const int slot = warp >> 1;
            const uint64_t dq = smem_desc_sw128(smem_u32(smem + Lay::kQ), 16, 1024);
            const uint64_t dk = smem_desc_sw128(smem_u32(smem + Lay::kK), 16, 1024);
            const uint32_t s0 = tmem + kTrS + 2 * kTrKeys * slot;
            TrRing<Lay::kKStages> at;
            TrRing<Lay::kKEmpties> back;
            TrRing<kTrQStages> q;
            int t = 0;
            bool ok = true;
            auto wait = [&](uint64_t* bar, int phase) { ok = ok && tr_wait(p, bar, phase); };
            while (ok && walk.next(p, side, head, P)) {
                const int q0 = q.at;
                for (int i = 0; i < P.query_tiles(); ++i, q.step()) wait(&room.q_full[q.at], q.lap);
                const uint64_t query = dq + (P.share ? q0 ^ slot : q0) * (Lay::kQTile >> 4);
                for (int k = P.k0; ok && k < P.k1; ++k, at.step(), back.step()) {
                    wait(&room.k_full[at.at], at.lap);
                    if (P.has(slot, k)) {
                        const int buf = t & 1;
                        if (t > 1) wait(&room.o_done[slot][buf], (t >> 1) - 1);
                        if (!ok) break;
                        ++t;
                        tc_fence_after_sync();
                        const uint64_t key = dk + at.at * (Lay::kTile >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                mma_f16_ss(s0 + kTrKeys * buf, query + (kk >> 2) * (Lay::kQHalf >> 4) + (kk & 3) * 2,
                                           key + (kk >> 2) * (Lay::kHalf >> 4) + (kk & 3) * 2, kId, kk > 0);
                            mma_commit(&room.s_full[slot][buf]);
                            mma_commit(&room.k_empty[back.at]);
                        }
                    } else if (ok && elect_one()) {
                        mbar_arrive(&room.k_empty[back.at]);
                    }
                    __syncwarp();
                }
                if (ok && elect_one()) {
                    mma_commit(&room.q_empty[q0]);
                    if (P.share) mma_commit(&room.q_empty[q0 ^ 1]);
                }
                __syncwarp();
            }
            // the products are done before tensor memory and operands are given up
            if (elect_one()) mma_commit(&room.done[slot]);
            __syncwarp();
            ok = tr_wait(p, &room.done[slot], 0) && ok;
            if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
        }
    } else if (warp >= kTrLineWarp && warp < kTrConvertWarp) {
        control_registers();
        if (warp == kTrLineWarp) {
            // --------------------------------------------------------------
            // the trees' lines, a piece ahead of those who read them
            // --------------------------------------------------------------
            bool ok = true;
            int before = 0;                                        // key tiles of the piece before
            for (int i = 0; ok && walk.next(p, side, head, P); ++i) {
                uint32_t w[kLineWords][kLineWords] = {};
                const bool tree = P.k1 * kTrKeys > P.s.L - P.s.C;      // the piece has some of it
                if (tree) {
                    int up[kLineWords];
#pragma unroll
                    for (int j = 0; j < kLineWords; ++j) {
                        const int node = lane + 32 * j;
                        up[j] = node < P.s.C ? tree_parent(p.parents, P.s.q0, node, p.err) : -1;
                    }
                    warp_lines(w, up, P.s.C);
                }
                // the room is free where the piece before ends, which may be long:
                // another limit for every 2^17 of its tiles
                if (i > 0) ok = tr_wait(p, &room.lines_empty, i - 1);
                for (int more = before >> 17; !ok && more > 0; --more) ok = tr_wait(p, &room.lines_empty, i - 1);
                before = P.k1 - P.k0;
                if (!ok) break;
                if (tree) {
#pragma unroll
                    for (int j = 0; j < kLineWords; ++j)
                        room.line[lane + 32 * j] = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&room.lines_full);
            }
            if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
        } else if (warp >= kTrValueWarp) {
            // --------------------------------------------------------------
            // issuers of P V
            // --------------------------------------------------------------
            constexpr uint32_t kId = idesc_f16(kTrRows, D, kBf16, true);
            const int slot = warp - kTrValueWarp;
            const uint64_t dv = smem_desc_sw128(smem_u32(smem + Lay::kV), Lay::kHalf, 1024);
            const uint32_t o = tmem + kTrO + D * slot, p0 = tmem + kTrS + 2 * kTrKeys * slot;
            TrRing<Lay::kVStages> at;
            TrRing<Lay::kVEmpties> back;
            int t = 0;
            bool ok = true;
            auto wait = [&](uint64_t* bar, int phase) { ok = ok && tr_wait(p, bar, phase); };
            while (ok && walk.next(p, side, head, P)) {
                int j = 0;                                             // tiles of the slot
                for (int k = P.k0; ok && k < P.k1; ++k, at.step(), back.step()) {
                    wait(&room.v_full[at.at], at.lap);
                    if (P.has(slot, k)) {
                        const int buf = t & 1;
                        if (ok && P.masked(k) && P.clears(slot) && elect_one()) mbar_arrive(&room.v_there[slot]);
                        __syncwarp();
                        wait(&room.p_full[slot][buf], t >> 1);
                        if (!ok) break;
                        ++t;
                        tc_fence_after_sync();
                        const uint64_t value = dv + at.at * (Lay::kTile >> 4);
                        const bool first = j++ % kTrRun == 0;
                        if (elect_one()) {
                            // keys 16 kk .. 16 kk + 15: hi parts in columns 16 kk ..
                            // 16 kk + 7, lo parts in the next eight
#pragma unroll
                            for (int kk = 0; kk < kTrKeys / 16; ++kk) {
#pragma unroll
                                for (int part = 0; part < 2; ++part)
                                    mma_f16_ts(o, p0 + kTrKeys * buf + 16 * kk + 8 * part, value + kk * (16 * 128 >> 4), kId,
                                               !first || kk > 0 || part > 0);
                            }
                            mma_commit(&room.o_done[slot][buf]);
                            mma_commit(&room.v_empty[back.at]);
                        }
                    } else if (ok && elect_one()) {
                        mbar_arrive(&room.v_empty[back.at]);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) mma_commit(&room.done[kTrSlots + slot]);
            __syncwarp();
            ok = tr_wait(p, &room.done[kTrSlots + slot], 0) && ok;
            if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
        }
    } else if (warp >= kTrConvertWarp) {
        control_registers();
        if constexpr (kFp8) {
            // --------------------------------------------------------------
            // converters, a warp for the even tiles' K, one for their V, and
            // two for the odd tiles'.  A pass brings 16 codes a lane of four
            // rows; lanes are laid out so that eight neighbours read and write
            // different banks: four chunks of a row beside the other four of
            // the next.
            // Each warp sees every other use of an operand stage only, and the
            // slots give a stage back in no order (whoever took no part in it
            // at once, beside products under way): one barrier a stage could
            // have two phases open that a parity does not tell apart.  So tile
            // n comes back on barrier n modulo twice the stages, whose tiles
            // are all one warp's: tile n waits for tile n - S on barrier
            // (n + S) mod 2 S, each of its phases in turn, and the next of them,
            // for tile n + S, needs tile n converted.  A stage of codes, their
            // number being even, is one warp's too.
            // --------------------------------------------------------------
            static_assert(kTrConverters == 4 && Lay::kCodeStages % 2 == 0 && Lay::kKStages == Lay::kVStages &&
                          Lay::kKEmpties == 2 * Lay::kKStages && Lay::kVEmpties == 2 * Lay::kVStages, "see above");
            const int who = warp - kTrConvertWarp;
            const bool keys = (who & 1) == 0;
            const int c = lane & 7, upper = c >> 2;
            const int r4 = 2 * (lane >> 4) + (upper ^ ((lane >> 3) & 1));
            uint64_t* const codes_full = keys ? room.kc_full : room.vc_full;
            uint64_t* const codes_empty = keys ? room.kc_empty : room.vc_empty;
            uint64_t* const full = keys ? room.k_full : room.v_full;
            uint64_t* const empty = keys ? room.k_empty : room.v_empty;
            constexpr int kStages = Lay::kKStages;
            // bits of the row's number that the swizzles use are those of r4,
            // and of pass & 1 for the next four rows
            const uint8_t* const src0 = smem + (keys ? Lay::kKCodes : Lay::kVCodes) + r4 * 128;
            uint8_t* const dst0 = smem + (keys ? Lay::kK : Lay::kV) + upper * Lay::kHalf + r4 * 128;
            int n = 0;
            TrRing<2 * kStages> to;
            TrRing<Lay::kCodeStages> at;
            bool ok = true;
            while (ok && walk.next(p, side, head, P)) {
                for (int k = P.k0; ok && k < P.k1; ++k, ++n, at.step(), to.step()) {
                    if ((n & 1) == (who >> 1)) {
                        const bool upper_lap = to.at >= kStages;
                        const int st = upper_lap ? to.at - kStages : to.at;
                        if (upper_lap || to.lap > 0)
                            ok = tr_wait(p, &empty[upper_lap ? st : st + kStages], upper_lap ? to.lap : to.lap - 1);
                        if (ok) ok = tr_wait(p, &codes_full[at.at], at.lap);
                        if (!ok) break;
                        const uint8_t* src = src0 + at.at * Lay::kCodes;
                        uint8_t* dst = dst0 + st * Lay::kTile;
                        // Four instructions a pair of codes in bf16, one in fp16.
                        // Requesting the next pass's codes a pass ahead takes
                        // longer (64 x up to 2048 tokens in bf16 87.4 us, so 79.2).
#pragma unroll 1
                        for (int i = 0; i < kTrKeys / 16; ++i, src += 16 * 128, dst += 16 * 128) {
                            uint4 x[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[j] = lds128(src + j * 512 + ((c ^ ((r4 + 4 * j) & 7)) << 4));
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t y[8];
#pragma unroll
                                for (int w = 0; w < 4; ++w) {
                                    const uint32_t codes = word_of(x[j], w);
                                    if constexpr (kBf16) {
                                        y[2 * w] = e4m3x2_to<T>((uint16_t)(codes & 0xffffu));
                                        y[2 * w + 1] = e4m3x2_to<T>((uint16_t)(codes >> 16));
                                    } else {
                                        e4m3x4_to_f16x2x2(codes, y[2 * w], y[2 * w + 1]);
                                    }
                                }
                                // chunks 2c and 2c + 1 of the row's 16
                                const int chunk = ((2 * c) & 7) ^ ((r4 + 4 * j) & 7);
                                *reinterpret_cast<uint4*>(dst + j * 512 + (chunk << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                                *reinterpret_cast<uint4*>(dst + j * 512 + ((chunk ^ 1) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&full[st]);
                            mbar_arrive(&codes_empty[at.at]);
                        }
                    }
                }
            }
            if (!ok && lane == 0) flag_error(p.err, PA_DEVERR_WAIT_TIMEOUT);
        }
    } else {
        softmax_registers<tr_softmax_regs(kFp8)>();
        // ------------------------------------------------------------------
        // softmax and epilogue: this thread owns row r of its slot's tiles
        // ------------------------------------------------------------------
        const int slot = (warp >> 2) - 1;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes_at = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tO = tmem + kTrO + lanes_at;                // slot 0's, slot 1's D columns on
        const int barrier = 1 + slot, both = 3;                    // named barriers
        const int in_tile = r / G, in_group = r - in_tile * G;
        const float sl = p.scale_log2;
        const uint64_t sl2 = f32x2_pack(sl, sl);
        bool failed = false;                  // a wait ran out: finish the loops without waiting
        auto wait = [&](uint64_t* bar, int phase) {
            if (!failed && !tr_wait(p, bar, phase)) failed = true;
        };
        auto node_of = [&](const TrPiece& X) { return (kTrSlots * side + (X.share ? slot : 0)) * per_tile + in_tile; };
        auto row_of = [&](const TrPiece& X) {
            return (int64_t)(X.s.q0 + node_of(X)) * p.num_q_heads + X.g * G + in_group;
        };
        int n = 0, t = 0;                     // tiles of the CTA and of the slot so far
        int cleared = 0;                      // of those, V's that this slot has cleared
        for (int piece = 0; walk.next(p, side, head, P); ++piece) {
            const int base = P.s.L - P.s.C;
            const int count = P.k1 - P.k0, own = P.own(slot);
            const int node = node_of(P);
            const bool valid = in_tile < per_tile && node < P.s.C;
            const bool live = __any_sync(0xffffffffu, valid);      // a warp without rows only keeps step
            // this row's line, read where the first key of the tree comes
            TreeLine line{};
            bool taken = false;
            auto take_line = [&] {
                wait(&room.lines_full, piece);
                if (valid && P.k1 * kTrKeys > base) {
                    const uint4 w = room.line[node];
                    line = TreeLine{{w.x, w.y, w.z, w.w}};
                }
                if (P.alone) {                                     // else the statistics come there first
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&room.lines_empty);
                }
                taken = true;
            };
            if (own == 0) {
                take_line();
                n += count;
                continue;
            }
            float m = -INFINITY, l = 0.f;
            float held_m = -INFINITY, held_l = 0.f;                // of the runs before this one
            bool bad = false;                 // V of the tree has elements that are not finite
            // this row's O of those runs, [D / 4][row][4] as in a record; the
            // piece's own record is written when it has been read
            float4* const held = reinterpret_cast<float4*>(p.rec_o) +
                                 (((int64_t)blockIdx.x * 2 + (P.k0 > 0 ? 0 : 1)) * kTrSlots + slot) * (D / 4) * kTrRows + r;
            // What is held in terms of the present reference.
            auto held_scale = [&] { return held_m == m ? 1.f : ex2(held_m - m); };
            const int run = P.share ? kTrRun : 2 * kTrRun;         // of keys: kTrRun tiles of the slot
            const int skip = P.share || P.alone ? 0 : slot;        // to the slot's first tile
            for (int k0 = P.k0; k0 + skip < P.k1; k0 += run) {
                if (k0 > P.k0 && live) {
                    // the run before: added to those before it
                    wait(&room.o_done[slot][(t - 1) & 1], (t - 1) >> 1);
                    tc_fence_after_sync();
                    const float f = held_scale();
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        uint32_t o[32];
                        tmem_ld32(tO + D * slot + d, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            float4 x = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                                   __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
                            float4* at = held + (d / 4 + q) * kTrRows;
                            if (k0 > P.k0 + run) {
                                const float4 y = *at;
                                x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y);
                                x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
                            }
                            *at = x;
                        }
                    }
                    held_l = fmaf(held_l, f, l), l = 0.f, held_m = m;
                }
                for (int k = k0, j = 0; k < min(k0 + run, P.k1); ++k) {
                    if (!P.has(slot, k)) continue;
                    const int key0 = k * kTrKeys;
                    const bool masked = P.masked(k);
                    if (masked && !taken) take_line();
                    const uint32_t tS = tmem + kTrS + kTrKeys * (2 * slot + (t & 1)) + lanes_at;
                    wait(&room.s_full[slot][t & 1], t >> 1);
                    tc_fence_after_sync();
                    if (live) {
                        auto hide = [&](uint32_t(&v)[32], int c) {
                            const uint32_t seen = seen_word(line, key0 + c - base);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = (seen >> e) & 1u ? v[e] : 0xff800000u;
                        };
                        // The row's maximum on the raw scores (the scale is positive),
                        // then P, 32 keys at a time and each time from tensor memory:
                        // held between the two they cost registers and, unrolled,
                        // instruction cache (E4M3 96 us, so 93).
                        float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                        for (int c = 0; c < kTrKeys; c += 32) {
                            uint32_t v[32];
                            tmem_ld32(tS + c, v);
                            tmem_wait_ld(v);
                            if (masked) hide(v, c);
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) pm[i] = fmaxf(pm[i], __uint_as_float(v[e + i]));
                            }
                        }
                        const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])) * sl;
                        const bool raise = mx > m + kRaise;            // the first finite maximum, too
                        if (__any_sync(0xffffffffu, raise)) {
                            const float m_new = raise ? mx - kBelow : m;
                            const float f = raise ? ex2(m - m_new) : 1.f;
                            l *= f;
                            m = m_new;
                            if (j > 0) {
                                wait(&room.o_done[slot][(t - 1) & 1], (t - 1) >> 1);
                                tc_fence_after_sync();
#pragma unroll 1
                                for (int c = 0; c < D; c += 32) {
                                    uint32_t o[32];
                                    tmem_ld32(tO + D * slot + c, o);
                                    tmem_wait_ld(o);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                    tmem_st32(tO + D * slot + c, o);
                                }
                            }
                        }
                        const float ref = m == -INFINITY ? 0.f : m;    // nothing seen yet
                        const uint64_t neg2 = f32x2_pack(-ref, -ref);
                        uint64_t ps[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
                        for (int c = 0; c < kTrKeys; c += 32) {
                            uint32_t v[32];
                            tmem_ld32(tS + c, v);
                            tmem_wait_ld(v);
                            if (masked) hide(v, c);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t parts[16];                    // hi, then lo
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    float a0, a1;
                                    f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(v[16 * h + 2 * i]),
                                                                      __uint_as_float(v[16 * h + 2 * i + 1])), sl2, neg2), a0, a1);
                                    const float p0 = ex2(a0), p1 = ex2(a1);
                                    ps[i & 3] = f32x2_add(ps[i & 3], f32x2_pack(p0, p1));
                                    split_pair<T>(p0, p1, parts[i], parts[8 + i]);
                                }
                                tmem_st16(tS + c + 16 * h, parts);
                            }
                        }
                        float q8[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) f32x2_unpack(ps[e], q8[2 * e], q8[2 * e + 1]);
                        l += ((q8[0] + q8[1]) + (q8[2] + q8[3])) + ((q8[4] + q8[5]) + (q8[6] + q8[7]));
                        // the next tile's scores, where they are there already
                        tmem_wait_st();
                    }
                    if (masked) {
                        // V rows past the context may hold anything: clear them.
                        // Of the tree's, elements that are not finite are cleared
                        // too, since the tensor cores would carry them into rows
                        // that do not see them; rows that do get them back below.
                        // Thread r has half r / 64 of key r % 64.  That the tile is
                        // there its issuer of P V says, which waits for every phase
                        // of V's barriers in turn: this slot's tile before may be
                        // five back (the last but one of a piece, two that the
                        // other slot took alone, the first of this one), so a
                        // parity alone could be that of an earlier tile.
                        bool odd = false;
                        if (P.clears(slot)) {
                            const int tile = n + (k - P.k0), vs = tile % Lay::kVStages;
                            wait(&room.v_there[slot], cleared++);
                            wait(&room.v_full[vs], tile / Lay::kVStages);
                            const int key = key0 + (r & 63);
                            uint8_t* vd = smem + Lay::kV + vs * Lay::kTile + (D == 128 ? (r >> 6) * Lay::kHalf : 0) +
                                          (r & 63) * 128;
                            if (D == 64 && r >= 64) {
                            } else if (key >= P.s.L) {
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    *reinterpret_cast<uint4*>(vd + (((c ^ r) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                            } else if (key >= base) {
                                uint32_t any = 0u;
#pragma unroll
                                for (int c = 0; c < 8; ++c) {
                                    const uint4 w = lds128(vd + (((c ^ r) & 7) << 4));
                                    any |= not_finite<T>(w.x) | not_finite<T>(w.y) | not_finite<T>(w.z) | not_finite<T>(w.w);
                                }
                                if (any != 0u) {
                                    odd = true;
                                    for (int c = 0; c < 32; ++c) {
                                        uint32_t* w = reinterpret_cast<uint32_t*>(vd) + c;
                                        *w &= ~(((not_finite<T>(*w) >> 15) & 0x00010001u) * 0xffffu);
                                    }
                                }
                            }
                            fence_proxy_async_smem();
                        }
                        bad |= P.share ? bar_or(both, 2 * kTrRows, odd) : bar_or(barrier, kTrRows, odd);
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&room.p_full[slot][t & 1]);
                    ++t, ++j;
                }
            }
            n += count;
            // ---- the piece's end ------------------------------------------------
            if (!taken) take_line();
            if (own > 0) {
                wait(&room.o_done[slot][(t - 1) & 1], (t - 1) >> 1);
                tc_fence_after_sync();
                if (live && own > kTrRun) {
                    const float f = held_scale();
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        uint32_t o[32];
                        tmem_ld32(tO + D * slot + d, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float4 y = held[(d / 4 + q) * kTrRows];
                            o[4 * q] = __float_as_uint(fmaf(y.x, f, __uint_as_float(o[4 * q])));
                            o[4 * q + 1] = __float_as_uint(fmaf(y.y, f, __uint_as_float(o[4 * q + 1])));
                            o[4 * q + 2] = __float_as_uint(fmaf(y.z, f, __uint_as_float(o[4 * q + 2])));
                            o[4 * q + 3] = __float_as_uint(fmaf(y.w, f, __uint_as_float(o[4 * q + 3])));
                        }
                        tmem_st32(tO + D * slot + d, o);
                    }
                    tmem_wait_st();
                    l = fmaf(held_l, f, l);
                }
                const bool full = count == P.n;
                const int64_t rec = ((int64_t)blockIdx.x * 2 + (P.k0 > 0 ? 0 : 1)) * kTrSlots + (P.share ? slot : 0);
                float w0 = slot == 0 ? 1.f : 0.f, w1 = 1.f - w0, top = m;
                if (!P.alone) {
                    // both slots have this row: joined, a half of the dims each
                    bar_sync(both, 2 * kTrRows);                   // the lines are not read any more
                    room.ml[slot][r] = make_float2(m, l);
                    tc_fence_before_sync();
                    bad = bar_or(both, 2 * kTrRows, bad);
                    tc_fence_after_sync();
                    const float2 a = room.ml[0][r], b = room.ml[1][r];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&room.lines_empty);
                    top = fmaxf(a.x, b.x);
                    const float ref = top == -INFINITY ? 0.f : top;
                    w0 = ex2(a.x - ref), w1 = ex2(b.x - ref);
                    l = a.y * w0 + b.y * w1;
                }
                const int from = P.alone ? 0 : slot * (D / 2), to = P.alone ? D : from + D / 2;
                const float norm = full ? (kFp8 ? p.v_scale : 1.f) / l : 1.f;
                const bool use0 = !P.alone || slot == 0, use1 = !P.alone || slot == 1;
                w0 *= norm, w1 *= norm;
                const int64_t row = row_of(P);
#pragma unroll 1
                for (int d = from; live && d < to; d += 32) {
                    float o[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                    uint32_t v[32];
                    if (use0) {
                        tmem_ld32(tO + d, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(v[e]) * w0;
                    }
                    if (use1) {
                        tmem_ld32(tO + D + d, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(v[e]), w1, o[e]);
                    }
                    if (!valid || failed) {
                    } else if (full) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * D + d);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            dst[q] = make_uint4(M::pack(o[8 * q], o[8 * q + 1]), M::pack(o[8 * q + 2], o[8 * q + 3]),
                                                M::pack(o[8 * q + 4], o[8 * q + 5]), M::pack(o[8 * q + 6], o[8 * q + 7]));
                    } else {
                        // [D / 4][row][4]: a warp writes whole lines
                        float4* dst = reinterpret_cast<float4*>(p.rec_o) + (rec * (D / 4) + d / 4) * kTrRows + r;
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dst[q * kTrRows] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                    }
                    __syncwarp();
                }
                if (bad && valid && !failed) {
                    // what was taken out of V, for a row that sees it: the sums are
                    // what adding it gives
                    for (int i = 0; i < P.s.C; ++i) {
                        const int key = base + i;
                        if (!line.has(i) || key < P.k0 * kTrKeys || key >= P.k1 * kTrKeys) continue;
                        const int blk = p.block_tables[(size_t)P.b * p.max_blocks_per_seq + key / p.block_size];
                        if (blk < 0 || blk >= p.num_blocks) continue;
                        const int64_t at = (((int64_t)blk * p.block_size + key % p.block_size) * p.num_kv_heads + P.g) * D;
#pragma unroll 1
                        for (int d = from; d < to; ++d) {
                            float y;
                            if constexpr (kFp8)
                                y = (static_cast<const uint8_t*>(p.v_cache)[at + d] & 0x7f) == 0x7f ? NAN : 0.f;
                            else
                                y = (float)static_cast<const T*>(p.v_cache)[at + d];
                            if (isfinite(y)) continue;
                            if (full) {
                                T& o = static_cast<T*>(p.out)[row * D + d];
                                o = from_float<T>((float)o + y);
                            } else {
                                p.rec_o[((rec * (D / 4) + d / 4) * kTrRows + r) * 4 + d % 4] += y;
                            }
                        }
                    }
                }
                if (!full && valid && !failed && (P.alone || slot == 0)) p.rec_ml[rec * kTrRows + r] = make_float2(top, l);
                // O of both slots is read: the next piece's products may overwrite it
                tc_fence_before_sync();
                if (!P.alone) bar_sync(both, 2 * kTrRows);
                __syncwarp();
            }
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

// Joins the records of the pairs that more than one lane met: a CTA for some
// rows of the pair that the range of lane blockIdx.x + 1 begins in, where that
// is the first range to begin there, or of pair blockIdx.x where there are few
// pairs (tr_merge_pairs); a lane per row, eight dims each.  Which
// pair that is it finds while the attention kernel ends: lengths and trees are
// not written by it, and it has waited for whoever wrote them.
constexpr int kTrMergeThreads = 256;
constexpr int kTrMergeDims = 8;                // of a thread

// Whether the joining grid goes by pairs, which finds its place with one load a
// lane, or by ranges, which walks.  One pair on 19 ranges 58.9 us by pairs and
// 65.0 by ranges (50,000 tokens), 20.3 and 23.9 (4096), four 14.1 and 15.1; 16
// pairs on 19 ranges 26.4 and 22.9: by pairs where there are two ranges a pair.
// A pair then has many records, and eight are requested at a time (one KV head,
// 50,000 tokens: four 28.2 us, eight 24.8); by ranges it has two or three, and
// the CTAs are small enough to be there all at once (64 of up to 2048 tokens,
// three CTAs an SM 62.6 us, five 61.0).
__host__ __device__ __forceinline__ bool tr_merge_pairs(const TreeParams& p) {
    return (int64_t)p.num_seqs * (p.num_kv_heads / p.heads) * 2 < p.ctas;
}

// A pair to join: its lanes [c0, c1], nodes (none: nothing to join) and their
// first row, and KV head.
struct TrJoin {
    unsigned c0, c1;
    int C, q0, g;
};

// By a warp.
template <bool kPairs>
__device__ __forceinline__ TrJoin tree_join(const TreeParams& p, int side, int head) {
    TrWalk<true> walk;
    const TrDeal deal(p, walk.count(p, false));
    TrPiece P;
    unsigned begin = 0, each = 0;
    bool join;
    if (kPairs) {
        const int per_seq = p.num_kv_heads / p.heads;
        P.b = blockIdx.x / per_seq;
        P.s = tree_sequence<true>(p, P.b, false);
        P.g = head + (int)blockIdx.x % per_seq * p.heads;
        unsigned before = 0;
        for (int i = threadIdx.x & 31; i < P.b; i += 32) before += TrWalk<true>::weight(p, tree_sequence<true>(p, i, false));
        each = TrWalk<true>::each(p, P.s);
        begin = __reduce_add_sync(0xffffffffu, before) + (unsigned)(blockIdx.x % per_seq) * each;
        join = P.s.C > 0;
    } else {
        walk.at = deal.begin(min(blockIdx.x + 1, deal.ctas));
        join = blockIdx.x + 1 < deal.ctas && walk.find(p, side, head, P, begin, each);
    }
    TrJoin x{0u, 0u, 0, 0, 0};
    if (!join) return x;
    // from the lane that has the first tile to the one that has the last
    x.c0 = deal.cta_of(begin + kTrPairWeight), x.c1 = deal.cta_of(begin + each - 1);
    x.q0 = P.s.q0, x.g = P.g;
    if (x.c1 > x.c0 && (kPairs || x.c0 == blockIdx.x)) x.C = P.s.C;
    return x;
}

template <typename T, int D, bool kFp8, bool kPairs>
__global__ void __launch_bounds__(kTrMergeThreads, kPairs ? 2 : 5)
    tree_merge_kernel(const __grid_constant__ TreeParams p) {
    allow_dependent_launch();
    const int head = blockIdx.y % p.heads, side = blockIdx.y / p.heads;
    // (dims, rows) of this thread: 32 rows a warp, the dims of a row in D / 8 warps
    constexpr int kParts = D / kTrMergeDims;
    const int at = blockIdx.z * (kTrMergeThreads / 32) + (int)(threadIdx.x >> 5);
    const int d = at % kParts * kTrMergeDims, row = at / kParts * 32 + (int)(threadIdx.x & 31);
    const int slot = row / kTrRows, r = row % kTrRows;
    // a warp finds the pair for all: every warp by itself, 4600 of them read the
    // same few lines of the L2
    __shared__ TrJoin found;
    if (threadIdx.x < 32) {
        const TrJoin x = tree_join<kPairs>(p, side, head);
        if (threadIdx.x == 0) found = x;
    }
    __syncthreads();
    const TrJoin J = found;
    // whoever has nothing to join makes room, but the grid is not over before
    // the attention kernel is: its first CTA waits
    if (J.C == 0 && (blockIdx.x | blockIdx.y | blockIdx.z) != 0) return;
    grid_dependency_wait();
    const int G = p.group, per_tile = tr_nodes_per_tile(G);
    const int in_tile = r / G, node = (kTrSlots * side + slot) * per_tile + in_tile;
    if (in_tile >= per_tile || node >= J.C) return;
    const unsigned c0 = J.c0, c1 = J.c1;
    float m = -INFINITY, l = 0.f, o[kTrMergeDims] = {};
    constexpr int kAhead = kPairs ? 8 : 2;
    for (unsigned c = c0; c <= c1; c += kAhead) {
        float2 ml[kAhead];
        float4 v[kAhead][2];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            ml[i] = make_float2(-INFINITY, 0.f);
            if (c + i > c1) continue;
            const int64_t cta = ((int64_t)(c + i) * p.sides + side) * p.heads + head;
            const int64_t rec = (cta * 2 + (c + i == c0 ? 1 : 0)) * kTrSlots + slot;
            ml[i] = p.rec_ml[rec * kTrRows + r];
            const float4* src = reinterpret_cast<const float4*>(p.rec_o) + (rec * (D / 4) + d / 4) * kTrRows + r;
            v[i][0] = src[0], v[i][1] = src[kTrRows];
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) top = fmaxf(top, ml[i].x);
        const float ref = top == -INFINITY ? 0.f : top, f = ex2(m - ref);
        m = top;
        l *= f;
#pragma unroll
        for (int k = 0; k < kTrMergeDims; ++k) o[k] *= f;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (c + i > c1) continue;
            const float w = ex2(ml[i].x - ref);
            l += w * ml[i].y;
            o[0] += w * v[i][0].x, o[1] += w * v[i][0].y, o[2] += w * v[i][0].z, o[3] += w * v[i][0].w;
            o[4] += w * v[i][1].x, o[5] += w * v[i][1].y, o[6] += w * v[i][1].z, o[7] += w * v[i][1].w;
        }
    }
    using M = Mma<T>;
    const float norm = (kFp8 ? p.v_scale : 1.f) / l;
    T* dst = static_cast<T*>(p.out) + ((int64_t)(J.q0 + node) * p.num_q_heads + J.g * G + (r - in_tile * G)) * D + d;
    *reinterpret_cast<uint4*>(dst) = make_uint4(M::pack(o[0] * norm, o[1] * norm), M::pack(o[2] * norm, o[3] * norm),
                                                M::pack(o[4] * norm, o[5] * norm), M::pack(o[6] * norm, o[7] * norm));
}

size_t tree_plan(TreeParams& p, int head_dim, void* workspace) {
    const int per_tile = kTrRows / p.group;
    const int query_tiles = (p.max_query + per_tile - 1) / per_tile;
    const int tiles = (p.max_context + kTrKeys - 1) / kTrKeys;
    p.sides = query_tiles > kTrSlots ? (query_tiles + kTrSlots - 1) / kTrSlots : 1;
    // as many KV heads side by side as leave at most 4 % of the SMs without a CTA
    p.heads = 1;
    for (int d = 2; d <= p.num_kv_heads && d * p.sides <= kTrCtas; ++d)
        if (p.num_kv_heads % d == 0 && kTrCtas / (d * p.sides) * (d * p.sides) * 25 >= kTrCtas * 24) p.heads = d;
    const int lanes = kTrCtas / (p.heads * p.sides);
    const int64_t pairs = (int64_t)p.num_seqs * (p.num_kv_heads / p.heads);       // of a lane's CTA
    p.whole = tiles <= (pairs <= lanes && 2 * pairs > lanes ? kTrWholeTilesAlone : kTrWholeTiles);
    auto of_lanes = [&](int64_t most) { return (int)(most < lanes ? (most > 0 ? most : 1) : lanes); };
    const int dealt = of_lanes((pairs * (tiles + kTrPairWeight) + kTrMinTiles - 1) / kTrMinTiles);
    p.ctas = p.whole ? of_lanes(pairs) : dealt;
    // as if dealt out: what is enough for a batch is enough with fewer sequences
    const size_t rows = tiles <= kTrWholeTiles ? 0 : (size_t)dealt * p.heads * p.sides * 2 * kTrSlots * kTrRows;
    p.rec_o = static_cast<float*>(workspace);
    p.rec_ml = reinterpret_cast<float2*>(p.rec_o + rows * head_dim);
    return rows * (head_dim * sizeof(float) + sizeof(float2)) + 16;
}

template <typename T, int D, bool kFp8>
cudaError_t launch_tree_t(const CUtensorMap& tmk, const CUtensorMap& tmv, const CUtensorMap& tmq, const TreeParams& p,
                          cudaStream_t stream) {
    constexpr int kSmem = tr_smem<D, kFp8>();
    cudaError_t e = cudaFuncSetAttribute(tree_attention_kernel<T, D, kFp8>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    e = launch_with_pdl(tree_attention_kernel<T, D, kFp8>, dim3((unsigned)(p.ctas * p.sides * p.heads)), dim3(tr_threads(kFp8)), kSmem,
                        stream, tmk, tmv, tmq, p);
    if (e != cudaSuccess || p.whole) return e;
    if (p.ctas == 1) return e;
    // rows of the slots, by 32
    const int per_tile = kTrRows / p.group;
    const int rows = p.max_query > per_tile ? kTrSlots * kTrRows : (p.max_query * p.group + 31) / 32 * 32;
    const int chunks = (rows / 32 * (D / kTrMergeDims) + kTrMergeThreads / 32 - 1) / (kTrMergeThreads / 32);
    const bool pairs = tr_merge_pairs(p);
    return launch_with_pdl(pairs ? tree_merge_kernel<T, D, kFp8, true> : tree_merge_kernel<T, D, kFp8, false>,
                           dim3((unsigned)(pairs ? p.num_seqs * (p.num_kv_heads / p.heads) : p.ctas - 1),
                                (unsigned)(p.heads * p.sides), (unsigned)chunks),
                           dim3(kTrMergeThreads), 0, stream, p);
}

cudaError_t launch_tree_attention(int dtype, int head_dim, bool fp8, const CUtensorMap& tmk,
                                  const CUtensorMap& tmv, const CUtensorMap& tmq, const TreeParams& p,
                                  cudaStream_t stream) {
    const bool bf16 = dtype == PA_BF16;
    if (fp8) return bf16 ? launch_tree_t<__nv_bfloat16, 128, true>(tmk, tmv, tmq, p, stream)
                         : launch_tree_t<__half, 128, true>(tmk, tmv, tmq, p, stream);
    if (head_dim == 64) return bf16 ? launch_tree_t<__nv_bfloat16, 64, false>(tmk, tmv, tmq, p, stream)
                                    : launch_tree_t<__half, 64, false>(tmk, tmv, tmq, p, stream);
    return bf16 ? launch_tree_t<__nv_bfloat16, 128, false>(tmk, tmv, tmq, p, stream)
                : launch_tree_t<__half, 128, false>(tmk, tmv, tmq, p, stream);
}

int tree_nodes_per_tile(int group) { return kTrRows / group; }

}  // namespace pa
