// Rotary positions of the new tokens' queries and keys together with the
// cache write: q and k are turned, k and v go to their slots (16-bit, or
// E4M3 codes of x / scale), all in one pass over the data.
//
// A pair (a, b) of a head's first R dims turns by t = position * inv_freq[i]:
//   a' = f (a cos t - b sin t),  b' = f (b cos t + a sin t),
// with pairs (i, i + R/2) or, interleaved, (2i, 2i + 1).  The angle is kept
// in turns as 64-bit fixed point: inv_freq / 2 pi times 2^64, times the
// position in wrapping integer arithmetic, so whole turns drop out exactly.
// The error is that of the turns per position, 2^-52 of the unreduced angle
// (1 / 2 pi and the product in 64 bits) and 2^-64 turns per position, and the
// phase's rounding to fp32, 2^-26 turns.  Products and sums are in fp32; each
// result is rounded once.
//
// With kNorm each head x of q and k is first taken to w x / sqrt(mean x^2 +
// eps), in fp32 and not rounded in between, and a pair's position is that of
// its axis.  The D / 16 threads that hold a head add up its squares by
// shuffles among themselves.
#include <type_traits>

#include "bounded_internal.h"
#include "pa_device.cuh"

namespace pa {

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 9;                  // per SM
// The same behind a norm, whose sums and weights take registers.
__host__ __device__ constexpr int norm_ctas(bool fp8) { return fp8 ? 9 : 8; }

// Position-independent part of the angle: turns per position, in 2^-64.
__device__ __forceinline__ int64_t rope_turns(float inv_freq) {
    const double t = (double)inv_freq * 0.15915494309189535;          // 1 / 2 pi
    return __double2ll_rn((t - rint(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ float2 rope_cos_sin(int64_t turns, int64_t position, float factor) {
    const int64_t phase = (int64_t)((uint64_t)turns * (uint64_t)position);
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    return make_float2(c * factor, s * factor);
}

template <typename T>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = Mma<T>::unpack(w[j]);
        x[2 * j] = f.x, x[2 * j + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(Mma<T>::pack(x[0], x[1]), Mma<T>::pack(x[2], x[3]),
                      Mma<T>::pack(x[4], x[5]), Mma<T>::pack(x[6], x[7]));
}

__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float scale) {
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        q[j] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * j + 1], scale), __fdiv_rn(x[2 * j], scale));
    return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// A CTA serves kTokens tokens.  A thread's item is 16 dims of one head of one
// token, two 16-byte chunks: the two halves of eight pairs, or two chunks
// past the rotated dims.  A thread keeps its place u inside the head and
// walks the heads of its CTA's tokens, q first, kRopeBatch at a time with all
// their loads in flight, then k and v of a head together; the first batch is
// requested before the positions have arrived and while cos and sin are formed.
constexpr int kRopeBatch = 2;
enum RopeRows { kRopeQ, kRopeK, kRopeV };
// places of the batch: q takes both for two heads, k and v one each
template <int kFirst, int kEnd>
struct RopePlaces {
    static constexpr int kFrom = kFirst, kTo = kEnd;
};

template <typename T, int D, bool kFp8, bool kInterleaved, bool kNorm, int kTokens>
__global__ void __launch_bounds__(kRopeThreads, kNorm ? norm_ctas(kFp8) : kRopeCtas)
    rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kUnits = D / 16, kHeads = kRopeThreads / kUnits;      // items side by side
    // cos and sin of pairs 8 u + 2 j and the next, and weights 8 c + 4 j .. + 3,
    // at [j][u] and [j][c]: a head's threads read neighbouring words
    __shared__ __align__(16) float4 cs[kTokens][4][kUnits];
    __shared__ int64_t slot_s[kTokens];
    __shared__ __align__(16) float4 weight_s[kNorm ? 2 : 1][2][kNorm ? D / 8 : 1];      // of q, of k
    grid_dependency_wait();
    allow_dependent_launch();
    const int tid = threadIdx.x, u = tid % kUnits, first = tid / kUnits;
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    const int tokens = (int)min((int64_t)kTokens, p.num_tokens - t0);
    const int turned = p.rotary_dim / 16;              // units with rotated pairs
    const bool rot = u < turned;
    const int c0 = rot && !kInterleaved ? u : 2 * u;   // chunks of q and k; v: 2u, 2u + 1
    const int c1 = rot && !kInterleaved ? u + turned : 2 * u + 1;
    auto token_of = [&](int v, int heads) {
        int tk = 0;
#pragma unroll
        for (int i = 1; i < kTokens; ++i) tk += v >= i * heads;
        return tk;
    };
    uint4 v0[kRopeBatch], v1[kRopeBatch];
    auto load = [&](auto rows, auto places, int at) {
        constexpr int kRows = decltype(rows)::value, kFrom = decltype(places)::kFrom, kTo = decltype(places)::kTo;
        const int heads = kRows == kRopeQ ? p.num_q_heads : p.num_kv_heads;
        const T* base = static_cast<const T*>(kRows == kRopeQ ? p.q : (kRows == kRopeK ? p.k : p.v));
        const int64_t stride = kRows == kRopeQ ? p.q_stride : (kRows == kRopeK ? p.k_stride : p.v_stride);
#pragma unroll
        for (int k = kFrom; k < kTo; ++k) {
            const int v = at + (k - kFrom) * kHeads;
            if (v >= tokens * heads) break;
            const int tk = token_of(v, heads);
            const uint4* src = reinterpret_cast<const uint4*>(base + (t0 + tk) * stride + (v - tk * heads) * D);
            v0[k] = src[kRows == kRopeV ? 2 * u : c0];
            v1[k] = src[kRows == kRopeV ? 2 * u + 1 : c1];
        }
    };
    auto store = [&](auto rows, auto places, int at) {
        constexpr int kRows = decltype(rows)::value, kFrom = decltype(places)::kFrom, kTo = decltype(places)::kTo;
        const int heads = kRows == kRopeQ ? p.num_q_heads : p.num_kv_heads;
#pragma unroll
        for (int k = kFrom; k < kTo; ++k) {
            const int v = at + (k - kFrom) * kHeads;
            if (v >= tokens * heads) break;
            const int tk = token_of(v, heads), h = v - tk * heads;
            const int64_t slot = kRows == kRopeQ ? 0 : slot_s[tk];
            if (slot < 0) continue;
            constexpr bool kCodes = kFp8 && kRows != kRopeQ;
            float x0[8], x1[8];
            if (kCodes || (kRows != kRopeV && (rot || kNorm))) {
                unpack8<T>(v0[k], x0);
                unpack8<T>(v1[k], x1);
            }
            if constexpr (kNorm && kRows != kRopeV) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(x0[j], x0[j], fmaf(x1[j], x1[j], sum));
                // the head's threads run together
                const uint32_t head = ((1u << kUnits) - 1u) << ((int)(threadIdx.x & 31u) & ~(kUnits - 1));
#pragma unroll
                for (int d = kUnits / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(head, sum, d);
                const float inv = rsqrtf(fmaf(sum, 1.f / D, p.eps));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 a = weight_s[kRows][j][c0], b = weight_s[kRows][j][c1];
                    x0[4 * j] *= inv * a.x, x0[4 * j + 1] *= inv * a.y;
                    x0[4 * j + 2] *= inv * a.z, x0[4 * j + 3] *= inv * a.w;
                    x1[4 * j] *= inv * b.x, x1[4 * j + 1] *= inv * b.y;
                    x1[4 * j + 2] *= inv * b.z, x1[4 * j + 3] *= inv * b.w;
                }
            }
            if (kRows != kRopeV && rot) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 w = cs[tk][j][u];                                     // two pairs
                    if (kInterleaved) {
                        float(&x)[8] = j < 2 ? x0 : x1;
                        const int o = 4 * (j & 1);
                        const float r0 = x[o] * w.x - x[o + 1] * w.y, r1 = x[o + 2] * w.z - x[o + 3] * w.w;
                        x[o + 1] = x[o + 1] * w.x + x[o] * w.y;
                        x[o + 3] = x[o + 3] * w.z + x[o + 2] * w.w;
                        x[o] = r0, x[o + 2] = r1;
                    } else {
                        const float r0 = x0[2 * j] * w.x - x1[2 * j] * w.y;
                        const float r1 = x0[2 * j + 1] * w.z - x1[2 * j + 1] * w.w;
                        x1[2 * j] = x1[2 * j] * w.x + x0[2 * j] * w.y;
                        x1[2 * j + 1] = x1[2 * j + 1] * w.z + x0[2 * j + 1] * w.w;
                        x0[2 * j] = r0, x0[2 * j + 1] = r1;
                    }
                }
            }
            if (!kCodes && kRows != kRopeV && (rot || kNorm)) v0[k] = pack8<T>(x0), v1[k] = pack8<T>(x1);
            const int d0 = kRows == kRopeV ? 2 * u : c0, d1 = kRows == kRopeV ? 2 * u + 1 : c1;
            if (kRows == kRopeQ) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + (t0 + tk) * p.q_out_stride + h * D);
                dst[d0] = v0[k], dst[d1] = v1[k];
            } else if (kCodes) {
                const float sc = kRows == kRopeK ? p.k_scale : p.v_scale;
                uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(kRows == kRopeK ? p.k_cache : p.v_cache) +
                                                      (slot * heads + h) * D);
                const uint2 q0 = quantise8(x0, sc), q1 = quantise8(x1, sc);
                // two neighbouring chunks go out as one
                if (kRows == kRopeV || kInterleaved || !rot)
                    *reinterpret_cast<uint4*>(dst + d0) = make_uint4(q0.x, q0.y, q1.x, q1.y);
                else
                    dst[d0] = q0, dst[d1] = q1;
            } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(kRows == kRopeK ? p.k_cache : p.v_cache) +
                                                      (slot * heads + h) * D);
                dst[d0] = v0[k], dst[d1] = v1[k];
            }
        }
    };
    using Q = std::integral_constant<int, kRopeQ>;
    using K = std::integral_constant<int, kRopeK>;
    using V = std::integral_constant<int, kRopeV>;
    using All = RopePlaces<0, kRopeBatch>;
    using First = RopePlaces<0, 1>;
    using Second = RopePlaces<1, 2>;
    load(Q(), All(), first);
    const int pairs = p.rotary_dim / 2;
    for (int i = tid; i < tokens * pairs; i += kRopeThreads) {
        const int tk = i / pairs, j = i - tk * pairs;
        int64_t row = t0 + tk;
        if constexpr (kNorm) {
            const int axis = p.axes ? p.axes[j] : 0;
            if (axis >= 0 && axis < p.num_axes)
                row += axis * p.num_tokens;
            else
                flag_error(p.err, PA_DEVERR_BAD_INDEX);
        }
        reinterpret_cast<float2*>(&cs[tk][j % 8 / 2][j / 8])[j & 1] =
            rope_cos_sin(rope_turns(p.inv_freq[j]), p.positions[row], p.factor);
    }
    if constexpr (kNorm) {
        static_assert(kRopeThreads >= D, "a thread per weight");
        if (tid < D) {
            const float wq = p.q_weight ? (float)static_cast<const T*>(p.q_weight)[tid] : 1.f;
            const float wk = p.k_weight ? (float)static_cast<const T*>(p.k_weight)[tid] : 1.f;
            reinterpret_cast<float*>(&weight_s[kRopeQ][tid % 8 / 4][tid / 8])[tid & 3] = wq;
            reinterpret_cast<float*>(&weight_s[kRopeK][tid % 8 / 4][tid / 8])[tid & 3] = wk;
        }
    }
    if (tid < tokens) {
        const int64_t slot = p.slots[t0 + tid];
        slot_s[tid] = slot < p.num_slots ? slot : -1;
        if (slot >= p.num_slots) flag_error(p.err, PA_DEVERR_BAD_SLOT);
    }
    __syncthreads();
    store(Q(), All(), first);
    for (int at = first + kRopeBatch * kHeads; at < tokens * p.num_q_heads; at += kRopeBatch * kHeads) {
        load(Q(), All(), at);
        store(Q(), All(), at);
    }
    for (int at = first; at < tokens * p.num_kv_heads; at += kHeads) {
        load(K(), First(), at);
        load(V(), Second(), at);
        store(K(), First(), at);
        store(V(), Second(), at);
    }
}

// Many small CTAs keep the grid's last wave short: 8192 tokens of 64 + 16
// heads (336 MB) take 52.2 us with 128 threads, two tokens and nine CTAs an SM
// (6.4 TB/s, 95 % of the copy rate; 58.9 with 256 threads, four tokens and four
// CTAs); into an E4M3 cache, 5001 tokens of 32 + 16 heads 20.7 (with eight
// CTAs 21.8).  Behind a norm the same take 54.8 us (ten CTAs 59.8, four tokens
// 68) and 25.9 (eight 26.7, ten 30.9); with cos, sin and weights in the order
// of the pairs, a head's threads on the same banks, they took 65.5 and 30.4.
// A single wave of tokens goes one to a CTA, which spreads it wider.
template <typename T, int D, bool kFp8, bool kInterleaved, bool kNorm>
cudaError_t launch_rope_i(const RopeParams& p, cudaStream_t stream) {
    const dim3 threads(kRopeThreads);
    if (p.num_tokens <= 152 * kRopeCtas)
        return launch_with_pdl(rope_and_cache_kernel<T, D, kFp8, kInterleaved, kNorm, 1>,
                               dim3((unsigned)p.num_tokens), threads, 0, stream, p);
    return launch_with_pdl(rope_and_cache_kernel<T, D, kFp8, kInterleaved, kNorm, 2>,
                           dim3((unsigned)((p.num_tokens + 1) / 2)), threads, 0, stream, p);
}

template <typename T, int D, bool kFp8>
cudaError_t launch_rope_t(bool interleaved, bool norm, const RopeParams& p, cudaStream_t stream) {
    if (norm) return interleaved ? launch_rope_i<T, D, kFp8, true, true>(p, stream)
                                 : launch_rope_i<T, D, kFp8, false, true>(p, stream);
    return interleaved ? launch_rope_i<T, D, kFp8, true, false>(p, stream)
                       : launch_rope_i<T, D, kFp8, false, false>(p, stream);
}

cudaError_t launch_rope_and_cache(int dtype, int head_dim, bool fp8, bool interleaved, bool norm,
                                  const RopeParams& p, cudaStream_t stream) {
    const bool bf16 = dtype == PA_BF16;
    if (fp8) return bf16 ? launch_rope_t<__nv_bfloat16, 128, true>(interleaved, norm, p, stream)
                         : launch_rope_t<__half, 128, true>(interleaved, norm, p, stream);
    if (head_dim == 64) return bf16 ? launch_rope_t<__nv_bfloat16, 64, false>(interleaved, norm, p, stream)
                                    : launch_rope_t<__half, 64, false>(interleaved, norm, p, stream);
    return bf16 ? launch_rope_t<__nv_bfloat16, 128, false>(interleaved, norm, p, stream)
                : launch_rope_t<__half, 128, false>(interleaved, norm, p, stream);
}

}  // namespace pa
