// Rotary positions of the new tokens' queries and keys together with the
// cache write: q and k are turned, k and v go to their slots (16-bit, or
// E4M3 codes of x / scale), all in one pass over the data.
//
// A pair (a, b) of a head's first R dims turns by t = position * inv_freq[i]:
//   a' = f (a cos t - b sin t),  b' = f (b cos t + a sin t),
// with pairs (i, i + R/2) or, interleaved, (2i, 2i + 1).  The angle is kept
// in turns as 64-bit fixed point: inv_freq / 2 pi times 2^64, times the
// position in wrapping integer arithmetic, so whole turns drop out exactly
// and the error is 2^-53 of the unreduced angle plus 2^-33 turns, at any
// position.  Products and sums are in fp32; each result is rounded once.
#include "bounded_internal.h"
#include "pa_device.cuh"

namespace pa {

constexpr int kRopeThreads = 256;

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

// One CTA per token.  A thread's unit of work is 16 dims of one head, two
// 16-byte chunks: the two halves of eight pairs, or two chunks past the
// rotated dims.
template <typename T, int D, bool kFp8, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads)
    rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kUnits = D / 16;
    __shared__ float2 cs[D / 2];
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t t = blockIdx.x;
    const int turned = p.rotary_dim / 16;              // units with rotated pairs
    const int64_t position = p.positions[t];
    const int64_t slot = p.slots[t];
    if (slot >= p.num_slots && threadIdx.x == 0) flag_error(p.err, PA_DEVERR_BAD_SLOT);
    const bool cached = slot >= 0 && slot < p.num_slots;
    for (int i = threadIdx.x; i < p.rotary_dim / 2; i += kRopeThreads)
        cs[i] = rope_cos_sin(rope_turns(p.inv_freq[i]), position, p.factor);
    __syncthreads();
    const int hq = p.num_q_heads, hkv = p.num_kv_heads;
    const int units = (hq + (cached ? 2 * hkv : 0)) * kUnits;
    for (int i = threadIdx.x; i < units; i += kRopeThreads) {
        int h = i / kUnits;
        const int u = i % kUnits;
        const bool is_q = h < hq, is_v = h >= hq + hkv;
        const bool rot = !is_v && u < turned;
        const int c0 = rot && !kInterleaved ? u : 2 * u;
        const int c1 = rot && !kInterleaved ? u + turned : 2 * u + 1;
        h -= is_q ? 0 : (is_v ? hq + hkv : hq);
        const T* src = static_cast<const T*>(is_q ? p.q : (is_v ? p.v : p.k)) +
                       t * (is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride)) + h * D;
        uint4 v0 = reinterpret_cast<const uint4*>(src)[c0];
        uint4 v1 = reinterpret_cast<const uint4*>(src)[c1];
        float x0[8], x1[8];
        if (rot || kFp8) {
            unpack8<T>(v0, x0);
            unpack8<T>(v1, x1);
        }
        if (rot) {
            const float2* a = cs + 8 * u;
            if (kInterleaved) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 e = a[j], f = a[4 + j];
                    const float r0 = x0[2 * j] * e.x - x0[2 * j + 1] * e.y;
                    const float r1 = x1[2 * j] * f.x - x1[2 * j + 1] * f.y;
                    x0[2 * j + 1] = x0[2 * j + 1] * e.x + x0[2 * j] * e.y;
                    x1[2 * j + 1] = x1[2 * j + 1] * f.x + x1[2 * j] * f.y;
                    x0[2 * j] = r0, x1[2 * j] = r1;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 e = a[j];
                    const float r = x0[j] * e.x - x1[j] * e.y;
                    x1[j] = x1[j] * e.x + x0[j] * e.y;
                    x0[j] = r;
                }
            }
        }
        if (rot && (is_q || !kFp8)) v0 = pack8<T>(x0), v1 = pack8<T>(x1);
        if (is_q) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + t * p.q_out_stride + h * D);
            dst[c0] = v0, dst[c1] = v1;
        } else {
            const int64_t row = slot * hkv + h;
            void* cache = is_v ? p.v_cache : p.k_cache;
            if (kFp8) {
                const float sc = is_v ? p.v_scale : p.k_scale;
                uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + row * D);
                dst[c0] = quantise8(x0, sc), dst[c1] = quantise8(x1, sc);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(cache) + row * D);
                dst[c0] = v0, dst[c1] = v1;
            }
        }
    }
}

template <typename T, int D, bool kFp8>
cudaError_t launch_rope_t(bool interleaved, const RopeParams& p, cudaStream_t stream) {
    const dim3 grid((unsigned)p.num_tokens), threads(kRopeThreads);
    if (interleaved)
        return launch_with_pdl(rope_and_cache_kernel<T, D, kFp8, true>, grid, threads, 0, stream, p);
    return launch_with_pdl(rope_and_cache_kernel<T, D, kFp8, false>, grid, threads, 0, stream, p);
}

cudaError_t launch_rope_and_cache(int dtype, int head_dim, bool fp8, bool interleaved,
                                  const RopeParams& p, cudaStream_t stream) {
    const bool bf16 = dtype == PA_BF16;
    if (fp8) return bf16 ? launch_rope_t<__nv_bfloat16, 128, true>(interleaved, p, stream)
                         : launch_rope_t<__half, 128, true>(interleaved, p, stream);
    if (head_dim == 64) return bf16 ? launch_rope_t<__nv_bfloat16, 64, false>(interleaved, p, stream)
                                    : launch_rope_t<__half, 64, false>(interleaved, p, stream);
    return bf16 ? launch_rope_t<__nv_bfloat16, 128, false>(interleaved, p, stream)
                : launch_rope_t<__half, 128, false>(interleaved, p, stream);
}

}  // namespace pa
