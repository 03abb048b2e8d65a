// Attention weights that a prefill chunk's queries give to the cached tokens.
//
// Sequence b holds L tokens, the last C of which are new; the counted queries
// are the chunk's last W (window; all C without one), query i at position
// L - C + i seeing the tokens up to itself:
//   weights[b][g][j] (+)= sum over the group's heads h and the counted i with
//                         position >= j of softmax_j(scale q_ih . K_j)
// Two passes over Q K^T: the first leaves each row's maximum and the inverse
// of its sum of exponentials, the second adds up the columns.  Tokens of the
// chunk have nothing added up yet and are set.
//
// One warp per row or column, products in fp32.
#include "bounded_internal.h"
#include "pa_device.cuh"

namespace pa {

constexpr int kPwThreads = 128;

struct PwSeq {
    int L, C, first, counted;      // context, chunk, first counted query, their number
    int64_t q0;                    // row of the chunk's first query in q
};

__device__ __forceinline__ bool pw_sequence(const PrefillWeightsParams& p, int b, bool report,
                                            PwSeq& s) {
    int L = p.context_lens[b];
    const int64_t q0 = p.query_start[b];
    int64_t C = (int64_t)p.query_start[b + 1] - q0;
    bool bad = false;
    if (L < 0 || L > p.max_context) bad = true, L = L < 0 ? 0 : p.max_context;
    if (C < 0 || C > L) bad = true, C = C < 0 ? 0 : L;
    if (q0 < 0 || q0 + C > p.num_tokens) bad = true, C = 0;
    s.L = L, s.C = (int)C, s.q0 = q0;
    s.counted = p.window > 0 ? min(p.window, s.C) : s.C;
    if (s.counted > p.max_counted) bad = true, s.counted = p.max_counted;
    s.first = s.C - s.counted;
    if (bad && report) flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
    return s.L > 0;
}

template <typename T, int D>
__device__ __forceinline__ float pw_score(const PrefillWeightsParams& p, int b, int g, int j,
                                          const float (&q)[D / 32], int lane) {
    const int blk = p.block_tables[(size_t)b * p.max_blocks_per_seq + j / p.block_size];
    float s = 0.f;
    if (blk >= 0 && blk < p.num_blocks) {
        const T* k = static_cast<const T*>(p.k_cache) +
                     (((size_t)blk * p.block_size + j % p.block_size) * p.num_kv_heads + g) * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) s += q[e] * (float)k[lane + 32 * e];
    } else if (lane == 0) {
        flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s * p.scale_log2;
}

template <typename T, int D>
__device__ __forceinline__ void pw_query(const PrefillWeightsParams& p, const PwSeq& s, int i,
                                         int head, float (&q)[D / 32], int lane) {
    const T* src = static_cast<const T*>(p.q) + ((size_t)(s.q0 + i) * p.num_q_heads + head) * D;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) q[e] = (float)src[lane + 32 * e];
}

template <typename T, int D>
__global__ void __launch_bounds__(kPwThreads)
    prefill_stats_kernel(const __grid_constant__ PrefillWeightsParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.z, head = blockIdx.y, lane = threadIdx.x & 31;
    const int r = blockIdx.x * (kPwThreads / 32) + (threadIdx.x >> 5);
    PwSeq s;
    if (!pw_sequence(p, b, threadIdx.x == 0 && blockIdx.x == 0 && head == 0, s) || r >= s.counted) return;
    float q[D / 32];
    pw_query<T, D>(p, s, s.first + r, head, q, lane);
    const int pos = s.L - s.C + s.first + r;
    float m = -INFINITY, z = 0.f;
    for (int j = 0; j <= pos; ++j) {
        const float x = pw_score<T, D>(p, b, head / p.group, j, q, lane);
        const float n = fmaxf(m, x);
        z = z * ex2(m - n) + ex2(x - n);
        m = n;
    }
    if (lane == 0) {
        float* dst = p.stats + (((size_t)b * p.max_counted + r) * p.num_q_heads + head) * 2;
        dst[0] = m, dst[1] = 1.f / z;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kPwThreads)
    prefill_columns_kernel(const __grid_constant__ PrefillWeightsParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.z, g = blockIdx.y, lane = threadIdx.x & 31;
    const int j = blockIdx.x * (kPwThreads / 32) + (threadIdx.x >> 5);
    PwSeq s;
    if (!pw_sequence(p, b, false, s) || j >= s.L) return;
    float w = 0.f;
    for (int r = max(0, j - (s.L - s.C + s.first)); r < s.counted; ++r) {
        for (int h = 0; h < p.group; ++h) {
            const int head = g * p.group + h;
            float q[D / 32];
            pw_query<T, D>(p, s, s.first + r, head, q, lane);
            const float* st = p.stats + (((size_t)b * p.max_counted + r) * p.num_q_heads + head) * 2;
            w += ex2(pw_score<T, D>(p, b, g, j, q, lane) - st[0]) * st[1];
        }
    }
    if (lane == 0) {
        const size_t at = ((size_t)b * p.num_kv_heads + g) * p.weights_stride + j;
        if (p.weights && j < s.L - s.C) w += p.weights[at];
        p.weights_out[at] = w;
    }
}

template <typename T, int D>
cudaError_t launch_prefill_weights_t(const PrefillWeightsParams& p, cudaStream_t stream) {
    constexpr int kRows = kPwThreads / 32;
    if (p.max_counted > 0) {
        const dim3 grid((p.max_counted + kRows - 1) / kRows, p.num_q_heads, p.num_seqs);
        cudaError_t e = launch_with_pdl(prefill_stats_kernel<T, D>, grid, dim3(kPwThreads), 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((p.max_context + kRows - 1) / kRows, p.num_kv_heads, p.num_seqs);
    return launch_with_pdl(prefill_columns_kernel<T, D>, grid, dim3(kPwThreads), 0, stream, p);
}

cudaError_t launch_prefill_weights(int dtype, int head_dim, const PrefillWeightsParams& p,
                                   cudaStream_t stream) {
    if (dtype == PA_BF16)
        return head_dim == 64 ? launch_prefill_weights_t<__nv_bfloat16, 64>(p, stream)
                              : launch_prefill_weights_t<__nv_bfloat16, 128>(p, stream);
    return head_dim == 64 ? launch_prefill_weights_t<__half, 64>(p, stream)
                          : launch_prefill_weights_t<__half, 128>(p, stream);
}

}  // namespace pa
