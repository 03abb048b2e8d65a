// Merge of the decode kernel's weights mode: out from the partitions, and the
// attention weight of every cached token.
//
// The decode kernel (weights mode) leaves, per (sequence b, query head h,
// partition s), m_s = max_i x_i, l_s = sum_i 2^(x_i - m_s) and the partition's
// normalised output, with x_i = scale log2(e) q . K_i, and every x_i itself.
// With M = max_s m_s and Z = sum_s l_s 2^(m_s - M):
//   out[b][h]     = sum_s l_s 2^(m_s - M) o_s / Z
//   weights[b][g][i] (+)= sum over the group's heads h of 2^(x_i - M_h) / Z_h,
// where the newest token (i = L - 1) has nothing added up yet and is set.
// The sums l_s are of the unrounded exponentials, so that the weights hold
// fp32 accuracy.
#include "bounded_internal.h"
#include "pa_device.cuh"

namespace pa {

constexpr int kMergeThreads = 256;

// Grid (sequences, KV heads, 1 + partitions): z = 0 merges out, z = 1 + s
// adds up the weights of partition s.
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads)
    weights_merge_kernel(const __grid_constant__ WeightsMergeParams p) {
    __shared__ float top[kMaxGroup], inv[kMaxGroup];
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.x, g = blockIdx.y, G = p.group;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int L = min(max(p.context_lens[b], 0), p.max_context);
    const int parts = min((L + p.partition_tokens - 1) / p.partition_tokens, p.max_parts);
    const size_t qh0 = (size_t)b * p.num_q_heads + (size_t)g * G;
    if (parts == 0) {
        if (blockIdx.z == 0) {
            T* out = static_cast<T*>(p.out) + qh0 * D;
            for (int i = tid; i < G * D; i += kMergeThreads) out[i] = from_float<T>(0.f);
        }
        return;
    }
    if (blockIdx.z > parts) return;
    // M and 1 / Z of each head of the group, one warp per head
    if (warp < G) {
        const float* ml = p.max_logits + (qh0 + warp) * p.max_parts;
        const float* es = p.exp_sums + (qh0 + warp) * p.max_parts;
        float m = -INFINITY;
        for (int s = lane; s < parts; s += 32) m = fmaxf(m, ml[s]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float z = 0.f;
        for (int s = lane; s < parts; s += 32) z += es[s] * ex2(ml[s] - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0) top[warp] = m, inv[warp] = 1.f / z;
    }
    __syncthreads();
    if (blockIdx.z == 0) {
        for (int item = tid; item < G * (D / 4); item += kMergeThreads) {
            const int h = item / (D / 4), d = (item % (D / 4)) * 4;
            const float* ml = p.max_logits + (qh0 + h) * p.max_parts;
            const float* es = p.exp_sums + (qh0 + h) * p.max_parts;
            const float* src = p.tmp_out + (qh0 + h) * p.max_parts * D + d;
            const float m = top[h], iz = inv[h];
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int s = 0; s < parts; ++s) {
                const float w = es[s] * ex2(ml[s] - m) * iz;
                const float4 x = *reinterpret_cast<const float4*>(src + (size_t)s * D);
                acc.x += w * x.x, acc.y += w * x.y, acc.z += w * x.z, acc.w += w * x.w;
            }
            *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (qh0 + h) * D + d) =
                make_uint2(Mma<T>::pack(acc.x, acc.y), Mma<T>::pack(acc.z, acc.w));
        }
        return;
    }
    const int t0 = (blockIdx.z - 1) * p.partition_tokens;
    const int t1 = min(t0 + p.partition_tokens, L);
    const size_t pair = (size_t)b * p.num_kv_heads + g;
    const float* sc = p.scores + pair * p.max_parts * p.partition_tokens * G;
    const float* before = p.weights ? p.weights + pair * p.weights_stride : nullptr;
    float* after = p.weights_out + pair * p.weights_stride;
    for (int i = t0 + tid; i < t1; i += kMergeThreads) {
        const float* x = sc + (size_t)i * G;
        float w = 0.f;
        for (int h = 0; h < G; ++h) w += ex2(x[h] - top[h]) * inv[h];
        if (before && i < L - 1) w += before[i];
        after[i] = w;
    }
}

template <typename T>
cudaError_t launch_weights_merge_t(int head_dim, const WeightsMergeParams& p, dim3 grid,
                                   cudaStream_t stream) {
    const dim3 threads(kMergeThreads);
    if (head_dim == 64)
        return launch_with_pdl(weights_merge_kernel<T, 64>, grid, threads, 0, stream, p);
    return launch_with_pdl(weights_merge_kernel<T, 128>, grid, threads, 0, stream, p);
}

cudaError_t launch_weights_merge(int dtype, int head_dim, const WeightsMergeParams& p,
                                 int num_seqs, cudaStream_t stream) {
    const dim3 grid(num_seqs, p.num_kv_heads, 1 + p.max_parts);
    if (dtype == PA_BF16) return launch_weights_merge_t<__nv_bfloat16>(head_dim, p, grid, stream);
    return launch_weights_merge_t<__half>(head_dim, p, grid, stream);
}

}  // namespace pa
