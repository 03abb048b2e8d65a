// Merge of the decode kernel's weights mode: out from the partitions, and the
// attention weight of every cached token (short contexts: the decode kernel
// does this itself, join_weights in decode_kernel.cuh).
//
// The decode kernel (weights mode) leaves, per (sequence b, query head h,
// partition s), m_s = max_i x_i, l_s = sum_i 2^(x_i - m_s) and the partition's
// normalised output, with x_i = scale log2(e) q . K_i, and every x_i itself.
// With M = max_s m_s and Z = sum_s l_s 2^(m_s - M):
//   out[b][h]     = sum_s l_s 2^(m_s - M) o_s / Z
//   weights[b][g][i] (+)= sum over the group's heads h of 2^(x_i - M_h) / Z_h,
// where the newest token (i = L - 1) has nothing added up yet and is set.
// The sums l_s are of the unrounded exponentials, so that the weights hold
// fp32 accuracy.  Bound by the scores, read back from L2, and by the start of
// a launch of few microseconds: 7 to 11 us of 57 (64 ragged sequences), 71 (E4M3)
// and 229 (8 long ones).
#include <algorithm>

#include "bounded_internal.h"
#include "pa_device.cuh"

namespace pa {

constexpr int kMergeThreads = 256;
// Tokens of a thread, their scores in flight together, and CTAs per SM that
// the registers are held to.  Many scores a token: one, in eight CTAs (E4M3,
// 256 pairs of 4096 tokens, decode and merge 68.8 us; two in five 70.7, four
// in four 70.2).  Four: four in six (512 pairs of up to 2048 56.6, four in
// four 57.3, two in eight 60.8).
__host__ __device__ constexpr int merge_tokens(int group) { return group == 8 ? 1 : 4; }
__host__ __device__ constexpr int merge_ctas(int group) { return group == 8 ? 8 : group == 4 ? 6 : 4; }

// The group's scores of one token; kG = 0: any group, read one by one.
template <int kG>
struct TokenScores {
    float x[kG == 0 ? kMaxGroup : kG];
    __device__ __forceinline__ void load(const float* src, int group) {
        if constexpr (kG == 8 || kG == 4) {
#pragma unroll
            for (int i = 0; i < kG / 4; ++i) {
                const float4 v = __ldcs(reinterpret_cast<const float4*>(src) + i);
                x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
            }
        } else if constexpr (kG == 2) {
            const float2 v = __ldcs(reinterpret_cast<const float2*>(src));
            x[0] = v.x, x[1] = v.y;
        } else {
#pragma unroll
            for (int h = 0; h < (kG == 0 ? kMaxGroup : kG); ++h) x[h] = kG != 0 || h < group ? src[h] : 0.f;
        }
    }
};

// Grid (sequences, KV heads, 1 + chunks of tokens): z = 0 merges out,
// z = 1 + c adds up the weights of chunk c.  A chunk's scores and earlier
// weights are requested before the row sums that they wait for are formed.
template <typename T, int D, int kG>
__global__ void __launch_bounds__(kMergeThreads, merge_ctas(kG))
    weights_merge_kernel(const __grid_constant__ WeightsMergeParams p) {
    __shared__ float top[kMaxGroup], inv[kMaxGroup];
    __shared__ float4 part_out[kMergeThreads];
    grid_dependency_wait();
    allow_dependent_launch();
    const int b = blockIdx.x, g = blockIdx.y, G = kG == 0 ? p.group : kG;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int L = min(max(p.context_lens[b], 0), p.max_context);
    const int parts = min((L + p.partition_tokens - 1) / p.partition_tokens, p.max_parts);
    const int end = min(L, parts * p.partition_tokens);          // tokens attended to
    const size_t qh0 = (size_t)b * p.num_q_heads + (size_t)g * G;
    constexpr int kMergeTokens = merge_tokens(kG), kMergeChunk = kMergeThreads * kMergeTokens;
    const int t0 = ((int)blockIdx.z - 1) * kMergeChunk + tid;
    if (parts == 0) {
        if (blockIdx.z == 0) {
            T* out = static_cast<T*>(p.out) + qh0 * D;
            for (int i = tid; i < G * D; i += kMergeThreads) out[i] = from_float<T>(0.f);
        }
        return;
    }
    if (blockIdx.z > 0 && t0 - tid >= end) return;
    const size_t pair = (size_t)b * p.num_kv_heads + g;
    TokenScores<kG> sc[kMergeTokens];
    float before[kMergeTokens];
    if (blockIdx.z > 0) {
        const float* src = p.scores + pair * p.max_parts * p.partition_tokens * G;
#pragma unroll
        for (int k = 0; k < kMergeTokens; ++k) {
            const int i = t0 + k * kMergeThreads;
            before[k] = 0.f;
            if (i < end) {
                sc[k].load(src + (size_t)i * G, G);
                if (p.weights && i < L - 1) before[k] = p.weights[pair * p.weights_stride + i];
            }
        }
    }
    // M and 1 / Z of each head of the group, one warp per head
    if (warp < G) {
        const float* ml = p.max_logits + (qh0 + warp) * p.max_parts;
        const float* es = p.exp_sums + (qh0 + warp) * p.max_parts;
        float m = -INFINITY, z = 0.f;
        for (int s = lane; s < parts; s += 32) {
            const float n = fmaxf(m, ml[s]);
            z = z * ex2(m - n) + es[s] * ex2(ml[s] - n);
            m = n;
        }
        float M = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        z = m == -INFINITY ? 0.f : z * ex2(m - M);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0) top[warp] = M, inv[warp] = 1.f / z;
    }
    __syncthreads();
    if (blockIdx.z == 0) {
        // four output dims of a head to a thread; the threads beyond one set
        // take their share of the partitions
        const int items = G * (D / 4), sets = kMergeThreads / items;
        const int item = tid % items, set = tid / items;
        const int h = item / (D / 4), d = (item % (D / 4)) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (set < sets) {
            const float* ml = p.max_logits + (qh0 + h) * p.max_parts;
            const float* es = p.exp_sums + (qh0 + h) * p.max_parts;
            const float* src = p.tmp_out + (qh0 + h) * p.max_parts * D + d;
            const float m = top[h];
#pragma unroll 4
            for (int s = set; s < parts; s += sets) {
                const float w = es[s] * ex2(ml[s] - m);
                const float4 x = *reinterpret_cast<const float4*>(src + (size_t)s * D);
                acc.x += w * x.x, acc.y += w * x.y, acc.z += w * x.z, acc.w += w * x.w;
            }
        }
        part_out[tid] = acc;
        __syncthreads();
        if (set == 0) {
            for (int k = 1; k < sets; ++k) {
                const float4 x = part_out[tid + k * items];
                acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
            }
            const float iz = inv[h];
            *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (qh0 + h) * D + d) =
                make_uint2(Mma<T>::pack(acc.x * iz, acc.y * iz), Mma<T>::pack(acc.z * iz, acc.w * iz));
        }
        return;
    }
    float* after = p.weights_out + pair * p.weights_stride;
#pragma unroll
    for (int k = 0; k < kMergeTokens; ++k) {
        const int i = t0 + k * kMergeThreads;
        if (i >= end) break;
        float w = 0.f;
#pragma unroll
        for (int h = 0; h < (kG == 0 ? kMaxGroup : kG); ++h)
            if (kG != 0 || h < G) w += ex2(sc[k].x[h] - top[h]) * inv[h];
        after[i] = before[k] + w;
    }
}

template <typename T, int D>
cudaError_t launch_weights_merge_g(const WeightsMergeParams& p, dim3 grid, cudaStream_t stream) {
    const dim3 threads(kMergeThreads);
    switch (p.group) {
        case 1: return launch_with_pdl(weights_merge_kernel<T, D, 1>, grid, threads, 0, stream, p);
        case 2: return launch_with_pdl(weights_merge_kernel<T, D, 2>, grid, threads, 0, stream, p);
        case 4: return launch_with_pdl(weights_merge_kernel<T, D, 4>, grid, threads, 0, stream, p);
        case 8: return launch_with_pdl(weights_merge_kernel<T, D, 8>, grid, threads, 0, stream, p);
        default: return launch_with_pdl(weights_merge_kernel<T, D, 0>, grid, threads, 0, stream, p);
    }
}

cudaError_t launch_weights_merge(int dtype, int head_dim, const WeightsMergeParams& p,
                                 int num_seqs, cudaStream_t stream) {
    const int longest = (int)std::min<int64_t>((int64_t)p.max_parts * p.partition_tokens, p.max_context);
    const int chunk = kMergeThreads * merge_tokens(p.group);
    const dim3 grid(num_seqs, p.num_kv_heads, 1 + (longest + chunk - 1) / chunk);
    if (dtype == PA_BF16)
        return head_dim == 64 ? launch_weights_merge_g<__nv_bfloat16, 64>(p, grid, stream)
                              : launch_weights_merge_g<__nv_bfloat16, 128>(p, grid, stream);
    return head_dim == 64 ? launch_weights_merge_g<__half, 64>(p, grid, stream)
                          : launch_weights_merge_g<__half, 128>(p, grid, stream);
}

}  // namespace pa
