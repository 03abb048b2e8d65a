// Attention of a tree of drafted tokens: node i of a sequence's tree sees the
// sequence's context, its own ancestors and itself,
//   out = sum_j p_j V_j,   p = softmax_j(scale q . K_j),   j < base or
//   j - base on node i's line, base being the tokens before the tree.
//
// A warp makes one (node, query head).  Per 32 keys each lane forms one score
// (q in shared memory), the running maximum and sum follow in the warp, and
// the lanes then own D / 32 dims of the output.
#include "tree_device.cuh"

namespace pa {

constexpr int kTreeWarps = 4;

template <typename T, int D, bool kFp8>
__global__ void __launch_bounds__(kTreeWarps * 32)
    tree_codes_kernel(const __grid_constant__ TreeParams p) {
    constexpr int kDims = D / 32;
    __shared__ float q_s[kTreeWarps][D];
    grid_dependency_wait();
    allow_dependent_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, i = blockIdx.y, h = blockIdx.x * kTreeWarps + warp;
    const TreeSeq s = tree_sequence(p, b, blockIdx.x == 0 && i == 0 && threadIdx.x == 0);
    if (i >= s.C || h >= p.num_q_heads) return;
    TreeLine line{};
    for (int n = i; n >= 0; n = tree_parent(p.parents, s.q0, n, p.err)) line.w[n >> 5] |= 1u << (n & 31);
    const int g = h / p.group, base = s.L - s.C;
    const int64_t row = ((int64_t)(s.q0 + i) * p.num_q_heads + h) * D;
    const T* q = static_cast<const T*>(p.q) + row;
    for (int d = lane; d < D; d += 32) q_s[warp][d] = (float)q[d];
    __syncwarp();
    const int32_t* table = p.block_tables + (int64_t)b * p.max_blocks_per_seq;
    auto at = [&](const void* cache, int64_t token, int d) -> float {      // -1: a block outside the pool
        if (token < 0) return 0.f;
        const int64_t e = (token * p.num_kv_heads + g) * D + d;
        if constexpr (kFp8) {
            const uint32_t h2 = e4m3x2_to_f16x2(static_cast<const uint8_t*>(cache)[e]);
            return __half2float(__ushort_as_half((unsigned short)h2));
        } else {
            return (float)static_cast<const T*>(cache)[e];
        }
    };
    float m = -INFINITY, l = 0.f, o[kDims] = {};
    for (int key0 = 0; key0 < s.L; key0 += 32) {
        const int key = key0 + lane;
        int64_t token = -1;
        float x = -INFINITY;
        if (key < s.L && (key < base || line.has(key - base))) {
            const int blk = table[key / p.block_size];
            if (blk >= 0 && blk < p.num_blocks)
                token = (int64_t)blk * p.block_size + key % p.block_size;
            else
                flag_error(p.err, PA_DEVERR_BAD_CONTEXT);
            x = 0.f;
            for (int d = 0; d < D; ++d) x += q_s[warp][d] * at(p.k_cache, token, d);
            x *= p.scale_log2;
        }
        float top = x;
        for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        top = fmaxf(top, m);
        const float ref = top == -INFINITY ? 0.f : top;
        const float f = ex2(m - ref), e = ex2(x - ref);
        m = top;
        float sum = e;
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        l = l * f + sum;
#pragma unroll
        for (int k = 0; k < kDims; ++k) o[k] *= f;
        for (uint32_t seen = __ballot_sync(0xffffffffu, x != -INFINITY); seen != 0u; seen &= seen - 1u) {
            const int who = __ffs((int)seen) - 1;
            const float w = __shfl_sync(0xffffffffu, e, who);
            const int64_t tk = __shfl_sync(0xffffffffu, token, who);
#pragma unroll
            for (int k = 0; k < kDims; ++k) o[k] += w * at(p.v_cache, tk, 32 * k + lane);
        }
    }
    T* out = static_cast<T*>(p.out) + row;
    const float scale = (kFp8 ? p.v_scale : 1.f) / l;
#pragma unroll
    for (int k = 0; k < kDims; ++k) out[32 * k + lane] = from_float<T>(o[k] * scale);
}

template <typename T, int D, bool kFp8>
cudaError_t launch_codes_t(const TreeParams& p, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.num_q_heads + kTreeWarps - 1) / kTreeWarps), (unsigned)p.max_query,
                    (unsigned)p.num_seqs);
    return launch_with_pdl(tree_codes_kernel<T, D, kFp8>, grid, dim3(kTreeWarps * 32), 0, stream, p);
}

cudaError_t launch_tree_codes(int dtype, const TreeParams& p, cudaStream_t stream) {
    return dtype == PA_BF16 ? launch_codes_t<__nv_bfloat16, 128, true>(p, stream)
                            : launch_codes_t<__half, 128, true>(p, stream);
}

}  // namespace pa
