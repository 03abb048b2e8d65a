/*
 * pa.h -- C ABI of the paged decode attention library (libpa.so).
 *
 * The operation (from the pages on vLLM / PagedAttention):
 *   - The KV cache is split into fixed-size blocks (16 tokens by default) that
 *     may sit anywhere in a preallocated physical pool; a per-request block
 *     table maps logical block j to its physical block (techfeed summary of
 *     ngrok's "Serving models at scale with vLLM", section on PagedAttention;
 *     youngju.dev "vLLM inference optimization", section "PagedAttention").
 *   - A new token's K and V go to slot (last block, count % block_size)
 *     (youngju.dev post, PagedAttentionManager.append_token).
 *   - Decode attention follows the table, gathering K and V while it computes
 *     (ta-paperlens "LLM serving from scratch", section on fragmentation and
 *     PagedAttention).
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 * Layouts are row-major and contiguous; every pointer marked (device) is
 * CUDA device memory (or managed memory) of the current device:
 *   q, out          [num_seqs][num_q_heads][head_dim]                 T
 *   k, v (new)      [num_tokens][num_kv_heads][head_dim]              T
 *   k_cache,v_cache [num_blocks][block_size][num_kv_heads][head_dim]  T
 *   block_tables    [num_seqs][max_blocks_per_seq]                    int32
 *   context_lens    [num_seqs]                                        int32
 *   slot_mapping    [num_tokens]                                      int64
 * where T is fp16 or bf16 (pa_shape.dtype).  Query head h reads KV head
 * h / (num_q_heads / num_kv_heads).  context_lens[b] counts every token of
 * sequence b including the one just written; token i lives at offset
 * i % block_size of physical block block_tables[b][i / block_size].
 * Attention is softmax(scale * q . K^T) . V with fp32 accumulation; outputs
 * are rounded to nearest-even into T.  An empty context gives zeros.
 *
 * Ownership: the caller owns every buffer, including split workspaces.  The
 * library allocates nothing, frees nothing and never synchronises: work is
 * enqueued on `stream` (a cudaStream_t passed as void*; NULL = the legacy
 * default stream) and the call returns once it is enqueued.
 *
 * Errors: arguments are validated on the host before anything is enqueued;
 * a failed check returns a non-zero pa_status and launches nothing.  A
 * failed launch returns PA_ERR_CUDA (pa_last_cuda_error gives the code).
 * Device-side values are bounded rather than trusted: a context length is
 * clamped to [0, max_blocks_per_seq * block_size]; a physical block id
 * outside [0, num_blocks) reads as zeros (never out of the pool); a slot
 * outside the pool is skipped.  Those events, and any wait in a kernel that
 * ran past its time limit, set bits of a device error word read with
 * pa_read_device_errors.
 *
 * Supported shapes: head_dim 64 or 128; block_size 16 or 32; 1 <= num_q_heads /
 * num_kv_heads <= 8; every device pointer 16-byte aligned.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, inconsistent shape */
    PA_ERR_UNSUPPORTED = 2,   /* valid but not built: head_dim, block_size, group */
    PA_ERR_WORKSPACE = 3,     /* split workspace too small for the request */
    PA_ERR_CUDA = 4           /* a CUDA call failed; see pa_last_cuda_error */
} pa_status;

typedef enum { PA_FP16 = 0, PA_BF16 = 1 } pa_dtype;

/* Device error word bits (pa_read_device_errors). */
#define PA_DEVERR_WAIT_TIMEOUT   0x1  /* a pipeline wait gave up after ~1 s */
#define PA_DEVERR_BAD_CONTEXT    0x2  /* a context length was clamped */
#define PA_DEVERR_BAD_SLOT       0x4  /* a slot past the pool was skipped */
#define PA_DEVERR_BAD_INDEX      0x8  /* an axis, a parent or a path entry was set aside */

typedef struct {
    int32_t num_seqs;
    int32_t num_q_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t block_size;
    int32_t max_blocks_per_seq;
    int64_t num_blocks;
    int32_t dtype;            /* pa_dtype */
    int32_t reserved;         /* must be 0 */
} pa_shape;

/*
 * reshape_and_cache: write each new token's K and V into its cache slot.
 * For t < num_tokens with s = slot_mapping[t] (device):
 *   s < 0                       -> padding, nothing written;
 *   0 <= s < num_blocks*block_size
 *       -> k_cache[s / block_size][s % block_size][:][:] = k[t][:][:],
 *          v_cache likewise (bit copy);
 *   otherwise                   -> skipped, PA_DEVERR_BAD_SLOT set.
 * (youngju.dev post, PagedAttentionManager.append_token.)
 * k, v, slot_mapping, k_cache, v_cache: device.  Uses shp->num_kv_heads,
 * head_dim, block_size, num_blocks and dtype; num_seqs may differ from
 * num_tokens and is ignored.  num_tokens == 0 enqueues nothing.
 */
int pa_reshape_and_cache(const void* k, const void* v, const int64_t* slot_mapping,
                         void* k_cache, void* v_cache, int64_t num_tokens,
                         const pa_shape* shp, void* stream);

/*
 * pa_decode: single-pass paged decode attention, one query token per sequence
 * (ta-paperlens page, PagedAttention paragraph): for every b, h
 *   out[b][h][:] = sum_i softmax_i(scale * q[b][h] . K_i) V_i,  i < context_lens[b].
 * One CTA walks the whole context of a (sequence, KV head) and serves the
 * group of query heads that share the KV head.
 * q, k_cache, v_cache, block_tables, context_lens, out: device.
 */
int pa_decode(const void* q, const void* k_cache, const void* v_cache,
              const int32_t* block_tables, const int32_t* context_lens, float scale,
              void* out, const pa_shape* shp, void* stream);

/*
 * Bytes of one contiguous split workspace for pa_decode_split / pa_reduce:
 * [tmp_out][max_logits][exp_sums], each part rounded up to 256 bytes, with
 * max_num_partitions = ceil(max_context_len / partition_size).
 * Returns 0 for invalid arguments.
 */
size_t pa_split_workspace_size(const pa_shape* shp, int32_t max_context_len,
                               int32_t partition_size);

/*
 * pa_decode_split: the context of each sequence is cut into partitions of
 * partition_size tokens (a multiple of block_size); partition s covers
 * tokens [s*P, min((s+1)*P, L_b)).  For each (b, h, s) with s*P < L_b and
 * s < max_num_partitions it writes, in fp32:
 *   max_logits[b][h][s]   = m_s = max_i scale * q . K_i
 *   exp_sums[b][h][s]     = l_s = sum_i exp(scale * q . K_i - m_s)
 *   tmp_out[b][h][s][:]   = sum_i exp(scale * q . K_i - m_s) V_i / l_s
 * Partitions at or past the context end are not written.  Tokens at or past
 * max_num_partitions * partition_size are not attended: the caller sizes
 * max_num_partitions >= ceil(max_b L_b / partition_size).
 * tmp_out [B][Hq][max_num_partitions][D], max_logits and exp_sums
 * [B][Hq][max_num_partitions]: device, fp32, 16-byte aligned.
 * (Context split and log-sum-exp merge are not in the pages; they follow
 * the split-context decoding used for long contexts.)
 */
int pa_decode_split(const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, const int32_t* context_lens, float scale,
                    int32_t partition_size, int32_t max_num_partitions,
                    float* tmp_out, float* max_logits, float* exp_sums,
                    const pa_shape* shp, void* stream);

/*
 * pa_reduce: log-sum-exp merge of pa_decode_split's partitions.  For each
 * (b, h) with S_b = min(ceil(L_b / P), max_num_partitions):
 *   M = max_s m_s,  w_s = l_s * exp(m_s - M),
 *   out[b][h][:] = sum_s w_s tmp_out[b][h][s][:] / sum_s w_s   (zeros if S_b = 0).
 * tmp_out, max_logits, exp_sums, context_lens, out: device.
 */
int pa_reduce(const float* tmp_out, const float* max_logits, const float* exp_sums,
              const int32_t* context_lens, int32_t partition_size,
              int32_t max_num_partitions, void* out, const pa_shape* shp, void* stream);

/*
 * pa_decode_step_balanced: the fused layer-step of pa_decode_step (same
 * inputs, same results) with the work balanced over one wave of CTAs instead
 * of one CTA per context partition: the 16-token tiles of all (sequence,
 * KV head) pairs, in order, are dealt out in equal contiguous ranges to the
 * consumer warps of the grid, each CTA's TMA producer warp serving its two
 * consumers; a warp's range may cover the end of one sequence and the start
 * of the next, and pieces of one (sequence, KV head) are merged
 * (log-sum-exp) by the warp that finishes last.  Suited to batches of many
 * short or ragged contexts.
 * workspace: device memory of at least pa_balanced_workspace_size(shp)
 * bytes, 16-byte aligned, all zero before the first call (it holds
 * per-(sequence, KV head) counters that every call leaves at zero; zero it
 * again after a PA_DEVERR_WAIT_TIMEOUT).  Calls that overlap on the GPU must
 * not share a workspace.  Other arguments and errors as pa_decode_step.
 * One launch.
 */
size_t pa_balanced_workspace_size(const pa_shape* shp);
int pa_decode_step_balanced(const void* q, const void* k, const void* v,
                            const int64_t* slot_mapping, void* k_cache, void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens, float scale,
                            void* workspace, size_t workspace_bytes, void* out,
                            const pa_shape* shp, void* stream);

/*
 * FP8 KV cache.  The pages name the KV-cache data type as a knob that, like
 * weight quantisation, shrinks the KV pool so that more requests fit
 * (ta-paperlens page, --quantization / --kv-cache-dtype; youngju.dev post,
 * quantisation section).  Here the cache holds OCP E4M3 codes (1 byte per
 * element, [num_blocks][block_size][num_kv_heads][head_dim] bytes) with one
 * scale per tensor: element = e4m3(code) * k_scale (K) or * v_scale (V).
 * q, k, v (new tokens) and out keep the 16-bit type of shp->dtype.
 * head_dim must be 128 (else PA_ERR_UNSUPPORTED); scales must be finite and
 * > 0 (else PA_ERR_INVALID_ARG).  Otherwise these mirror the 16-bit entry
 * points, argument for argument, with the scales added.
 *
 * pa_reshape_and_cache_fp8: code = E4M3 of x / k_scale (x / v_scale), the
 * quotient in fp32, rounded to nearest even, saturating at +-448.
 */
int pa_reshape_and_cache_fp8(const void* k, const void* v, const int64_t* slot_mapping,
                             void* k_cache, void* v_cache, int64_t num_tokens, float k_scale,
                             float v_scale, const pa_shape* shp, void* stream);

/* pa_decode over an E4M3 cache. */
int pa_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, const int32_t* context_lens, float scale,
                  float k_scale, float v_scale, void* out, const pa_shape* shp, void* stream);

/* pa_decode_split over an E4M3 cache (merge the partitions with pa_reduce). */
int pa_decode_split_fp8(const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_tables, const int32_t* context_lens, float scale,
                        float k_scale, float v_scale, int32_t partition_size,
                        int32_t max_num_partitions, float* tmp_out, float* max_logits,
                        float* exp_sums, const pa_shape* shp, void* stream);

/* pa_decode_step over an E4M3 cache (the same memory rules, pinned host
 * inputs and output included): the new token is quantised as in
 * pa_reshape_and_cache_fp8 and attention reads the quantised values. */
int pa_decode_step_fp8(const void* q, const void* k, const void* v, const int64_t* slot_mapping,
                       void* k_cache, void* v_cache, const int32_t* block_tables,
                       const int32_t* context_lens, float scale, float k_scale, float v_scale,
                       int32_t partition_size, int32_t max_num_partitions, float* tmp_out,
                       float* max_logits, float* exp_sums, int32_t* counters, void* out,
                       const pa_shape* shp, void* stream);

/* pa_decode_step_balanced over an E4M3 cache. */
int pa_decode_step_balanced_fp8(const void* q, const void* k, const void* v,
                                const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                const int32_t* block_tables, const int32_t* context_lens,
                                float scale, float k_scale, float v_scale, void* workspace,
                                size_t workspace_bytes, void* out, const pa_shape* shp,
                                void* stream);

/*
 * pa_prefill: paged prefill / chunked-prefill attention.  Sequence b holds
 * L_b = context_lens[b] tokens in the cache, the last C_b = query_start[b+1]
 * - query_start[b] of which are new in this step (written beforehand with
 * pa_reshape_and_cache).  New token i of b sits at position p = L_b - C_b + i
 * and attends causally:
 *   out[query_start[b] + i][h][:] = sum_{j <= p} softmax_j(scale q.K_j) V_j
 * (ta-paperlens page, prefill vs decode and chunked prefill; techfeed
 * summary, chunked prefill of long prompts).  A one-token chunk is a decode.
 * q, out: [total_tokens][num_q_heads][head_dim] with total_tokens =
 * query_start[num_seqs]; query_start int32 [num_seqs + 1], non-decreasing,
 * from 0; max_query_len >= every C_b (it sizes the grid: query tokens past
 * 16 * ceil(max_query_len / 16) are not computed).  C_b > L_b is clamped to
 * L_b and flagged (PA_DEVERR_BAD_CONTEXT).  All pointers device.
 */
int pa_prefill(const void* q, const void* k_cache, const void* v_cache,
               const int32_t* block_tables, const int32_t* context_lens,
               const int32_t* query_start, float scale, int32_t max_query_len, void* out,
               const pa_shape* shp, void* stream);

/*
 * pa_prefill_ws: pa_prefill with a workspace in which a one-CTA plan kernel
 * orders the tcgen05 kernel's (sequence, chunk) work items by the number of
 * key tiles they read, longest first, so that the longest start first and
 * the SMs finish together (the kernel's persistent CTAs, one per SM, deal
 * that order out in a snake; pa_prefill, without one, takes each sequence's
 * chunks last-first: later chunks read more keys).  The pages describe
 * prefill cost growing with the square of the prompt length (ta-paperlens
 * page, the quadratic cost of prefill); the ordering itself is this
 * library's.  workspace: device memory of at least
 * pa_prefill_workspace_size(shp, max_query_len) bytes, 16-byte aligned, no
 * initial contents, owned by the caller; calls that overlap on the GPU must
 * not share it.  A size of 0 (the mma.sync kernel is taken) accepts a null
 * workspace, which otherwise also falls back to pa_prefill's order.  Too
 * small or misaligned: PA_ERR_INVALID_ARG.  Two launches when the tcgen05
 * kernel is taken with a workspace, else one.  Results are bitwise the same
 * as pa_prefill's.
 */
size_t pa_prefill_workspace_size(const pa_shape* shp, int32_t max_query_len);
int pa_prefill_ws(const void* q, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, const int32_t* context_lens,
                  const int32_t* query_start, float scale, int32_t max_query_len,
                  void* workspace, size_t workspace_bytes, void* out, const pa_shape* shp,
                  void* stream);

/*
 * pa_prefill_mma: the same operation, arguments and errors as pa_prefill,
 * always on the mma.sync kernel (16 query tokens per CTA, any group size and
 * head_dim 64 or 128).  pa_prefill takes the tcgen05 kernel (128 query rows
 * per CTA, accumulators in tensor memory) when head_dim is 128, the group
 * size G = Hq / Hkv is 1, 2, 4 or 8, scale > 0 and max_query_len >= 128 / G
 * (a chunk can fill its 128 rows), and this one otherwise.
 */
int pa_prefill_mma(const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, const int32_t* context_lens,
                   const int32_t* query_start, float scale, int32_t max_query_len, void* out,
                   const pa_shape* shp, void* stream);

/*
 * pa_copy_async: copy nbytes from src to dst with a short kernel on the
 * stream (SM loads and stores, not a copy-engine transfer).  For a
 * layer-step's small transfers: dst and src may each be device memory or
 * pinned host memory (reached through unified addressing), both 16-byte
 * aligned, nbytes a multiple of 16; the buffers must not overlap.  The launch
 * takes part in programmatic dependent launch like the step kernels, so an
 * upload, a step and a read-back chain without gaps.  No counterpart in the
 * pages: it is the transport of the step's inputs and output.
 */
int pa_copy_async(void* dst, const void* src, size_t nbytes, void* stream);

/*
 * pa_copy_blocks: copy whole physical blocks between two block pools.  For
 * each pair p < num_pairs of block_mapping (int64 [num_pairs][2], device):
 *   src = block_mapping[2p], dst = block_mapping[2p+1],
 *   k_dst[dst][:][:][:] = k_src[src][:][:][:], v_dst likewise (bit copy).
 * Copy-on-write: before a request writes into a block it shares with others
 * (parallel sampling, beam search, a shared prompt), it gets a private copy
 * (tcdigital article, memory sharing for parallel sampling; youngju.dev post,
 * Copy-on-Write prefix sharing) -- src and dst pools are the same pool.
 * Swap: a preempted request's blocks move to CPU memory and back (tcdigital
 * article, --swap-space; ta-paperlens scheduler, preemption) -- one pool is
 * pinned host memory reachable from the device (cudaHostAlloc / registered
 * memory under unified addressing), passed by its device-visible address.
 * Both pools are laid out [num_blocks][block_size][num_kv_heads][head_dim]
 * with shp's block_size, num_kv_heads, head_dim and dtype (shp->num_blocks is
 * not used); src_num_blocks / dst_num_blocks bound the ids.  A pair with an
 * id out of range is skipped and sets PA_DEVERR_BAD_SLOT.  Pairs must not
 * write the same destination block twice, nor read a block another pair
 * writes.  num_pairs <= 65535; num_pairs == 0 enqueues nothing.
 */
int pa_copy_blocks(const void* k_src, const void* v_src, int64_t src_num_blocks, void* k_dst,
                   void* v_dst, int64_t dst_num_blocks, const int64_t* block_mapping,
                   int64_t num_pairs, const pa_shape* shp, void* stream);

/*
 * Size of the device buffer behind pa_decode_static_workspace: 32 MiB,
 * held on every GPU that loads the library until the process exits.
 */
#define PA_STATIC_WORKSPACE_BYTES (32u << 20)

/*
 * pa_decode_static_workspace: pa_decode_split followed by pa_reduce, with the
 * partition workspace (tmp_out, max_logits, exp_sums) taken from a fixed
 * device buffer inside the library instead of from the caller.  It allocates
 * nothing.  The pages have no counterpart: this entry point exists for
 * callers that cannot allocate device memory -- code running inside a host
 * framework that owns the device memory pool (a private cudaMalloc would
 * bypass the pool and may fail once the pool holds the free memory), or a
 * latency-critical loop that cannot take the device-wide synchronisation of
 * cudaMalloc / cudaFree.  The caller passes its inputs and `out` exactly as
 * for pa_decode_split + pa_reduce (same layouts, same device pointers,
 * partition_size a multiple of block_size, max_num_partitions >=
 * ceil(max_b L_b / partition_size)); out [B][Hq][D] receives the merged
 * attention output.
 *
 * Limit: the workspace, laid out [tmp_out][max_logits][exp_sums] with each
 * part rounded up to 256 bytes (4*B*Hq*S*D, then 4*B*Hq*S twice), must fit in
 * PA_STATIC_WORKSPACE_BYTES; larger requests return PA_ERR_WORKSPACE and
 * enqueue nothing.
 *
 * Set-up: the first call on a device (with that device current) looks up the
 * buffer's device address; make that first call before any stream capture.
 * The address belongs to the CUDA context it was looked up in: a call under
 * another context (a driver-API context made current by the caller, or the
 * primary context created anew after cudaDeviceReset) looks it up again, so
 * the first call under each new context must also come before any capture.
 *
 * Sharing: every call on a device uses the same buffer, which keeps the last
 * call's contents (nothing in it needs to start at zero).  Calls whose work
 * overlaps on the GPU -- e.g. issued on two streams without ordering between
 * them -- race on the buffer and corrupt each other's results; order them.
 * Errors: the argument checks of pa_decode_split and pa_reduce run first and
 * give the same statuses; then PA_ERR_WORKSPACE for the limit above.
 */
int pa_decode_static_workspace(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_tables, const int32_t* context_lens,
                               float scale, int32_t partition_size,
                               int32_t max_num_partitions, void* out, const pa_shape* shp,
                               void* stream);

/*
 * pa_decode_step: one decode layer-step in a single launch -- the cache write
 * of each sequence's new token followed by split decode attention and the
 * log-sum-exp merge.  Same results as
 *   pa_reshape_and_cache(k, v, slot_mapping, k_cache, v_cache, num_seqs, ...);
 *   pa_decode_split(...); pa_reduce(...);
 * for the decode step the pages describe (youngju.dev post,
 * PagedAttentionManager.append_token, then the table-walking attention of
 * the ta-paperlens page): token b of k, v ([num_seqs][Hkv][D]) is sequence
 * b's newest token, position L_b - 1, and slot_mapping[b] must be that
 * position's slot, block_tables[b][(L_b-1)/bs]*bs + (L_b-1)%bs, or negative
 * (no new token for b: nothing written).  Any other slot is not written and
 * sets PA_DEVERR_BAD_SLOT.  The CTA of each sequence's last partition writes
 * the new token into the cache and uses it directly; the last CTA of each
 * (sequence, KV head) to finish merges its partitions, so no second launch
 * is needed.
 *
 * Workspace: tmp_out, max_logits, exp_sums as for pa_decode_split, plus
 * counters, int32 [num_seqs][num_kv_heads], which must be zero on entry and
 * are zero again when the step has run (set them to zero once after
 * allocation; after a PA_DEVERR_WAIT_TIMEOUT, zero them again).  The merge
 * reads the partition records four at a time from global memory, so any
 * partition count pa_decode_split accepts works.  out [B][Hq][D] receives
 * the attention output.  k_cache, v_cache and the workspace are device memory;
 * q, k, v, slot_mapping, block_tables, context_lens and out may be device
 * memory or pinned host memory that the device reaches through unified
 * addressing (each CTA reads its inputs and writes its output directly, so
 * a step needs no separate upload or read-back; on a Grace-Blackwell node
 * this moves them over the coherent host link).  k, v, out, tmp_out,
 * max_logits, exp_sums 16-byte aligned; errors as pa_decode_split.
 */
int pa_decode_step(const void* q, const void* k, const void* v, const int64_t* slot_mapping,
                   void* k_cache, void* v_cache, const int32_t* block_tables,
                   const int32_t* context_lens, float scale, int32_t partition_size,
                   int32_t max_num_partitions, float* tmp_out, float* max_logits,
                   float* exp_sums, int32_t* counters, void* out, const pa_shape* shp,
                   void* stream);

/*
 * ---------------------------------------------------------------------------
 * A cache within a budget of tokens
 * ---------------------------------------------------------------------------
 * Long contexts outgrow the pool, and the pages' only answers are preemption
 * and swapping (tcdigital article, --swap-space; ta-paperlens scheduler).
 * The entry points below let a sequence stay on the device with fewer
 * tokens: keys are turned to their positions before they are cached
 * (pa_rope_and_cache), so that a token's place in the cache is free to
 * change; decode and prefill account for the attention weight each cached
 * token receives (pa_decode_weights, pa_prefill_weights); and pa_evict keeps
 * the first, the newest and the most attended tokens and closes the gaps.
 *
 * State of a batch, device memory owned by the caller, per (sequence, KV
 * head) one row of `stride` elements (stride >= max_blocks_per_seq *
 * block_size; entry i belongs to the token at cache index i):
 *   weights    [num_seqs][num_kv_heads][stride]  fp32   weight added up so far
 *   positions  [num_seqs][num_kv_heads][stride]  int32  the token's position
 * Each call takes the state to read and the state to write; the two may be
 * the same arrays, and must not overlap otherwise.  Entries at or past the
 * context length are neither read nor written.
 */

/*
 * pa_rope_and_cache: rotary positions, and the cache write of
 * pa_reshape_and_cache, in one launch.  For t < num_tokens, head h and pair
 * i < rotary_dim / 2 of its first rotary_dim dims, with the angle
 * a = positions[t] * inv_freq[i]:
 *   x' = factor * (x cos a - y sin a),   y' = factor * (y cos a + x sin a),
 * (x, y) being dims (i, i + rotary_dim / 2), or (2i, 2i + 1) with
 * interleaved = 1; dims past rotary_dim are copied.  Turned q rows go to
 * q_out, turned k rows and v rows to cache slot slot_mapping[t], which is
 * treated as in pa_reshape_and_cache (slots that are not negative must
 * differ).  Scaling of the positions for long contexts is part of inv_freq
 * and factor.  The angle is taken in turns, whole ones dropped in integers, at
 * any int64 position and finite inv_freq: it is off by at most 2^-52 of
 * position * inv_freq, 2^-64 turns per position, and 2^-26 turns; the products
 * are in fp32 and each result is rounded once.
 * q, k, v: row t starts t * stride elements on, [heads][head_dim] inside (so
 * they may be slices of one projection's output); strides are multiples of 8
 * elements, of at least a row.  q may be null (keys only: q_stride, q_out
 * and num_q_heads are not used).  q_out may be q itself with the same stride,
 * and must not overlap the inputs otherwise.  positions, slot_mapping [T]
 * int64, inv_freq [rotary_dim / 2] fp32: device.
 * rotary_dim: a multiple of 16 (else PA_ERR_UNSUPPORTED), 0 to head_dim.
 * shp: num_q_heads, num_kv_heads (any ratio), head_dim, block_size,
 * num_blocks, dtype.
 */
int pa_rope_and_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      const void* v, int64_t v_stride, const int64_t* positions,
                      const int64_t* slot_mapping, const float* inv_freq, int32_t rotary_dim,
                      int32_t interleaved, float factor, void* q_out, int64_t q_out_stride,
                      void* k_cache, void* v_cache, int64_t num_tokens, const pa_shape* shp,
                      void* stream);

/* pa_rope_and_cache into an E4M3 cache: the turned key is quantised from
 * fp32, without a rounding to the 16-bit type before. */
int pa_rope_and_cache_fp8(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int64_t* positions,
                          const int64_t* slot_mapping, const float* inv_freq, int32_t rotary_dim,
                          int32_t interleaved, float factor, void* q_out, int64_t q_out_stride,
                          void* k_cache, void* v_cache, int64_t num_tokens, float k_scale,
                          float v_scale, const pa_shape* shp, void* stream);

/*
 * pa_decode_weights: decode attention (the result of pa_decode_split +
 * pa_reduce) that also adds up what it attends to.  With p[h][i] the softmax
 * weight of token i for query head h, and g the KV head of a group of heads:
 *   weights_out[b][g][i] = weights[b][g][i] + sum over the group of p[h][i]
 * for i < L_b; the newest token, i = L_b - 1, has nothing added up yet and
 * gets the sum alone.  weights may be null (nothing added up yet).
 * Softmax statistics and weights are in fp32; p meets V in two fp16 or three
 * bf16 parts, which hold it to 2^-22 (and to 2^-32 of the row's largest).
 * max_context_len >= every L_b (tokens past its partitions are not attended,
 * and their entries not written), partition_size a multiple of block_size.
 * workspace: device memory of at
 * least pa_decode_weights_workspace_size bytes, 16-byte aligned, no initial
 * contents; calls that overlap on the GPU must not share it.  One or two launches.
 */
size_t pa_decode_weights_workspace_size(const pa_shape* shp, int32_t max_context_len,
                                        int32_t partition_size);
int pa_decode_weights(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, const int32_t* context_lens, float scale,
                      int32_t max_context_len, int32_t partition_size, const float* weights,
                      float* weights_out, int64_t weights_stride, void* workspace,
                      size_t workspace_bytes, void* out, const pa_shape* shp, void* stream);

/* pa_decode_weights over an E4M3 cache. */
int pa_decode_weights_fp8(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens, float scale,
                          float k_scale, float v_scale, int32_t max_context_len,
                          int32_t partition_size, const float* weights, float* weights_out,
                          int64_t weights_stride, void* workspace, size_t workspace_bytes,
                          void* out, const pa_shape* shp, void* stream);

/*
 * pa_prefill_weights: the attention weights that a chunk's queries give to
 * the cached tokens (attention itself is pa_prefill, on the same q,
 * query_start and cache).  Queries are those of pa_prefill: new token i of
 * sequence b sits at cache index L_b - C_b + i and sees the tokens up to its
 * own.  The last min(window, C_b) of them are counted, all with window = 0:
 *   weights_out[b][g][j] = weights[b][g][j]
 *       + sum over the group's heads h and the counted i of p[i][h][j]
 * for j < L_b, with weights taken as zero for the chunk's own tokens
 * (j >= L_b - C_b) and where weights is null.
 * num_tokens: rows of q; max_query_len >= every C_b; max_context_len >= every
 * L_b.  Values outside these bounds are clamped and set
 * PA_DEVERR_BAD_CONTEXT.  scale must be finite and > 0.  16-bit caches.
 * workspace as in pa_decode_weights, of pa_prefill_weights_workspace_size
 * bytes.  One to four launches.
 */
size_t pa_prefill_weights_workspace_size(const pa_shape* shp, int32_t max_query_len,
                                         int32_t max_context_len, int32_t window);
int pa_prefill_weights(const void* q, const void* k_cache, const int32_t* block_tables,
                       const int32_t* context_lens, const int32_t* query_start, float scale,
                       int64_t num_tokens, int32_t max_query_len, int32_t max_context_len,
                       int32_t window, const float* weights, float* weights_out,
                       int64_t weights_stride, void* workspace, size_t workspace_bytes,
                       const pa_shape* shp, void* stream);

/*
 * pa_evict: cut every sequence of more than `trigger` tokens down to
 * `budget`.  Token i of (b, g) has the position
 *   pos = i < known_lens[b] ? positions[b][g][i] : i + seen_lens[b] - L_b,
 * seen_lens[b] being the tokens the sequence has had in all (tokens appended
 * since the last cut are in order; known_lens null: 0).  Of a sequence with
 * L_b > trigger each KV head keeps `budget` tokens: those with pos < sinks or
 * pos >= seen_lens[b] - recent, then those of the largest weight, ties (-0
 * and +0 are equal) to the lowest index, NaN below every number.  Kept tokens
 * at index < budget stay in place; the n-th kept token at index >= budget
 * moves to the n-th gap (K and V rows, weight, position).  Afterwards
 *   new_lens[b]      = budget, or L_b where nothing was cut
 *   weights_out, positions_out hold the entries i < new_lens[b],
 * and the next calls take new_lens as context_lens and known_lens (advanced
 * by the tokens appended in the case of context_lens alone).  Every KV head
 * keeps tokens of its own choice, so the caches' rows of one index belong to
 * different positions in different heads.
 * k_cache and v_cache are changed in place: the blocks of a sequence that is
 * cut must not be shared with another (pa_copy_blocks gives it its own).  A
 * block id outside the pool sets PA_DEVERR_BAD_CONTEXT and its rows are not
 * moved.  budget >= 1, budget >= sinks + recent, trigger >= budget; new_lens
 * must not be one of the input arrays.  workspace as in pa_decode_weights,
 * of pa_evict_workspace_size bytes.  pa_evict_fp8: the same on an E4M3 cache.
 */
size_t pa_evict_workspace_size(const pa_shape* shp, int32_t budget);
int pa_evict(void* k_cache, void* v_cache, const int32_t* block_tables,
             const int32_t* context_lens, const int32_t* seen_lens, const int32_t* known_lens,
             const float* weights, const int32_t* positions, int64_t stride, int32_t budget,
             int32_t trigger, int32_t sinks, int32_t recent, float* weights_out,
             int32_t* positions_out, int32_t* new_lens, void* workspace, size_t workspace_bytes,
             const pa_shape* shp, void* stream);
int pa_evict_fp8(void* k_cache, void* v_cache, const int32_t* block_tables,
                 const int32_t* context_lens, const int32_t* seen_lens, const int32_t* known_lens,
                 const float* weights, const int32_t* positions, int64_t stride, int32_t budget,
                 int32_t trigger, int32_t sinks, int32_t recent, float* weights_out,
                 int32_t* positions_out, int32_t* new_lens, void* workspace,
                 size_t workspace_bytes, const pa_shape* shp, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Speculative decoding: a tree of drafted tokens per sequence
 * ---------------------------------------------------------------------------
 * The pages leave speculative decoding to the engine; what it asks of a paged
 * cache is below.  In a verification step sequence b has C_b nodes, C_b being
 * query_start[b + 1] - query_start[b]: the last C_b of its L_b cached tokens.
 * Node i is row query_start[b] + i of the batch and stands at cache index
 * L_b - C_b + i.  Node 0 is the sequence's newest
 * token, the others are drafted after it: parents[row] < i is the node (of the
 * same sequence) that node i follows, negative: the context itself.  A parent
 * that is not below its node counts as negative and sets PA_DEVERR_BAD_INDEX.
 * Sequences have at most PA_TREE_NODES nodes (and max_query_len, where a call
 * has it); those past the first so many are cut off: their rows are not written
 * and the others' results are what they would be.  That sets
 * PA_DEVERR_BAD_CONTEXT, as do a C_b below 0 or above L_b and rows outside
 * [0, num_tokens).  A step: pa_norm_rope_and_cache (or pa_rope_and_cache) and
 * pa_tree_attention in every layer, then pa_accept_tree and pa_commit_path.
 */
#define PA_TREE_NODES 128

/*
 * pa_norm_rope_and_cache: pa_rope_and_cache with the heads of q and k
 * normalised first and positions on several axes.  For every head x of q or k
 *   y[d] = weight[d] * x[d] / sqrt(mean_d(x[d]^2) + eps)
 * in fp32, not rounded before it is turned (values past 2^60 make squares that
 * leave fp32 and a head of zeros; a head of zeros with eps = 0 is NaN, as the
 * formula has it); q_weight and k_weight [head_dim] of type T, null: ones.  Pair i turns by positions[axes[i]][t] * inv_freq[i]:
 * positions is [num_axes][num_tokens] int64, axes [rotary_dim / 2] int32
 * (null: all 0), 1 <= num_axes <= 8; an axis outside them counts as 0 and sets
 * PA_DEVERR_BAD_INDEX.  eps must be finite and not negative.  Everything else
 * is as in pa_rope_and_cache.
 */
int pa_norm_rope_and_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const void* q_weight,
                           const void* k_weight, float eps, const int64_t* positions,
                           int32_t num_axes, const int32_t* axes, const int64_t* slot_mapping,
                           const float* inv_freq, int32_t rotary_dim, int32_t interleaved,
                           float factor, void* q_out, int64_t q_out_stride, void* k_cache,
                           void* v_cache, int64_t num_tokens, const pa_shape* shp, void* stream);

/* pa_norm_rope_and_cache into an E4M3 cache, quantised from fp32. */
int pa_norm_rope_and_cache_fp8(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const void* q_weight,
                               const void* k_weight, float eps, const int64_t* positions,
                               int32_t num_axes, const int32_t* axes, const int64_t* slot_mapping,
                               const float* inv_freq, int32_t rotary_dim, int32_t interleaved,
                               float factor, void* q_out, int64_t q_out_stride, void* k_cache,
                               void* v_cache, int64_t num_tokens, float k_scale, float v_scale,
                               const pa_shape* shp, void* stream);

/*
 * pa_tree_attention: attention of the trees' nodes over the cache, which
 * holds their K and V already.  Node i of sequence b sees the L_b - C_b tokens
 * before the tree, its ancestors and itself:
 *   out[row][h] = sum_j p_j V_j,  p = softmax_j(scale * q[row][h] . K_j).
 * q, out [num_tokens][num_q_heads][head_dim], not overlapping; rows behind the
 * last sequence are not written.  parents [num_tokens] int32, null: every node
 * follows the one before it (a line of drafted tokens, or the chunks of
 * pa_prefill).  scale times log2(e) (and k_scale) must be a normal positive fp32
 * number.
 * max_query_len >= every C_b, at most PA_TREE_NODES (else PA_ERR_UNSUPPORTED);
 * max_context_len >= every L_b; values outside these bounds are clamped and
 * set PA_DEVERR_BAD_CONTEXT.  Bounds that come to 2^31 key tiles of 64 or more
 * over all sequences and KV heads, four added to each, are PA_ERR_UNSUPPORTED.
 * Softmax statistics and sums are in fp32; p meets V in two parts of the
 * 16-bit type, which hold it to 2^-15 (bf16) or 2^-22 (fp16; and to 2^-31 of
 * the row's largest).  The tensor cores cut sums off toward zero, for up to 128
 * key tiles before a rounding add: at most 2^-13 of sum_j p_j |V_j| (measured
 * 5e-5), at any context length.  out is rounded once.  A token that a node does not
 * see has no part in its row, also where its K or V is not finite; an infinite
 * V that it does see makes these elements of its row infinite or NaN.
 * workspace: device memory of at least pa_tree_attention_workspace_size bytes,
 * 16-byte aligned, no initial contents; calls that overlap on the GPU must
 * not share it.  What is enough for a batch is enough for fewer sequences and
 * shorter contexts of the same heads and max_query_len.  One or two launches.
 */
size_t pa_tree_attention_workspace_size(const pa_shape* shp, int32_t max_query_len,
                                        int32_t max_context_len);
int pa_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, const int32_t* context_lens,
                      const int32_t* query_start, const int32_t* parents, float scale,
                      int64_t num_tokens, int32_t max_query_len, int32_t max_context_len,
                      void* workspace, size_t workspace_bytes, void* out, const pa_shape* shp,
                      void* stream);

/* pa_tree_attention over an E4M3 cache. */
int pa_tree_attention_fp8(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens,
                          const int32_t* query_start, const int32_t* parents, float scale,
                          float k_scale, float v_scale, int64_t num_tokens, int32_t max_query_len,
                          int32_t max_context_len, void* workspace, size_t workspace_bytes,
                          void* out, const pa_shape* shp, void* stream);

/*
 * pa_accept_tree: the longest path of drafted tokens that the model agrees
 * with.  target[row] is the token that the model gives after node `row`,
 * draft[row] the token of the node itself.  Node 0 is accepted; any other with
 * a parent is where its parent is and draft[node] = target[parent].  Of the
 * accepted nodes the deepest, the lowest among equals, ends the path:
 *   path[b][0 .. path_lens[b] - 1]  its ancestors and itself, from node 0 on
 *   path[b][path_lens[b] ..]        -1, up to max_query_len
 *   next[b]                         target of the path's end
 * A sequence without nodes gets length 0 and next -1.  draft, target, parents:
 * [num_tokens]; path [num_seqs][max_query_len], 1 <= max_query_len <=
 * PA_TREE_NODES.  path, path_lens and next must not overlap the inputs or one
 * another.  One launch.
 */
int pa_accept_tree(const int64_t* draft, const int64_t* target, const int32_t* parents,
                   const int32_t* query_start, int32_t num_seqs, int64_t num_tokens,
                   int32_t max_query_len, int32_t* path, int32_t* path_lens, int64_t* next,
                   void* stream);

/*
 * pa_commit_path: keeps of each tree the path's nodes, in the caches of all
 * layers.  With base = L_b - C_b the K and V rows of node path[b][j] move to
 * cache index base + j, and
 *   new_lens[b] = base + path_lens[b].
 * A path is ascending (as pa_accept_tree gives it) within [0, C_b); one that
 * is not, or longer than C_b, sets PA_DEVERR_BAD_INDEX, and its sequence is
 * left as it is (new_lens[b] = L_b).  So is, with PA_DEVERR_BAD_CONTEXT, one
 * whose L_b is not within its table (new_lens[b] is clamped to that) or whose
 * C_b is below 0 or above L_b.  Of a tree with more than PA_TREE_NODES nodes the
 * first so many can be kept.  path [num_seqs][path_stride] int32.
 * k_caches, v_caches: host arrays of num_layers (at most 1024) device pointers,
 * one cache pair per layer, all of the shape shp and of the same block tables;
 * no cache may be listed twice or lie over another.  The blocks that hold a
 * tree must not be shared with another sequence.  A block id outside the pool
 * sets PA_DEVERR_BAD_CONTEXT and its rows are not moved.  new_lens must not
 * overlap an input array.  One launch for every 64 layers.  pa_commit_path_fp8: the
 * same on E4M3 caches.
 */
int pa_commit_path(void* const* k_caches, void* const* v_caches, int32_t num_layers,
                   const int32_t* block_tables, const int32_t* context_lens,
                   const int32_t* query_start, const int32_t* path, int32_t path_stride,
                   const int32_t* path_lens, int32_t* new_lens, const pa_shape* shp, void* stream);
int pa_commit_path_fp8(void* const* k_caches, void* const* v_caches, int32_t num_layers,
                       const int32_t* block_tables, const int32_t* context_lens,
                       const int32_t* query_start, const int32_t* path, int32_t path_stride,
                       const int32_t* path_lens, int32_t* new_lens, const pa_shape* shp,
                       void* stream);

/* Static description of a status code. */
const char* pa_status_string(int status);

/* cudaError_t of the most recent PA_ERR_CUDA on this host thread (0 if none). */
int pa_last_cuda_error(void);

/*
 * Copy the device error word (PA_DEVERR_* bits accumulated by kernels of this
 * library on the current device) to *flags, then clear it.  Synchronises
 * `stream`.  Returns PA_OK or PA_ERR_CUDA.
 */
int pa_read_device_errors(int32_t* flags, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
