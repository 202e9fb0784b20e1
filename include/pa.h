/*
 * pa.h -- C ABI of the paged varlen attention library (libpa.so), sm_103a.
 *
 * The operations follow the web pages that describe vLLM's attention
 * backends:
 *   [FA-vLLM] "FlashAttention 在 vLLM 中的实现分析" (blog.chen3feng.top,
 *             vllm-analysis/07): §1.1 tiled online softmax, §4 forward() and the
 *             flash_attn_varlen_func call, §4.2 KV-cache update, §5 PagedAttention
 *             integration (block_table addressing), §6.3 cascade execution,
 *             §8.2 reshape_and_cache_flash / merge_attn_states, §9 DCP, §10 feature
 *             table.
 *   [FA/FI]   "FlashAttention と FlashInfer:2 大 GPU アテンションバックエンド":
 *             データフロー (KV cache shape, block size multiple of 16),
 *             境界と失敗 (head-size and dtype limits, FP8 KV cache).
 *   [Backend] "AttentionBackend:アテンションバックエンド抽象レイヤー": 境界と失敗
 *             (head size, block size ValueError, natural-log LSE).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller. The library
 *     never allocates device memory: temporaries live in a caller-provided
 *     workspace whose size the *_workspace_size functions return.
 *   - Work is enqueued on the caller's stream (`stream` is a cudaStream_t; NULL
 *     means the legacy default stream). Calls are asynchronous, make no
 *     host<->device copies, never synchronize, and keep no state between calls,
 *     so they can be recorded into a CUDA graph and called from several host
 *     threads on different streams with different workspaces.
 *   - Element type (the dtype argument): PA_BF16 (bfloat16) or PA_F16 (IEEE
 *     half) for Q, K, V and outputs, the same type for all of them within a
 *     call ([FA-vLLM] §2.1 lists float16 and bfloat16 as the supported
 *     dtypes); LSE is float32. The FP8 entry points (pa_*_fp8kv,
 *     pa_reshape_and_cache_fp8, or the fp8 option of pa_*_fwd_ex) hold K and
 *     V in the page pools as e4m3 bytes instead (Q, the new tokens and the
 *     outputs keep dtype). Arithmetic accumulates in float32; P enters the
 *     P V product in dtype (f16 over e4m3 pools).
 *   - Strides are in ELEMENTS. Every tensor pointer must be 16-byte aligned and
 *     every stride a multiple of 8 elements (16 bytes).
 *   - Return value: PA_OK, or an error code. On any host-side error nothing is
 *     launched and nothing is written. PA_ERR_CUDA reports a failed launch.
 *   - dev_status (nullable): a device int32 the kernels OR error bits into
 *     (PA_DEV_*) when they meet metadata they cannot use (a page id outside the
 *     pool, a slot outside the pool, a sequence longer than its page-table row,
 *     a bounded wait that gave up). The offending access is skipped, never
 *     performed: bad metadata cannot make a kernel read or write out of bounds.
 *     The caller clears the word; the library only ORs bits into it.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int pa_status;

#define PA_OK 0
#define PA_ERR_INVALID_ARG 1 /* null pointer, negative size, bad stride/alignment, H % H_kv != 0 */
#define PA_ERR_BLOCK_SIZE 2  /* block_size not a positive multiple of 16, or > 1024 */
#define PA_ERR_UNSUPPORTED 3 /* head_size or dtype not supported (see each entry point) */
#define PA_ERR_WORKSPACE 4   /* workspace NULL, misaligned or smaller than required */
#define PA_ERR_CUDA 5        /* a kernel launch or a CUDA runtime query failed */
#define PA_ERR_NOALLOC_LIMIT 6 /* problem needs more scratch than pa_varlen_fwd_noalloc's fixed buffer */

/* bits OR-ed into *dev_status by the kernels */
#define PA_DEV_BAD_PAGE 1    /* a block_table entry outside [0, num_blocks): its keys read as 0 */
#define PA_DEV_BAD_SLOT 2    /* a slot_mapping entry >= num_blocks * block_size: token skipped */
#define PA_DEV_BAD_SEQLEN 4  /* cu_seqlens_q / seqused_k inconsistent with the stated bounds */
#define PA_DEV_TIMEOUT 8     /* a bounded wait on a pipeline barrier gave up */
#define PA_DEV_CASCADE 16    /* cascade precondition violated (see pa_cascade_fwd) */
#define PA_DEV_BAD_POSITION 32 /* a token position past the cos/sin table: token skipped */

#define PA_BF16 0 /* bfloat16 */
#define PA_F16 1  /* IEEE half (float16) */

/* Human-readable name of a pa_status value (static string). */
const char* pa_status_string(pa_status status);

/* ABI version of this header (increments on any signature change). */
int pa_abi_version(void);

/*
 * pa_reshape_and_cache -- the slot_mapping scatter that writes new K/V rows
 * into their pages before attention ([FA-vLLM] §4.2 and §8.2
 * reshape_and_cache_flash; [FA/FI] 役割: the cache write is its own op).
 *
 *   key[t], value[t]  : [num_kv_heads, head_size] rows, token t at
 *                       key + t * key_token_stride (likewise value).
 *   key_cache, value_cache : page pools; page b starts at b * cache_block_stride
 *                       and holds [block_size, num_kv_heads, head_size]
 *                       contiguous (the NHD layout of [FA-vLLM] §5). Passing
 *                       cache_block_stride = 2*block_size*H_kv*D with value_cache
 *                       = key_cache + block_size*H_kv*D addresses a combined
 *                       [num_blocks, 2, block_size, H_kv, D] tensor ([FA/FI]
 *                       データフロー); the [2, num_blocks, ...] layout is two
 *                       plain pools.
 *   slot_mapping[t]   : int64 flat slot; the token goes to page slot / block_size,
 *                       row slot % block_size. slot < 0 skips the token (padding).
 *                       Slots must be distinct (duplicates: unspecified winner).
 * Bit-exact copy; no arithmetic on values.
 */
pa_status pa_reshape_and_cache(const void* key, const void* value, int64_t key_token_stride,
                               int64_t value_token_stride, void* key_cache, void* value_cache,
                               int64_t cache_block_stride, const int64_t* slot_mapping,
                               int num_tokens, int num_kv_heads, int head_size, int block_size,
                               int num_blocks, int dtype, int32_t* dev_status, void* stream);

/*
 * Workspace bytes pa_varlen_fwd needs for these bounds. sm_count is the
 * multiprocessor count of the device the call will run on (0: query the
 * current device). Returns 0 if the arguments are invalid.
 */
size_t pa_varlen_fwd_workspace_size(int num_seqs, int total_q, int max_seqlen_q, int max_seqlen_k,
                                    int num_heads, int num_kv_heads, int head_size, int block_size,
                                    int sm_count);

/*
 * pa_varlen_fwd -- varlen attention over a paged KV cache ([FA-vLLM] §4 call
 * flash_attn_varlen_func(q, k_cache, v_cache, cu_seqlens_q, seqused_k,
 * block_table, ...), §5 addressing, §1.1 tiled online softmax).
 *
 *   q            : [total_q, num_heads, head_size]; token t at q + t*q_token_stride,
 *                  heads contiguous.
 *   key_cache, value_cache, cache_block_stride : as in pa_reshape_and_cache.
 *   cu_seqlens_q : int32 [num_seqs + 1], nondecreasing prefix sums of query
 *                  lengths, cu_seqlens_q[0] = 0, cu_seqlens_q[num_seqs] = total_q.
 *   seqused_k    : int32 [num_seqs], number of keys of each sequence (>= 0).
 *   block_table  : int32 [num_seqs, bt_stride]; logical key j of sequence s is
 *                  row j % block_size of page block_table[s * bt_stride + j / block_size].
 *                  Only entries j / block_size < ceil(seqused_k[s] / block_size)
 *                  are read.
 *   max_seqlen_q, max_seqlen_k : host upper bounds of the query / key lengths
 *                  (used to size launches and the workspace; no device value is
 *                  read on the host). A looser bound gives the same results;
 *                  a sequence above it sets PA_DEV_BAD_SEQLEN.
 *   softmax_scale: multiplies q.k (commonly 1/sqrt(head_size)); any finite
 *                  value (PA_ERR_INVALID_ARG for NaN or infinity). A zero or
 *                  negative scale runs every segment on the split-KV kernel.
 *   causal       : 0 or 1. Causal masking is bottom-right aligned: query i of a
 *                  sequence with q_len queries and kv_len keys sees keys
 *                  j <= kv_len - q_len + i (a decode query sees all keys).
 *   GQA          : query head h reads KV head h / (num_heads / num_kv_heads);
 *                  any ratio (num_heads % num_kv_heads == 0). Groups of more
 *                  than 128 heads run every segment on the split-KV kernel.
 *   out          : [total_q, num_heads, head_size] in dtype, contiguous.
 *   lse          : float32 [num_heads, total_q] natural-log log-sum-exp of the
 *                  scaled logits each row saw, or NULL. A row that sees no key
 *                  gets out = 0 and lse = -inf.
 *   workspace    : >= pa_varlen_fwd_workspace_size(...) bytes, 256-byte aligned;
 *                  its contents need no initialisation and are scratch after the
 *                  call. One workspace must not be used by two calls in flight.
 */
pa_status pa_varlen_fwd(const void* q, int64_t q_token_stride, const void* key_cache,
                        const void* value_cache, int64_t cache_block_stride,
                        const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                        const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                        int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                        int head_size, int block_size, int num_blocks, float softmax_scale,
                        int causal, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, int dtype, int32_t* dev_status, void* stream);

/*
 * pa_merge_attn_states -- LSE-weighted combine of two partial attention
 * results over disjoint key sets ([FA-vLLM] §6.3 step 3 and §8.2
 * merge_attn_states(prefix_out, suffix_out, prefix_lse, suffix_lse)).
 *
 *   prefix_out, suffix_out, out : [num_tokens, num_heads, head_size] in dtype, contiguous.
 *   prefix_lse, suffix_lse      : float32 [num_heads, num_tokens], natural log.
 *   out_lse                     : float32 [num_heads, num_tokens] or NULL.
 * With m = max(a, b), wa = e^(a-m), wb = e^(b-m):
 *   out = (wa*prefix_out + wb*suffix_out) / (wa + wb), out_lse = m + ln(wa + wb);
 * a row whose two LSEs are both -inf gets out = 0, out_lse = -inf.
 * out may alias prefix_out or suffix_out.
 */
pa_status pa_merge_attn_states(void* out, float* out_lse, const void* prefix_out,
                               const float* prefix_lse, const void* suffix_out,
                               const float* suffix_lse, int num_tokens, int num_heads,
                               int head_size, int dtype, void* stream);

/*
 * pa_merge_attn_states_n -- LSE-weighted combine of num_parts partial
 * attention results over disjoint key sets: the merge step of decode context
 * parallelism ([FA-vLLM] §9 and the DCP branch of §4: every rank attends over
 * its own KV shard, non-causal for decode, and the ranks' partial (out, lse)
 * are merged by LSE -- there by all-gather + reduce-scatter across GPUs; here
 * on one GPU, for ranks that are virtual), and the n-part form of
 * pa_merge_attn_states.
 *
 *   parts_out : dtype; part r is [num_tokens, num_heads, head_size] contiguous
 *               at parts_out + r * part_stride_out (elements, a multiple of 8,
 *               >= num_tokens * num_heads * head_size when num_parts > 1).
 *   parts_lse : float32; part r is [num_heads, num_tokens] at
 *               parts_lse + r * part_stride_lse (>= num_heads * num_tokens).
 *   out       : [num_tokens, num_heads, head_size] in dtype; may alias a part.
 *   out_lse   : float32 [num_heads, num_tokens] or NULL; must not overlap the
 *               parts' LSEs (PA_ERR_INVALID_ARG).
 * With m = max_r lse_r and w_r = e^(lse_r - m): out = sum_r w_r out_r /
 * sum_r w_r, out_lse = m + ln sum_r w_r (float32 throughout, out rounded to
 * dtype once). A row whose LSEs are all -inf gets out = 0, out_lse = -inf.
 * 1 <= num_parts <= PA_MERGE_N_MAX.
 *
 * A virtual-rank decode over R ranks is R pa_varlen_fwd calls (causal = 0),
 * one per rank with that rank's block table and key counts, writing into the
 * parts of one stacked buffer, followed by this merge.
 */
#define PA_MERGE_N_MAX 1024
pa_status pa_merge_attn_states_n(void* out, float* out_lse, const void* parts_out,
                                 int64_t part_stride_out, const float* parts_lse,
                                 int64_t part_stride_lse, int num_parts, int num_tokens,
                                 int num_heads, int head_size, int dtype, void* stream);

/* Workspace bytes pa_cascade_fwd needs (same arguments as the varlen query). */
size_t pa_cascade_fwd_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                     int max_seqlen_k, int num_heads, int num_kv_heads,
                                     int head_size, int block_size, int sm_count);

/*
 * pa_cascade_fwd -- shared-prefix (cascade) attention ([FA-vLLM] §6.3):
 *   1. prefix pass: all total_q query tokens, as one non-causal segment,
 *      against the first common_prefix_len keys of block_table row 0;
 *   2. suffix pass: each sequence, causal, against its own keys from position
 *      common_prefix_len on (block_table[s, common_prefix_len/block_size:]);
 *   3. the two states merged by LSE as in pa_merge_attn_states.
 * The result equals pa_varlen_fwd(causal = 1) over the whole KV. Arguments as
 * pa_varlen_fwd plus common_prefix_len. Preconditions: common_prefix_len is a
 * multiple of block_size (else PA_ERR_INVALID_ARG); every row's first
 * common_prefix_len / block_size block_table entries equal row 0's; and
 * seqused_k[s] - q_len(s) >= common_prefix_len for every sequence, so every
 * query lies in its private suffix. A sequence that breaks the last rule sets
 * PA_DEV_CASCADE; its rows still follow the three steps literally (every
 * prefix key, then the causal suffix), which then differs from flat attention.
 * The shared-entries rule is not checked (row 0's pages are used).
 */
pa_status pa_cascade_fwd(const void* q, int64_t q_token_stride, const void* key_cache,
                         const void* value_cache, int64_t cache_block_stride,
                         const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                         const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                         int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                         int head_size, int block_size, int num_blocks, float softmax_scale,
                         int common_prefix_len, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, int dtype, int32_t* dev_status, void* stream);

/*
 * pa_use_cascade_attention -- should a batch run as cascade attention?
 * ([FA-vLLM] §6.2, use_cascade_attention: a shared prefix of at least 256
 * tokens, at least 8 requests, no ALiBi / sliding window / local attention
 * and no DCP -- a layer with a sliding window calls pa_window_fwd, not a
 * cascade; the others this library does not have -- then cascade outright if
 * split-KV decoding is off, else whichever of the two is estimated faster.)
 * The pages leave the estimate open; this one compares bytes: flat attention
 * reads the shared prefix once per sequence, cascade reads it once and pays
 * a fixed cost for its extra pass and merge, so cascade is chosen when
 *   (num_seqs - 1) * common_prefix_len * num_kv_heads * head_size * 4 bytes
 *     > PA_CASCADE_FIXED_US * 1e-6 * PA_CASCADE_HBM_GBS * 1e9,
 * i.e. when re-reading the prefix would cost more than the extra pass.
 *   split_kv : 1 if the flat path may split keys over CTAs (pa_varlen_fwd
 *              does), 0 if not.
 * Writes 1 (cascade) or 0 (flat) to *use_cascade. Host only, no CUDA call.
 * PA_ERR_INVALID_ARG for negative sizes or a NULL use_cascade.
 */
#define PA_CASCADE_FIXED_US 20.0
#define PA_CASCADE_HBM_GBS 6500.0
pa_status pa_use_cascade_attention(int common_prefix_len, int num_seqs, int num_kv_heads,
                                   int head_size, int split_kv, int* use_cascade);

/*
 * New tokens' K/V for the update-and-attend entry points below: the
 * arguments of pa_reshape_and_cache that are not already arguments of the
 * attention call. key / value: [num_tokens, num_kv_heads, head_size] in dtype,
 * token t at key + t*key_token_stride; slot_mapping: int64 [num_tokens]
 * (slot < 0 skips the token). All device pointers, owned by the caller.
 */
typedef struct pa_kv_update {
  const void* key;
  const void* value;
  int64_t key_token_stride;
  int64_t value_token_stride;
  const int64_t* slot_mapping;
  int num_tokens;
} pa_kv_update;

/*
 * pa_varlen_fwd_with_update / pa_cascade_fwd_with_update -- one serving step
 * ([FA-vLLM] §4.2: the forward pass first writes the step's new K/V into the
 * paged cache by slot_mapping, then attends): the same result as
 * pa_reshape_and_cache(update, key_cache, value_cache, ...) followed by
 * pa_varlen_fwd / pa_cascade_fwd with the remaining arguments, on the same
 * stream. In one call the planner and the scatter run concurrently (the
 * planner reads only the sequence metadata), and the attention kernels start
 * once both have finished. update may be NULL or have num_tokens = 0 (then
 * these equal pa_varlen_fwd / pa_cascade_fwd). The cache arguments
 * (cache_block_stride, num_kv_heads, head_size, block_size, num_blocks) and
 * dev_status serve both parts; the update's arguments are checked like
 * pa_reshape_and_cache's before anything is launched.
 */
pa_status pa_varlen_fwd_with_update(const pa_kv_update* update, const void* q,
                                    int64_t q_token_stride, void* key_cache, void* value_cache,
                                    int64_t cache_block_stride, const int32_t* cu_seqlens_q,
                                    const int32_t* seqused_k, const int32_t* block_table,
                                    int bt_stride, int num_seqs, int total_q, int max_seqlen_q,
                                    int max_seqlen_k, int num_heads, int num_kv_heads,
                                    int head_size, int block_size, int num_blocks,
                                    float softmax_scale, int causal, void* out, float* lse,
                                    void* workspace, size_t workspace_bytes, int dtype,
                                    int32_t* dev_status, void* stream);
pa_status pa_cascade_fwd_with_update(const pa_kv_update* update, const void* q,
                                     int64_t q_token_stride, void* key_cache, void* value_cache,
                                     int64_t cache_block_stride, const int32_t* cu_seqlens_q,
                                     const int32_t* seqused_k, const int32_t* block_table,
                                     int bt_stride, int num_seqs, int total_q, int max_seqlen_q,
                                     int max_seqlen_k, int num_heads, int num_kv_heads,
                                     int head_size, int block_size, int num_blocks,
                                     float softmax_scale, int common_prefix_len, void* out,
                                     float* lse, void* workspace, size_t workspace_bytes,
                                     int dtype, int32_t* dev_status, void* stream);

/*
 * pa_varlen_fwd_noalloc -- pa_varlen_fwd for callers that cannot allocate
 * device memory, so cannot provide a workspace: for example a serving engine
 * whose allocator reserved all device memory for its page pool at start-up,
 * or a latency-critical path where cudaMalloc's implicit device
 * synchronisation is not acceptable. The web pages have no counterpart to
 * this entry point; it only changes where the scratch lives.
 *
 * Arguments, layouts and results are those of pa_varlen_fwd without
 * workspace / workspace_bytes. The scratch is a fixed, library-owned
 * PA_NOALLOC_SCRATCH_BYTES (32 MiB) device buffer: every GPU that loads
 * libpa.so holds it until the process exits. A problem whose
 * pa_varlen_fwd_workspace_size exceeds it is rejected with
 * PA_ERR_NOALLOC_LIMIT before anything is launched. The function never calls
 * cudaMalloc, cudaFree or any allocating routine.
 *  - The first call on a device looks up that buffer's device address (with
 *    the device current) and caches it with the device's current context;
 *    make that first call before any stream capture on the device. After
 *    cudaDeviceReset (a new context) the next call looks it up again, so
 *    make that call before any capture too. A failed lookup returns
 *    PA_ERR_CUDA and leaves no CUDA error pending.
 *  - Every call uses the same buffer, which keeps the previous call's
 *    contents; the kernels rewrite everything they read before reading it, so
 *    nothing needs clearing. Calls that overlap on the GPU (two streams, or
 *    two host threads without ordering) race on the buffer: serialise them.
 */
#define PA_NOALLOC_SCRATCH_BYTES (32u << 20)

pa_status pa_varlen_fwd_noalloc(const void* q, int64_t q_token_stride, const void* key_cache,
                                const void* value_cache, int64_t cache_block_stride,
                                const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                                const int32_t* block_table, int bt_stride, int num_seqs,
                                int total_q, int max_seqlen_q, int max_seqlen_k, int num_heads,
                                int num_kv_heads, int head_size, int block_size, int num_blocks,
                                float softmax_scale, int causal, void* out, float* lse, int dtype,
                                int32_t* dev_status, void* stream);

/*
 * FP8 (e4m3) KV cache ([FA/FI] 役割 and 境界と失敗: FlashInfer and FA3 accept
 * an fp8 / fp8_e4m3 KV cache with per-head quant scales; [FA-vLLM] §10 lists an
 * FP8 KV cache among the backends' features).
 *
 * The pools hold one byte per element: the OCP 8-bit floating point "E4M3"
 * format (1 sign, 4 exponent bits with bias 7, 3 mantissa bits; largest
 * finite value 448, no infinities, S.1111.111 is NaN). A stored byte c of KV
 * head h means the value e4m3(c) * scale[h]. Writes store
 * e4m3(x / scale[h]): x is the bf16 or f16 input widened to float32, the division
 * is IEEE float32 (correctly rounded), the result is rounded to the nearest
 * e4m3 value (ties to even) and saturates at +-448 (a NaN stays NaN).
 * Attention computes exactly the 2-byte pools' definition on the dequantized
 * keys and values e4m3(c) * scale[h], with float32 accumulation. Segments
 * of more than 32 packed query rows (prefill) run on the tensor-core kernel:
 * q.k on the e4m3 tensor MMA straight from the stored key bytes, p.v on the
 * f16 MMA with each e4m3 V tile widened to f16 in shared memory (exact).
 * Shorter segments run on the split-KV kernel: items of at most 8 packed
 * rows (decode with GQA <= 8) take q.k on the e4m3 MMA too, wider ones form
 * q.k from f16 q (there |q| must stay below 65504). Wherever q.k is on the
 * e4m3 MMA, q is taken as two e4m3 terms after a power-of-two row scale:
 * exact for every bf16 element of at least 2^-9 of its row's largest; an f16
 * element, which has eleven significant bits, is rounded to about eight (off
 * by at most 2^-9 of its power of two). pa_window_fwd takes the query as it is,
 * on the f16 MMA, in calls of at most 8 packed rows per sequence and KV head
 * (max_seqlen_q * num_heads / num_kv_heads; long windows of few sequences
 * apart).
 * Layout: the NHD pools of pa_reshape_and_cache with 1-byte elements;
 * cache_block_stride is in elements (= bytes) and a multiple of 16.
 * head_size must be 128 (PA_ERR_UNSUPPORTED otherwise).
 */
typedef struct pa_kv_fp8 {
  const float* k_scale; /* device float32 [num_kv_heads], finite and > 0 (not checked) */
  const float* v_scale; /* device float32 [num_kv_heads], finite and > 0 (not checked) */
} pa_kv_fp8;

/*
 * pa_reshape_and_cache_fp8 -- pa_reshape_and_cache into e4m3 pools: key /
 * value are bf16 or f16 rows as there (dtype); each element is quantized
 * with its KV head's scale as described above. scales must be non-NULL with
 * both pointers 4-byte aligned (PA_ERR_INVALID_ARG).
 */
pa_status pa_reshape_and_cache_fp8(const void* key, const void* value, int64_t key_token_stride,
                                   int64_t value_token_stride, void* key_cache, void* value_cache,
                                   int64_t cache_block_stride, const int64_t* slot_mapping,
                                   int num_tokens, int num_kv_heads, int head_size,
                                   int block_size, int num_blocks, const pa_kv_fp8* scales,
                                   int dtype, int32_t* dev_status, void* stream);

/* Workspace bytes of pa_varlen_fwd_fp8kv / pa_cascade_fwd_fp8kv (0 if invalid). */
size_t pa_varlen_fwd_fp8kv_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                          int max_seqlen_k, int num_heads, int num_kv_heads,
                                          int head_size, int block_size, int sm_count);
size_t pa_cascade_fwd_fp8kv_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                           int max_seqlen_k, int num_heads, int num_kv_heads,
                                           int head_size, int block_size, int sm_count);

/*
 * pa_varlen_fwd_fp8kv / pa_cascade_fwd_fp8kv -- pa_varlen_fwd_with_update /
 * pa_cascade_fwd_with_update over e4m3 pools: the optional update (NULL or
 * num_tokens = 0 for none) is quantized into the pools as by
 * pa_reshape_and_cache_fp8, then the attention reads the dequantized cache.
 * q, out and lse are as in the other entry points (dtype PA_BF16 or PA_F16).
 */
pa_status pa_varlen_fwd_fp8kv(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                              void* key_cache, void* value_cache, int64_t cache_block_stride,
                              const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                              const int32_t* block_table, int bt_stride, int num_seqs,
                              int total_q, int max_seqlen_q, int max_seqlen_k, int num_heads,
                              int num_kv_heads, int head_size, int block_size, int num_blocks,
                              float softmax_scale, int causal, const pa_kv_fp8* scales, void* out,
                              float* lse, void* workspace, size_t workspace_bytes, int dtype,
                              int32_t* dev_status, void* stream);
pa_status pa_cascade_fwd_fp8kv(const pa_kv_update* update, const void* q,
                               int64_t q_token_stride, void* key_cache, void* value_cache,
                               int64_t cache_block_stride, const int32_t* cu_seqlens_q,
                               const int32_t* seqused_k, const int32_t* block_table,
                               int bt_stride, int num_seqs, int total_q, int max_seqlen_q,
                               int max_seqlen_k, int num_heads, int num_kv_heads, int head_size,
                               int block_size, int num_blocks, float softmax_scale,
                               int common_prefix_len, const pa_kv_fp8* scales, void* out,
                               float* lse, void* workspace, size_t workspace_bytes, int dtype,
                               int32_t* dev_status, void* stream);

/*
 * Options of the pa_*_fwd_ex entry points (NULL, or a NULL field, means the
 * default).
 *   sinks : attention sinks ([FA-vLLM] §1.2 and §1.3: the s_aux learnable sink
 *           token of FA3/FA4) -- device float32 [num_heads], one logit per
 *           query head in the units of softmax_scale * q.k, 4-byte aligned.
 *           Each acts as one more key of that logit and value zero: with
 *           s_j = softmax_scale * q.k_j over the visible keys,
 *           out = sum_j e^(s_j) v_j / (sum_j e^(s_j) + e^(sink)) and
 *           lse = ln(sum_j e^(s_j) + e^(sink)); a row with no visible key gets
 *           out = 0 and lse = sink.
 *   fp8   : NULL for 2-byte pools (dtype), else the pools hold e4m3 bytes with these
 *           scales (as in pa_varlen_fwd_fp8kv; workspace then per
 *           pa_*_fwd_fp8kv_workspace_size).
 */
typedef struct pa_attn_opts {
  const float* sinks;
  const pa_kv_fp8* fp8;
} pa_attn_opts;

/*
 * pa_varlen_fwd_ex / pa_cascade_fwd_ex -- pa_varlen_fwd_with_update /
 * pa_cascade_fwd_with_update with options (opts may be NULL: then they are
 * those entry points exactly).
 */
pa_status pa_varlen_fwd_ex(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                           void* key_cache, void* value_cache, int64_t cache_block_stride,
                           const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                           const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                           int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                           int head_size, int block_size, int num_blocks, float softmax_scale,
                           int causal, const pa_attn_opts* opts, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, int dtype,
                           int32_t* dev_status, void* stream);
pa_status pa_cascade_fwd_ex(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                            void* key_cache, void* value_cache, int64_t cache_block_stride,
                            const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                            const int32_t* block_table, int bt_stride, int num_seqs,
                            int total_q, int max_seqlen_q, int max_seqlen_k, int num_heads,
                            int num_kv_heads, int head_size, int block_size, int num_blocks,
                            float softmax_scale, int common_prefix_len, const pa_attn_opts* opts,
                            void* out, float* lse, void* workspace, size_t workspace_bytes,
                            int dtype, int32_t* dev_status, void* stream);

/*
 * pa_window_fwd -- pa_varlen_fwd_ex (causal) with a sliding window and a few
 * first tokens that stay visible: the query at position p (p = kv_len - q_len
 * + i) sees key j <= p if j > p - window (the last `window` keys, its own
 * among them) or j < num_first. window >= 1, num_first >= 0
 * (PA_ERR_INVALID_ARG); a window of at least max_seqlen_k is plain causal
 * attention. opts->sinks and opts->fp8 as there; workspace as for
 * pa_varlen_fwd (pa_varlen_fwd_fp8kv with opts->fp8).
 * Keys that no query of the call sees are not read in whole pages: their
 * block_table entries may be stale (the pages freed), and what the pages hold
 * does not matter, in partly visible pages either.
 */
pa_status pa_window_fwd(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                        void* key_cache, void* value_cache, int64_t cache_block_stride,
                        const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                        const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                        int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                        int head_size, int block_size, int num_blocks, float softmax_scale,
                        int window, int num_first, const pa_attn_opts* opts, void* out,
                        float* lse, void* workspace, size_t workspace_bytes, int dtype,
                        int32_t* dev_status, void* stream);

/*
 * pa_rope_table -- the rotary cos/sin table of positions 0 .. table_len - 1.
 * Pair i of rot_dim / 2 turns by f_i = base^(-2i / rot_dim) radians per
 * position; row p holds mscale * cos(p f_i) for every i, then mscale *
 * sin(p f_i). Angles are exact to about 1e-9 radian at a million positions.
 *   cos_sin  : float32 [table_len, rot_dim], 16-byte aligned.
 *   table_len: at most 2^30.
 *   rot_dim  : even, 2 .. 256 (pa_rope_and_cache takes multiples of 16).
 *   base     : finite, > 0 (rates of 2^53 turns per position and more are
 *              refused).
 *   scaling  : NULL for none, else how the rates change for contexts longer
 *              than the model was trained on (orig_len positions):
 *     PA_ROPE_LINEAR      f_i / factor
 *     PA_ROPE_NTK         base * factor^(rot_dim / (rot_dim - 2)) as the base
 *                         (rot_dim > 2)
 *     PA_ROPE_WAVELENGTH  with n = orig_len f_i / 2 pi turns in the original
 *                         length: f_i / factor where n <= low, f_i where n >=
 *                         high, a mix linear in n in between
 *     PA_ROPE_YARN        with d(n) = rot_dim ln(orig_len / (2 pi n)) / (2 ln
 *                         base), the pair that makes n turns: f_i below pair
 *                         floor(d(high)), f_i / factor from pair ceil(d(low))
 *                         on, a mix linear in i in between (base > 1)
 *              factor, orig_len > 0 and high > low > 0 where used; mscale
 *              finite, multiplies every entry (PA_ROPE_YARN commonly 0.1 ln
 *              factor + 1).
 * The scaling struct is read on the host during the call.
 */
#define PA_ROPE_NONE 0
#define PA_ROPE_LINEAR 1
#define PA_ROPE_NTK 2
#define PA_ROPE_WAVELENGTH 3
#define PA_ROPE_YARN 4
typedef struct pa_rope_scaling {
  int kind; /* PA_ROPE_* */
  double factor;
  double orig_len;
  double low;
  double high;
  double mscale;
} pa_rope_scaling;
pa_status pa_rope_table(float* cos_sin, int table_len, int rot_dim, double base,
                        const pa_rope_scaling* scaling, void* stream);

/*
 * pa_rope_and_cache -- what a decoder layer does to a step's new q, k and v
 * before attention, in one pass: per-head RMS norm of q and k (optional),
 * rotation of q and k, and the write of k and v into their pages
 * (pa_reshape_and_cache, or with fp8 pa_reshape_and_cache_fp8). The attention
 * call that follows takes q_out and no update.
 *   positions : int64 [num_tokens]; token t turns by row positions[t] of the
 *               table. A negative position marks a padding token: nothing of
 *               it is written. A position >= table_len sets
 *               PA_DEV_BAD_POSITION and its token is skipped likewise.
 *   q         : [num_tokens, num_heads, head_size] in dtype, token t at
 *               q + t*q_token_stride; q_out likewise. q_out may be q (same
 *               pointer and stride), or its rows may lie between q's (same
 *               stride); it must not overlap q otherwise (PA_ERR_INVALID_ARG),
 *               nor the update's keys and values.
 *   update    : the new tokens' k and v, their slots and num_tokens, as in
 *               pa_varlen_fwd_with_update. slot < 0: the token's k and v are
 *               not written (its q is).
 *   key_cache, value_cache, ... : as in pa_reshape_and_cache.
 *   fp8       : NULL for pools in dtype, else e4m3 pools with these scales
 *               (head_size 128).
 * With x a head of q or k: if the norm weight w is given, x_j becomes
 * x_j w_j / sqrt(mean(x^2) + norm_eps); then each pair (a, b) of the first
 * rot_dim elements becomes (a cos - b sin, b cos + a sin) and the rest stays.
 * All in float32 with one rounding, to dtype or to e4m3 (after the division
 * by the head's scale). v is copied (or quantized) as it is.
 */
typedef struct pa_rope {
  const float* cos_sin; /* device float32 [table_len, rot_dim], 16-byte aligned */
  int table_len;
  int rot_dim;          /* multiple of 16, <= head_size */
  int interleaved;      /* 1: pair i is elements (2i, 2i + 1); 0: (i, i + rot_dim / 2) */
  const float* q_norm;  /* device float32 [head_size], 16-byte aligned, or NULL: no norm */
  const float* k_norm;
  float norm_eps;       /* finite, >= 0 */
} pa_rope;
pa_status pa_rope_and_cache(const pa_rope* rope, const int64_t* positions, const void* q,
                            int64_t q_token_stride, void* q_out, int64_t q_out_token_stride,
                            const pa_kv_update* update, void* key_cache, void* value_cache,
                            int64_t cache_block_stride, int num_heads, int num_kv_heads,
                            int head_size, int block_size, int num_blocks, const pa_kv_fp8* fp8,
                            int dtype, int32_t* dev_status, void* stream);

/*
 * pa_attn_weights -- adds up, for every cached key, the attention weight that
 * a call's queries gave it: the running sums that pa_evict keeps keys by.
 *   q, key_cache, cu_seqlens_q, seqused_k, block_table, max_seqlen_q,
 *   max_seqlen_k, softmax_scale, causal : as in the attention call.
 *   lse       : float32 [num_heads, total_q], that call's log-sum-exp (with
 *               its sinks, if any; a row of -inf saw nothing and adds nothing,
 *               whatever its query holds). Not pa_window_fwd's: every key a
 *               causal query sees counts, a window is not applied.
 *   weights   : float32, one value per cache slot and KV head: key row r of
 *               page b, head h at b * weights_block_stride + h * block_size +
 *               r. weights_block_stride a multiple of 4.
 *   fp8       : NULL for a pool in dtype, else an e4m3 pool with these scales
 *               (head_size 128; only k_scale is read).
 * For every key j of a sequence of kv_len keys and q_len queries:
 *   weights[h][j] = (j >= kv_len - q_len ? 0 : weights[h][j])
 *                   + sum over queries i that see j, over heads g of KV head h,
 *                     of e^(softmax_scale q_ig.k_j - lse_ig)
 * so a key starts from 0 in the call that brings it. Rows past a sequence's
 * keys are left as they were. Sums are float32 in a fixed order: the same
 * call gives the same bits. A sequence's pages must be its own (a page shared
 * with another sequence of the call gets the sum of one of them).
 * max_seqlen_k and total_q * num_heads / num_kv_heads are at most 2^30, and
 * num_seqs * num_kv_heads * ceil(max_seqlen_k / 128) is at most 2^31 - 2
 * (PA_ERR_INVALID_ARG).
 * A key in a page outside the pool sets PA_DEV_BAD_PAGE and is skipped; a
 * sequence whose lengths break the stated bounds sets PA_DEV_BAD_SEQLEN, and
 * with inconsistent cu_seqlens_q it is skipped.
 */
pa_status pa_attn_weights(const void* q, int64_t q_token_stride, const void* key_cache,
                          int64_t cache_block_stride, const float* lse,
                          const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                          const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                          int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                          int head_size, int block_size, int num_blocks, float softmax_scale,
                          int causal, float* weights, int64_t weights_block_stride,
                          const pa_kv_fp8* fp8, int dtype, int32_t* dev_status, void* stream);

/*
 * pa_evict -- eviction by accumulated attention weight: every sequence of
 * more than `budget` keys is cut down to `budget`, per KV head, in place.
 * Each KV head keeps the first num_first keys, the last num_recent keys and
 * of the others those of the largest weight (ties: the lowest index; a NaN
 * counts as -inf). Kept keys keep their order and move to rows 0 .. budget - 1
 * of the sequence's pages, K, V and weights alike; rows from budget on are
 * left as they were, so the pages past the first ceil(budget / block_size)
 * may be freed. Sequences of at most budget keys stay untouched.
 * Keys are cached after their rotation, so moving them does not change what
 * later queries compute with them; the heads of a row then belong to
 * different tokens.
 *   elem_size    : bytes of a cache element: 2, or 1 (e4m3, head_size 128).
 *   weights      : as in pa_attn_weights.
 *   budget       : 1 .. 2^30, num_first, num_recent >= 0, num_first +
 *                  num_recent <= budget.
 *   kept         : int32 [num_seqs, num_kv_heads, budget], out: the former
 *                  index of each row, ascending; rows past a shorter
 *                  sequence's keys get -1.
 *   new_lens     : int32 [num_seqs], out: min(keys, budget). May be seqused_k.
 * A sequence's pages must be its own (rows are rewritten in place). A page
 * outside the pool sets PA_DEV_BAD_PAGE: its keys count as the lightest and
 * no row moves out of it or into it.
 */
pa_status pa_evict(void* key_cache, void* value_cache, int64_t cache_block_stride, float* weights,
                   int64_t weights_block_stride, const int32_t* seqused_k,
                   const int32_t* block_table, int bt_stride, int num_seqs, int max_seqlen_k,
                   int num_kv_heads, int head_size, int block_size, int num_blocks, int elem_size,
                   int budget, int num_first, int num_recent, int32_t* kept, int32_t* new_lens,
                   int32_t* dev_status, void* stream);

/*
 * 4-bit K/V cache. The pools hold codes of four bits, and every row (one token
 * of one KV head) has a scale and a minimum of its own:
 *   value of an element = code * scale + minimum, codes 0 .. 15.
 *   codes  : page b of a pool starts at b * cache_block_stride (in bytes, a
 *            multiple of 16) and holds [block_size, num_kv_heads, head_size / 2]
 *            bytes contiguous. Of each 8 consecutive elements 8w .. 8w + 7 the
 *            32-bit little-endian word w holds element 8w + 2i in bits 4i .. 4i +
 *            3 and element 8w + 2i + 1 in bits 16 + 4i .. 19 + 4i.
 *   params : pairs of f16, (scale, minimum); row r of page b, KV head h is pair
 *            b * params_block_stride + h * block_size + r; 16-byte aligned,
 *            params_block_stride (in pairs) a multiple of 4.
 * A row x is written as follows, in float32 with every operation rounded once:
 *   elements beyond +-32752 count as +-32752;
 *   scale = f16((max x - min x) * (1 / 15)), minimum = f16(min x);
 *   code = (x - minimum) * (1 / scale), brought into [0, 15] and rounded to
 *   the nearest integer, ties to even (0 for a scale of 0).
 * A row with a NaN gets NaN for scale and minimum, so all of it reads as NaN.
 * Head sizes 64 and 128 (PA_ERR_UNSUPPORTED otherwise).
 */
typedef struct pa_kv_int4 {
  void* k_params; /* device f16 pairs, written by the cache writes */
  void* v_params;
  int64_t params_block_stride; /* in pairs, >= num_kv_heads * block_size */
} pa_kv_int4;

/*
 * pa_reshape_and_cache_int4 -- pa_reshape_and_cache into 4-bit pools. (Of a slot that
 * occurs twice, codes and (scale, minimum) may be those of different tokens.)
 */
pa_status pa_reshape_and_cache_int4(const void* key, const void* value, int64_t key_token_stride,
                                    int64_t value_token_stride, void* key_cache, void* value_cache,
                                    int64_t cache_block_stride, const pa_kv_int4* int4,
                                    const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                                    int head_size, int block_size, int num_blocks, int dtype,
                                    int32_t* dev_status, void* stream);

/*
 * pa_rope_and_cache_int4 -- pa_rope_and_cache into 4-bit pools: the rotated
 * key is quantized from its float32 value. A rotated element is a cos - b sin
 * (b cos + a sin) with both products and the sum rounded to float32; norm
 * weights are multiplied into cos and sin before, and the norm's 1 / rms is
 * multiplied on last.
 */
pa_status pa_rope_and_cache_int4(const pa_rope* rope, const int64_t* positions, const void* q,
                                 int64_t q_token_stride, void* q_out, int64_t q_out_token_stride,
                                 const pa_kv_update* update, void* key_cache, void* value_cache,
                                 int64_t cache_block_stride, const pa_kv_int4* int4, int num_heads,
                                 int num_kv_heads, int head_size, int block_size, int num_blocks,
                                 int dtype, int32_t* dev_status, void* stream);

/*
 * pa_gather_cache_int4 -- rows of a 4-bit cache back as values, to move them
 * into 2-byte pools or to look at them: key and value, [num_tokens,
 * num_kv_heads, head_size] in dtype and contiguous, get code * scale + minimum
 * (float32, rounded once to dtype) of the rows at slot_mapping. A slot may
 * occur more than once; a token whose slot is negative, or past the pool
 * (PA_DEV_BAD_SLOT), gets zeros. The outputs must not overlap the pools.
 */
pa_status pa_gather_cache_int4(const void* key_cache, const void* value_cache,
                               int64_t cache_block_stride, const pa_kv_int4* int4,
                               const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                               int head_size, int block_size, int num_blocks, void* key,
                               void* value, int dtype, int32_t* dev_status, void* stream);

/*
 * pa_varlen_fwd_int4kv -- pa_varlen_fwd_ex over 4-bit pools: the optional
 * update (NULL or num_tokens = 0 for none) is written as by
 * pa_reshape_and_cache_int4, then the attention reads the cache's values code *
 * scale + minimum. sinks as in pa_attn_opts (NULL for none). Groups of at most
 * 128 query heads per KV head (PA_ERR_UNSUPPORTED otherwise); max_seqlen_k at
 * most 2^30 (PA_ERR_INVALID_ARG).
 * q.k is formed from the codes themselves, which the products take exactly, and
 * scale and minimum are applied to the sums in float32.
 * Sequences of at most 32 packed query rows (tokens x heads of the group; decode
 * and short queries): q is taken as f16 after a power-of-two row scale, exact for
 * every bf16 element of at least 2^-27 of its row's largest. The weights times V's
 * scale are rounded to f16 after a power of two. Longer sequences run on the
 * tensor-core kernel: q as it is, V widened to f16 values (one rounding, at most
 * 2^-11 of a value, 2^-25 of one below 2^-14) and the weights in f16; there, as in
 * the other prefill kernels, a NaN in V also reaches queries of the call that stand
 * less than a key tile in front of it.
 * In pages that are read, rows past a sequence's keys do not matter.
 * The workspace has a place for what any warp of the device may leave: for up to 8
 * (32) packed rows 20 MB (40 MB) at head size 128 and 152 multiprocessors, however few
 * the sequences; where neither 3 nor 4 divides num_kv_heads, half of that and 17 kB (66
 * kB) per sequence and pair of KV heads (per KV head, if their number is odd).
 */
size_t pa_varlen_fwd_int4kv_workspace_size(int num_seqs, int total_q, int max_seqlen_q,
                                           int max_seqlen_k, int num_heads, int num_kv_heads,
                                           int head_size, int block_size, int sm_count);
pa_status pa_varlen_fwd_int4kv(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                               void* key_cache, void* value_cache, int64_t cache_block_stride,
                               const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                               const int32_t* block_table, int bt_stride, int num_seqs,
                               int total_q, int max_seqlen_q, int max_seqlen_k, int num_heads,
                               int num_kv_heads, int head_size, int block_size, int num_blocks,
                               float softmax_scale, int causal, const pa_kv_int4* int4,
                               const float* sinks, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, int dtype, int32_t* dev_status,
                               void* stream);

/*
 * pa_score_fwd -- pa_varlen_fwd_ex (causal) with changed scores and masks: the
 * query of head h at position p (p = kv_len - q_len + i) gives a key j that it
 * sees the score
 *   s = softmax_scale q.k_j,
 *   s = softcap tanh(s / softcap)              (softcap > 0),
 *   s = s - alibi_slopes[h] |p - j|            (alibi_slopes given),
 * and it sees key j if
 *   j >= first_key[its token]                  (first_key given: documents packed
 *                                               into one sequence), and
 *   j <= p, or j < prefix_lens[its sequence]   (prefix_lens given: a prefix that
 *                                               sees itself whole).
 * (A window of w tokens beside a cap or a bias: first_key = position - w + 1.)
 * score may be NULL, its pointers too; without any, this is pa_varlen_fwd_ex. A
 * row that sees no key gets out = 0 and lse = -inf (with a sink: lse = the sink).
 * A cap moves a score by at most 2^-20 of the score from its exact value (while
 * softmax_scale / softcap is a normal float32), one up to 128 by at most 2^-20 of the
 * cap.
 * Pools in dtype only: opts->fp8 must be NULL (PA_ERR_UNSUPPORTED). Workspace as
 * for pa_varlen_fwd.
 * Key tiles in front of the first key of all of a tile's queries are not read.
 * What a page holds past its sequence's keys, or in keys that no query of a row
 * tile sees in front of its first key, does not matter; keys that some of its
 * queries see must be finite in V.
 */
typedef struct pa_score {
  float softcap;              /* >= 0, 0: none; 2 log2(e) softmax_scale / softcap must be finite */
  const float* alibi_slopes;  /* device float32 [num_heads] or NULL */
  const int32_t* prefix_lens; /* device int32 [num_seqs] or NULL; outside [0, kv_len]: clamped */
  const int32_t* first_key;   /* device int32 [total_q] or NULL; negative: 0 */
} pa_score;
pa_status pa_score_fwd(const pa_kv_update* update, const void* q, int64_t q_token_stride,
                       void* key_cache, void* value_cache, int64_t cache_block_stride,
                       const int32_t* cu_seqlens_q, const int32_t* seqused_k,
                       const int32_t* block_table, int bt_stride, int num_seqs, int total_q,
                       int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                       int head_size, int block_size, int num_blocks, float softmax_scale,
                       const pa_score* score, const pa_attn_opts* opts, void* out, float* lse,
                       void* workspace, size_t workspace_bytes, int dtype, int32_t* dev_status,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
