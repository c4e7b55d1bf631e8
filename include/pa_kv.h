/*
 * pa_kv.h -- C ABI of the paged KV-cache attention library (libpa_kv.so).
 *
 * PagedAttention keeps each sequence's keys and values in fixed-size blocks
 * of `block_size` tokens per KV head; the blocks sit at arbitrary physical
 * block ids and a per-sequence block table maps logical block j (tokens
 * j*block_size .. (j+1)*block_size-1) to its physical id.  Sources:
 *   - vLLM PagedAttention design doc ("分页注意力机制", vllm.ooos.top):
 *     sections 输入参数 (q, k_cache, v_cache, out), 概念 (sequence, context,
 *     block), QK, Softmax, Value, Output.
 *   - "Paged 어텐션" (data-sketchers.com transformers paged-attention wiki):
 *     "Decode 경로" (block_table [batch, max_blocks_per_seq], -1 =
 *     unallocated, cache_seqlens, in-place cache update) and "Varlen 경로"
 *     (cu_seq_lens_q / cu_seq_lens_k, max_seqlen_q / max_seqlen_k).
 *   - "Как работает paged attention? (детально)" (aivaro.ru answers/837):
 *     sections 3.2 BlockManager, 3.3 copy-on-write, 4.1-4.2 allocation and
 *     deallocation, 5.1 block-wise attention.
 *   - vLLM paper summary (easyvpn24.com/25506.html): sections 2-4.
 *
 * Conventions for every call below:
 *   - Device pointers point to memory the caller owns (e.g. torch tensors);
 *     the device calls allocate nothing.  All device work is queued on
 *     `stream` (a cudaStream_t; NULL = the legacy default stream) and is
 *     asynchronous; the call returns once the work is queued.
 *   - Arguments are checked on the host before anything is launched; a bad
 *     argument returns PA_ERR_INVALID_ARG or PA_ERR_UNSUPPORTED and launches
 *     nothing.  A failed launch returns PA_ERR_CUDA.
 *   - Errors that depend on device data (a block id outside the pool, a slot
 *     outside the cache, a length above the stated maximum, a wait that ran
 *     out of time) are written to *dev_status (a device int32 the caller
 *     zeroes; may be NULL): the first error code wins.  The kernels never trap.
 *   - Cache layout (both K and V): [num_blocks][num_kv_heads][block_size]
 *     [head_size], row-major, so one (block, kv head) page is one contiguous
 *     block_size*head_size run.
 *   - GQA: query head h reads KV head h / (num_heads / num_kv_heads);
 *     num_heads must be a multiple of num_kv_heads.
 *   - Pool handles (pa_pool_*) hold host memory only and are not thread-safe.
 */
#ifndef PA_KV_H
#define PA_KV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* the same type as cudaStream_t */
typedef struct CUstream_st* pa_stream_t;

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,  /* bad pointer, size, shape or length */
    PA_ERR_UNSUPPORTED = 2,  /* valid, but a head size / dtype / block size not built */
    PA_ERR_OOM = 3,          /* the block pool has too few free blocks, or the host no memory */
    PA_ERR_CUDA = 4,         /* a CUDA launch or query failed */
    PA_ERR_TIMEOUT = 5,      /* device: a bounded wait ran out (dev_status only) */
    PA_ERR_BAD_BLOCK = 6     /* device: block id or slot outside the cache */
} pa_status;

typedef enum {
    PA_F16 = 0,       /* IEEE binary16 */
    PA_BF16 = 1,      /* bfloat16 */
    PA_FP8_E4M3 = 2,  /* OCP FP8 E4M3 (finite-only "fn"), KV cache only */
    PA_F32 = 3        /* IEEE binary32, logits only (pa_beam_select) */
} pa_dtype;

/* Description of one layer's paged KV cache (device memory owned by the
 * caller).  k_cache / v_cache: [num_blocks][num_kv_heads][block_size]
 * [head_size] elements of kv_dtype, 16-byte aligned.  For PA_FP8_E4M3 a
 * stored code c means the value c * k_scale (keys) or c * v_scale (values);
 * the scales are ignored for 16-bit caches. ("FP8 KV Cache" in the vLLM
 * feature list on "ChunkLlama", docsearch.algolia.com.) */
typedef struct {
    void* k_cache;
    void* v_cache;
    int64_t num_blocks;
    int32_t block_size;
    int32_t num_kv_heads;
    int32_t head_size;
    pa_dtype kv_dtype;
    float k_scale;
    float v_scale;
} pa_kv_cache;

/* Human-readable name of a status code (static string). */
const char* pa_status_str(pa_status s);

/* Library version, major*10000 + minor*100 + patch. */
int32_t pa_version(void);

/* ---------------------------------------------------------------------------
 * Write new K/V rows into their cache slots.
 * "Paged 어텐션", Decode 경로 (the cache is updated in place through the
 * block table); "Как работает paged attention?" 4.1 step 5 (the new token's
 * KV goes to its position in the physical block); vLLM paper summary §3.
 *
 * k, v: device, [num_tokens][num_kv_heads][head_size] of in_dtype (F16 or
 *   BF16); consecutive tokens are token_stride elements apart (>=
 *   num_kv_heads*head_size; lets k/v be views into a fused qkv buffer).
 * slot_mapping: device int64 [num_tokens]; slot s means physical block
 *   s / block_size, offset s % block_size; s < 0 skips the token (padding).
 *   A slot >= num_blocks*block_size is skipped and reported as
 *   PA_ERR_BAD_BLOCK in *dev_status.
 * A 16-bit cache must have kv_dtype == in_dtype: the bits are moved
 *   unchanged.  An E4M3 cache stores e4m3_satfinite(round-to-nearest-even(
 *   (float)x / scale)), the division done in IEEE binary32.
 * Several tokens with the same slot: which one's elements land is unspecified (a
 * mixture of theirs is possible).
 * ------------------------------------------------------------------------- */
pa_status pa_kv_cache_write(const pa_kv_cache* cache, const void* k, const void* v,
                            pa_dtype in_dtype, int64_t num_tokens, int64_t token_stride,
                            const int64_t* slot_mapping, int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Norms of the queries and keys of each head, the rotary position rotation and
 * the cache write.  (The pages start from ready queries and keys; a decoder
 * layer gets them this way: the new token's K/V of "Как работает paged
 * attention?" 4.1 are its normed and rotated projections.)
 *
 * Frequencies.  Pair i < rotary_dim/2 of a head's rotated part turns by
 * position * theta_i radians, theta_i = base^(-2i/rotary_dim), changed for
 * longer contexts by `scaling` (NULL: not at all):
 *   PA_ROPE_LINEAR  theta_i / factor
 *   PA_ROPE_NTK     theta_i of the base  base * factor^(r/(r-2)), r = rotary_dim
 *   PA_ROPE_YARN    theta_i (1 - g) + theta_i / factor * g, g going linearly from 0
 *                   at pair  floor(at(beta_fast))  to 1 at  ceil(at(beta_slow)),
 *                   at(x) = r ln(original_max_position / (2 pi x)) / (2 ln base)
 *                   (both clipped to 0 .. r-1); cos and sin times 0.1 ln(factor) + 1
 *   PA_ROPE_BANDED  theta_i w + theta_i / factor * (1 - w), with the pair's turns over
 *                   the original context  c = original_max_position theta_i / (2 pi):
 *                   w = clip((c - low_freq_factor) / (high_freq_factor -
 *                   low_freq_factor), 0, 1)
 *   PA_ROPE_GIVEN   inv_freq holds the caller's own theta_i (an input; any finite values)
 * pa_rope_frequencies is a host call on host arrays: it writes inv_freq
 * [rotary_dim/2] (theta_i) and turns [rotary_dim/2], the same as turns per position
 * in units of 2^-64 (what the kernels read: copy it to the device once), and the
 * factor of cos and sin.  rotary_dim even and >= 2, base > 1, factor >= 1.
 * ------------------------------------------------------------------------- */
typedef enum {
    PA_ROPE_NONE = 0,
    PA_ROPE_LINEAR = 1,
    PA_ROPE_NTK = 2,
    PA_ROPE_YARN = 3,
    PA_ROPE_BANDED = 4,
    PA_ROPE_GIVEN = 5
} pa_rope_kind;

typedef struct {
    pa_rope_kind kind;
    double factor;
    double original_max_position;             /* YARN, BANDED */
    double beta_fast, beta_slow;              /* YARN */
    double low_freq_factor, high_freq_factor; /* BANDED */
} pa_rope_scaling;

pa_status pa_rope_frequencies(int32_t rotary_dim, double base, const pa_rope_scaling* scaling, double* inv_freq,
                              uint64_t* turns, float* rope_factor);

/* What is done to a head's row x of D = head_size elements (host struct, device
 * pointers):
 *     y = x / sqrt(mean(x^2) + eps) * weight    (weight NULL: y = x)
 *     out_a = rope_factor (y_a cos(p theta_i) - y_b sin(p theta_i))
 *     out_b = rope_factor (y_b cos(p theta_i) + y_a sin(p theta_i))
 * for the pairs i < rotary_dim/2 of the first rotary_dim elements, (a, b) = (i, i +
 * rotary_dim/2), or (2i, 2i + 1) when interleaved != 0; the other elements are y.
 * p is the token's position.  Everything is computed in binary32 and rounded
 * once (to nearest even) to the output's type. */
typedef struct {
    const float* q_weight;   /* device [head_size], 16-byte aligned; NULL: queries are not normed */
    const float* k_weight;   /* likewise for the keys */
    float eps;               /* > 0 where a weight is given */
    const uint64_t* turns;   /* device [rotary_dim/2], from pa_rope_frequencies */
    float rope_factor;
    int32_t rotary_dim;      /* 0 (no rotation) or a multiple of 16, at most head_size */
    int32_t interleaved;
} pa_qk_transform;

/* Queries and keys to packed rows (as pa_prefill_varlen_packed reads them).
 * q, k: device rows of `dtype` (F16 or BF16), [num_tokens][num_heads or
 *   num_kv_heads][head_size], consecutive tokens q_stride / k_stride elements apart
 *   (views into a fused qkv buffer); q_out, k_out likewise.  Any alignment that the
 *   type has (16-byte aligned pointers and strides go faster).  q_out may be q
 *   itself with the same stride, and k_out k; no other overlap.
 * positions: device int64 [num_tokens], any values (NULL when rotary_dim is 0).
 * Supported: head_size 64 or 128; up to 4096 heads of each. */
pa_status pa_qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k, pa_dtype dtype, int64_t num_tokens,
                          int32_t num_heads, int32_t num_kv_heads, int32_t head_size, int64_t q_stride,
                          int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride, const int64_t* positions,
                          const pa_qk_transform* transform, pa_stream_t stream);

/* The same with the keys and values written to their cache slots: queries to q_out,
 * keys (normed and rotated) and values (as they are) to slot_mapping's slots, which
 * work as in pa_kv_cache_write (s < 0: the token's K/V are not written, its queries
 * still are; a slot past the cache is reported as PA_ERR_BAD_BLOCK).  A 16-bit cache
 * has kv_dtype == dtype; an E4M3 cache stores e4m3_satfinite(round-to-nearest-even(
 * out / scale)) of the binary32 out: no 16-bit rounding in between. */
pa_status pa_qk_norm_rope_write(void* q_out, const void* q, const void* k, const void* v, pa_dtype dtype,
                                const pa_kv_cache* cache, int64_t num_tokens, int32_t num_heads, int64_t q_stride,
                                int64_t k_stride, int64_t v_stride, int64_t q_out_stride, const int64_t* positions,
                                const int64_t* slot_mapping, const pa_qk_transform* transform, int32_t* dev_status,
                                pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Copy whole physical blocks (all KV heads, K and V): the device half of
 * copy-on-write ("Как работает paged attention?" 3.3: a shared block is
 * copied before a sequence writes into it).
 * src_dst_pairs: device int32 [n][2] = (source id, destination id).  A pair
 * with an id outside [0, num_blocks) is skipped and reported as
 * PA_ERR_BAD_BLOCK.  Destinations must be distinct and not also sources.
 * ------------------------------------------------------------------------- */
pa_status pa_copy_blocks(const pa_kv_cache* cache, const int32_t* src_dst_pairs, int32_t n,
                         int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Single-query decode attention over the paged cache.
 * vLLM PagedAttention design doc (whole walk-through: QK, Softmax, Value,
 * Output; the grid axis over context partitions); "Paged 어텐션" Decode 경로.
 *
 * For every sequence b and query head h, with L = seq_lens[b] and
 * kvh = h / (num_heads / num_kv_heads):
 *     s_t = scale * sum_d q[b][h][d] * K_b[t][d]      for t < L
 *     out[b][h][:] = sum_t softmax(s)_t * V_b[t][:]
 * where K_b[t] = k_cache[block_table[b][t / block_size]][kvh][t % block_size]
 * (times k_scale for E4M3), V_b likewise.  L = 0 gives out = 0.  Positions
 * t >= L take no part (they may hold anything, NaN included).
 *
 * out, q: device [num_seqs][num_heads][head_size] of q_dtype (F16 or BF16),
 *   16-byte aligned.  q_dtype must equal kv_dtype for 16-bit caches; an E4M3
 *   cache takes F16 or BF16 queries.  out is rounded to nearest even.
 * block_table: device int32 [num_seqs][max_blocks_per_seq]; only the first
 *   ceil(L / block_size) entries of a row are read; each must be in
 *   [0, num_blocks), otherwise PA_ERR_BAD_BLOCK is reported and that page is
 *   left out.
 * seq_lens: device int32 [num_seqs], the attended lengths ("cache_seqlens"
 *   counting the token just written).  Each must be <= max_seq_len and
 *   <= max_blocks_per_seq*block_size, otherwise PA_ERR_INVALID_ARG is
 *   reported and the sequence's output is 0.
 * partition_size: tokens per context partition (a multiple of block_size),
 *   0 = automatic (pa_decode_partition_size: 2048, or 1024 when num_heads /
 *   num_kv_heads >= 4; with fewer (sequence, KV head) pairs than resident
 *   decode blocks, doubled up to 8192 while the work items of max_seq_len
 *   still number four or more per block; with more pairs and num_heads /
 *   num_kv_heads >= 4, 1536; then halved, not below 512, while the items
 *   would not fill the GPU twice over; the workspace size query answers for
 *   512, which covers every automatic choice).  A
 *   sequence longer than one partition is split; the
 *   partitions' partial results go to `workspace` and a second kernel merges
 *   them by their log-sum-exp.
 * workspace: device scratch of at least pa_decode_workspace_size(...) bytes,
 *   16-byte aligned (may be NULL when that size is 0).
 * Supported: head_size 64 or 128; block_size 16, 32 or 64;
 *   num_heads / num_kv_heads in {1, 2, 4, 8}.
 * ------------------------------------------------------------------------- */
size_t pa_decode_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t head_size,
                                int32_t max_seq_len, int32_t block_size, int32_t partition_size);

/* The partition size pa_decode takes for partition_size = 0 on the current
 * device (host call, no launch); 0 for invalid arguments. */
int32_t pa_decode_partition_size(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                 int32_t max_seq_len);

pa_status pa_decode(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                    const int32_t* block_table, int32_t max_blocks_per_seq,
                    const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                    int32_t num_heads, float scale, int32_t partition_size, void* workspace,
                    size_t workspace_bytes, int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * pa_decode for callers that cannot allocate device memory.  (The pages have
 * no counterpart: this is a property of the library, not of the method.)
 *
 * Some callers cannot call cudaMalloc: a plugin or embedded runtime whose host
 * program owns all device memory through its own allocator, or a serving loop
 * that must not call cudaMalloc/cudaFree because they can synchronise the
 * device.  This call takes the same arguments as pa_decode minus the
 * workspace: the split-K partial results go to a scratch array of
 * PA_DECODE_STATIC_WS_BYTES that is built into the library and held by every
 * GPU that loads it until the process exits.  It allocates nothing.
 *   - partition_size 0 is resolved first (pa_decode_partition_size) and the
 *     resolved partition is the one both the size check and the launch use.
 *   - A call whose pa_decode_workspace_size(..., resolved partition) exceeds
 *     PA_DECODE_STATIC_WS_BYTES returns PA_ERR_UNSUPPORTED and launches
 *     nothing (use pa_decode with a workspace of your own instead).
 *   - The first call on a device looks up the scratch's device address
 *     (cudaGetSymbolAddress, with that device current) and remembers it
 *     together with the context then current; a call that finds another
 *     context current (after cudaDeviceReset, or in a context the caller
 *     created) looks it up again.  Make the first call on a device, and in
 *     each such new context, before any stream capture.
 *   - Every call on a device shares the one array and finds the previous
 *     call's data in it; nothing needs clearing, but calls whose kernels
 *     overlap on the GPU (e.g. on two unordered streams) race and give wrong
 *     results.  Order them on one stream.
 * ------------------------------------------------------------------------- */
#define PA_DECODE_STATIC_WS_BYTES (16u * 1024u * 1024u)

pa_status pa_decode_static_ws(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                              const int32_t* block_table, int32_t max_blocks_per_seq,
                              const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                              int32_t num_heads, float scale, int32_t partition_size,
                              int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Single-query decode with a sliding window and sinks.  (The pages attend the
 * whole context; this is the mask of layers whose queries see only the last
 * tokens and, so that the softmax keeps its anchor, a few first ones.)
 *
 * As pa_decode, but the query of sequence b, at position L - 1 (L = seq_lens[b]),
 * sees the positions t < L with
 *     t >= L - window   or   t < num_sinks,
 * window >= 1 counting the query's own position, num_sinks >= 0.  A window or a
 * sink count of L or more gives pa_decode's result.  Only the blocks that hold a
 * visible position are read: a row's other entries may be anything (-1 after
 * pa_pool_release_window), and what the blocks hold at positions that are not
 * seen (NaN included) takes no part.
 * partition_size counts the tokens of the blocks read (the sinks' whole blocks,
 * then the window's); 0 cuts them into equal parts that fill the GPU, of 128
 * tokens or more.  workspace: pa_decode_window_workspace_size
 * (...) bytes with the same arguments.  Everything else as pa_decode.
 * Rounding (pa_decode's too): scores, maxima, sums and outputs are binary32 up to the one
 * rounding of out, with these exceptions.  With num_heads / num_kv_heads of 4 or 8 a
 * weight meets its value in 16 bits on the tensor cores: fp16 and E4M3 caches as fp16
 * (off by 2^-11 of itself, below 2^-14 of the largest by 2^-25 of that), bf16 caches as
 * two bf16 parts (2^-16).  Over an E4M3 cache a head's query is taken in fp16 relative to
 * its largest component: exact but for components 2^28 times smaller.
 * ------------------------------------------------------------------------- */
size_t pa_decode_window_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t head_size, int32_t max_seq_len,
                                       int32_t block_size, int32_t window, int32_t num_sinks,
                                       int32_t partition_size);
pa_status pa_decode_window(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                           const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                           int32_t num_seqs, int32_t max_seq_len, int32_t num_heads, float scale, int32_t window,
                           int32_t num_sinks, int32_t partition_size, void* workspace, size_t workspace_bytes,
                           int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Varlen prefill (and mixed prefill + decode) attention over the paged cache.
 * "Paged 어텐션" Varlen 경로 (cu_seq_lens_q/k index a batch of sequences of
 * different lengths; max_seqlen_q/k bound them); keys and values are read
 * from the paged cache through block_table as in the Decode 경로; causal
 * masking per block as in "Как работает paged attention?" 5.1.
 *
 * Sequence b owns query rows cu_seq_lens_q[b] .. cu_seq_lens_q[b+1]-1 of q
 * and has Lk = cu_seq_lens_k[b+1] - cu_seq_lens_k[b] keys at logical
 * positions 0..Lk-1 of its block-table row (the new tokens' K/V must already
 * be in the cache, e.g. by pa_kv_cache_write).  With Lq query rows, query i
 * sits at position Lk - Lq + i; with causal != 0 it sees keys j <= Lk - Lq + i
 * (bottom-right alignment), otherwise all Lk keys.  A row that sees no key
 * outputs 0.  A value that some query of a sequence sees must be finite for the
 * sequence's other queries too (a weight of zero still multiplies it).
 * q, out: device [total_q][num_heads][head_size] of q_dtype (BF16 or F16,
 *   equal to kv_dtype), total_q = cu_seq_lens_q[num_seqs], 16-byte aligned.
 * cu_seq_lens_q, cu_seq_lens_k: device int32 [num_seqs + 1], non-decreasing,
 *   starting at 0.  max_seqlen_q / max_seqlen_k must bound the lengths (a
 *   sequence that breaks them is reported as PA_ERR_INVALID_ARG and its rows
 *   are not written).  A block id outside [0, num_blocks) among the entries
 *   a sequence needs is reported as PA_ERR_BAD_BLOCK; that sequence's rows are
 *   then unspecified.
 * Supported: head_size 128; block_size 16, 32 or 64;
 *   num_heads / num_kv_heads in {1, 2, 4, 8}; 16-bit caches.
 * ------------------------------------------------------------------------- */
pa_status pa_prefill_varlen(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                            const int32_t* block_table, int32_t max_blocks_per_seq,
                            const int32_t* cu_seq_lens_q, const int32_t* cu_seq_lens_k,
                            int32_t num_seqs, int32_t max_seqlen_q, int32_t max_seqlen_k,
                            int32_t num_heads, float scale, int32_t causal, int32_t* dev_status,
                            pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Varlen prefill with a sliding window and sinks: pa_prefill_varlen, causal, with
 * pa_decode_window's mask.  Query i of a sequence, at position x = Lk - Lq + i, sees
 * the keys
 *     j <= x   with   j > x - window   or   j < num_sinks.
 * A window of max_seqlen_k or more gives pa_prefill_varlen's causal result.
 * Block-table entries of blocks that no query of the sequence sees are not read,
 * and what a query does not see takes no part in its output, whatever it is (infinite
 * or NaN, and also where other queries see it).  A value that is not finite and that
 * a query sees costs time: the rows that share its tiles are worked out one by one.
 * scale > 0.  Everything else as pa_prefill_varlen (head_size 128).
 * Rounding (pa_prefill_varlen's too): scores, maxima, sums and outputs are binary32 up to
 * the one rounding of out; a weight meets its value in 16 bits on the tensor cores, as
 * fp16 (off by 2^-11 of itself) or, with bf16 caches, as two bf16 parts (2^-16).
 * ------------------------------------------------------------------------- */
pa_status pa_prefill_varlen_window(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                                   const int32_t* block_table, int32_t max_blocks_per_seq,
                                   const int32_t* cu_seq_lens_q, const int32_t* cu_seq_lens_k, int32_t num_seqs,
                                   int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t num_heads, float scale,
                                   int32_t window, int32_t num_sinks, int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Swap whole blocks between the device cache and page-locked host memory:
 * the data move of swap-based preemption ("Как работает paged attention?"
 * 4.3: the preempted request's KV cache goes to CPU memory and comes back
 * when it resumes; vLLM paper summary, section 5: a CPU block allocator
 * holds the swapped blocks).  Which requests to preempt, and the host-side
 * block ids, are the caller's (a scheduler's) business.
 *
 * host_k, host_v: page-locked host memory (cudaHostAlloc / cudaMallocHost /
 *   cudaHostRegister, or a pinned torch tensor), 16-byte aligned, laid out
 *   like the cache: [num_host_blocks][num_kv_heads][block_size][head_size]
 *   of the cache's dtype.  Pageable memory is rejected (PA_ERR_INVALID_ARG).
 * pairs: device int32 [n][2] = (device block id, host block id), n <= 65535.
 *   to_host != 0 copies device -> host (swap out), 0 copies host -> device
 *   (swap in).  A pair with an id out of range is skipped and reported as
 *   PA_ERR_BAD_BLOCK.  Destinations must be distinct.
 * Asynchronous on `stream`; the host buffers must stay valid (and, for swap
 * out, unread) until the stream reaches this point.
 * ------------------------------------------------------------------------- */
pa_status pa_swap_blocks(const pa_kv_cache* cache, void* host_k, void* host_v, int64_t num_host_blocks,
                         const int32_t* pairs, int32_t n, int32_t to_host, int32_t* dev_status,
                         pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Fused cache write + decode: for every sequence b with L = seq_lens[b] >= 1,
 * the new token's K/V (k_new[b], v_new[b]) is stored at position L-1 -- the
 * slot block_table[b][(L-1)/block_size]*block_size + (L-1)%block_size, as
 * pa_kv_cache_write would store it -- and the query attends over all L
 * tokens including it, in one launch.  Results and cache contents are
 * bit-identical to pa_kv_cache_write followed by pa_decode ("Paged 어텐션",
 * Decode 경로: the kernel updates the cache in place; the worked example's
 * new tokens at positions 30, 32, 70).  The new token's page is read only up
 * to the row before it.
 *
 * k_new, v_new: device [num_seqs][num_kv_heads][head_size] of q_dtype,
 *   16-byte aligned.  E4M3 caches store e4m3_satfinite(rne(x / scale)).
 * The block holding position L-1 must already be in the table (an id out of
 *   range is reported as PA_ERR_BAD_BLOCK and nothing is written for it).
 * Everything else as pa_decode (same workspace size).
 * ------------------------------------------------------------------------- */
pa_status pa_decode_append(void* out, const void* q, const void* k_new, const void* v_new, pa_dtype q_dtype,
                           const pa_kv_cache* cache, const int32_t* block_table, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len, int32_t num_heads,
                           float scale, int32_t partition_size, void* workspace, size_t workspace_bytes,
                           int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Shared-prefix ("cascade") decode.  "Как работает paged attention?
 * (детально)" §3.3: sequences of parallel sampling or beam search refer to the
 * same physical blocks for their common prefix (copy-on-write on change); §7:
 * requests with the same prefix reuse its physical blocks (prefix caching);
 * the vLLM paper summary lists parallel sampling and shared prefixes among its
 * decoding scenarios.  The pages give no kernel for it; this entry point
 * computes exactly what pa_decode computes (the same softmax(q K^T scale) V per
 * sequence and head, up to fp32 rounding order) but reads a group's shared
 * blocks once per 8 / (num_heads / num_kv_heads) members: one decode launch
 * attends every member's query to the shared tokens (those members' heads side
 * by side as the eight query rows of one sequence) and each member's own
 * tokens, all in partitions of one work list, and the log-sum-exp merge of
 * pa_decode combines all partitions.
 *
 * cu_groups: device int32 [num_groups+1], 0 = cu_groups[0] <= ... <=
 *   cu_groups[num_groups] = num_seqs; sequences cu_groups[g] .. cu_groups[g+1]-1
 *   form group g (consecutive rows of q, out, block_table and seq_lens).
 * shared_lens: device int32 [num_groups]: group g's first shared_lens[g] tokens
 *   are whole blocks (a multiple of block_size) that every member's block-table
 *   row names identically and every member attends (shared_lens[g] <= each
 *   member's length).  The blocks are read through the group's first row; a
 *   member whose row differs there, or a shared length that breaks these rules,
 *   is reported as PA_ERR_INVALID_ARG in dev_status.
 * max_group_size: the largest group (host bound, >= 1).  max_shared_len: host
 *   bound on shared_lens (a multiple of block_size, <= max_seq_len).
 * workspace: pa_decode_cascade_workspace_size(...) bytes, 16-byte aligned (never
 *   0: every (sequence, head) keeps a prefix and a suffix partial).
 * Supported: the shapes and types of pa_decode (fp16/bf16 caches with q of the
 *   same type, or E4M3 caches; head_size 64 or 128; block sizes 16/32/64;
 *   num_heads / num_kv_heads in {1, 2, 4, 8}); others return PA_ERR_UNSUPPORTED
 *   with nothing launched.  Everything else as pa_decode.
 * ------------------------------------------------------------------------- */
size_t pa_decode_cascade_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t head_size,
                                        int32_t max_seq_len, int32_t block_size, int32_t partition_size);
pa_status pa_decode_cascade(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                            const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                            int32_t num_seqs, int32_t max_seq_len, int32_t num_heads, float scale,
                            const int32_t* cu_groups, const int32_t* shared_lens, int32_t num_groups,
                            int32_t max_group_size, int32_t max_shared_len, int32_t partition_size,
                            void* workspace, size_t workspace_bytes, int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Varlen attention of groups of sequences that share a prefix, the prefix computed
 * once for a group.  (pa_decode_cascade's sharing, "Как работает paged attention?
 * (детально)" §3.3 and §7, for any number of query tokens a sequence: beams and
 * samples that decode, short questions to one document, prompts behind a system
 * prompt.)
 *
 * Computes what pa_prefill_varlen with causal != 0 computes (same arguments, same
 * rounding, up to the order of sums).  Over a group's shared blocks its members' query
 * rows stand together, 128 rows of one KV head's query heads to a tile, so the blocks
 * are read and multiplied once per 128 / (num_heads / num_kv_heads) query tokens of the
 * group instead of once per member; each member's own keys are attended apart, and a
 * merge joins the parts by their log-sum-exp.
 *
 * cu_groups, shared_lens, num_groups, max_group_size, max_shared_len: as in
 *   pa_decode_cascade.  Every query of a member comes after the shared tokens:
 *   shared_lens[g] <= Lk - Lq of each member with queries.  A shared length that breaks
 *   this or is no whole number of blocks, a member whose row differs over the
 *   shared blocks, and bounds that do not hold are reported as PA_ERR_INVALID_ARG; the
 *   group's rows are then unspecified.
 *   (A differing row is reported where it matters: in batches whose queries fill tiles of
 *   their own every sequence reads its own row.)  With max_seqlen_q 1 and total_q >=
 *   num_seqs, sequences without a query come last (otherwise possibly PA_ERR_INVALID_ARG).
 * total_q: query rows of q and out; cu_seq_lens_q[num_seqs] <= total_q (otherwise
 *   reported, and sequences past it are left out).  Rows behind the last sequence are
 *   left as they are.
 * workspace: pa_varlen_cascade_workspace_size(...) bytes with the same arguments,
 *   16-byte aligned.
 * scale > 0.  A value that some query of a sequence sees must be finite for the
 *   sequence's other queries, and a shared one for the group's (pa_prefill_varlen's
 *   rule); what other groups, and other members' own keys, hold takes no part.
 * Supported: as pa_prefill_varlen (head_size 128, 16-bit caches); num_seqs + num_groups
 *   <= 6144.
 * ------------------------------------------------------------------------- */
size_t pa_varlen_cascade_workspace_size(int32_t num_seqs, int64_t total_q, int32_t num_heads, int32_t num_kv_heads,
                                        int32_t head_size, int32_t max_seqlen_q, int32_t max_seqlen_k,
                                        int32_t max_shared_len, int32_t block_size);
pa_status pa_varlen_cascade(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                            const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* cu_seq_lens_q,
                            const int32_t* cu_seq_lens_k, int32_t num_seqs, int64_t total_q, int32_t max_seqlen_q,
                            int32_t max_seqlen_k, int32_t num_heads, float scale, const int32_t* cu_groups,
                            const int32_t* shared_lens, int32_t num_groups, int32_t max_group_size,
                            int32_t max_shared_len, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                            pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Beam search: selection.  ("Как работает paged attention? (детально)" 3.3 and the
 * vLLM paper summary name beam search among what shares blocks; its step is a selection,
 * then a reordering of the beams' states.)
 *
 * For the rows r = cu_beams[b] .. cu_beams[b+1]-1 (the beams of request b) with scores
 * c_r (sums of log-probabilities so far) and logits x_ri over the allowed tokens A_r:
 *     s(r, i) = c_r + (x_ri - log sum_{j in A_r} exp(x_rj)),   i in A_r
 * The request's num_select largest, in descending order, ties to the lower row, then
 * the lower token: scores_out, rows_out (r, a row of logits), tokens_out (i), each device
 * [num_requests][num_select]; past the candidates there are -inf, -1, -1.  s is computed
 * to 48 bits (its logarithm's sum to about 2^-27) and ordered so; scores_out is it rounded
 * once.  Scores below binary32's range are alike.
 *
 * logits: device, [num_rows][vocab] of dtype (F16, BF16 or F32), rows row_stride >=
 *   vocab elements apart, any alignment that the type has (16-byte aligned rows go
 *   faster).  A logit of -inf is no candidate.  An allowed logit that is NaN or +inf is
 *   reported as PA_ERR_INVALID_ARG and its row offers nothing.
 * scores: device float [num_rows].  -inf: the row offers nothing (a beam that a request
 *   does not have yet).  NaN or +inf is reported, the row offers nothing.
 * cu_beams: device int32 [num_requests + 1], non-decreasing, within 0 .. num_rows (a request
 *   that breaks this is reported and gets no candidates).
 * allowed: device bit masks [num_rows][ceil(vocab/32)] uint32, bit i % 32 of word i / 32
 *   set where token i is allowed, rows allowed_stride words apart; NULL: every
 *   token.  Logits that are not allowed may hold anything.
 * ended: device uint8 [num_rows], nullable: a row != 0 has one candidate, (r, end_token)
 *   with s = c_r; its logits are not read.
 * workspace: pa_beam_select_workspace_size(...) bytes, 16-byte aligned.
 * Supported: num_select <= 64, vocab <= 2^23.
 * ------------------------------------------------------------------------- */
size_t pa_beam_select_workspace_size(int32_t num_rows, int32_t vocab, int32_t num_select);
pa_status pa_beam_select(float* scores_out, int32_t* rows_out, int32_t* tokens_out, const void* logits,
                         pa_dtype dtype, int64_t row_stride, int32_t vocab, int32_t num_rows, const float* scores,
                         const int32_t* cu_beams, int32_t num_requests, const uint32_t* allowed,
                         int64_t allowed_stride, const uint8_t* ended, int32_t end_token, int32_t num_select,
                         void* workspace, size_t workspace_bytes, int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Beam search: reordering ("Как работает paged attention?" 3.3: beams refer to the same
 * blocks; a shared block is copied before a sequence writes into it).
 *
 * New row i goes on from row p = parents[i] of the old tables with one more token, at
 * position L = seq_lens[p]:
 *   block_table_out[i] is block_table[p]'s first ceil(L / block_size) entries, -1 behind;
 *   where L % block_size == 0, entry L / block_size is spare_blocks[i];
 *   otherwise the first row (lowest i) with this parent keeps the parent's partly
 *   filled block, and each other one has spare_blocks[i] there, to which the block's
 *   first L % block_size token rows are copied (all KV heads, K and V, every layer);
 *   seq_lens_out[i] = L + 1, slot_mapping_out[i] is position L's slot (for
 *   pa_kv_cache_write of the new token), spare_used_out[i] tells whether
 *   spare_blocks[i] went into the table.
 * parents[i] < 0: an empty row (-1 everywhere, length 0, slot -1).
 * So the partly filled block must be its row's alone (which these rules keep up: a
 *   beam's own last block is never shared); whole blocks are shared freely.
 *
 * caches: host array of num_layers caches of one shape and type, which the tables serve.
 * parents, spare_blocks, seq_lens_out, spare_used_out: device int32 [num_rows];
 * slot_mapping_out: device int64 [num_rows]; block_table, block_table_out: device int32
 * [num_rows_in], [num_rows] rows of max_blocks_per_seq; seq_lens: device int32
 * [num_rows_in].  The old tables and the new are different memory.
 * Reported in *dev_status: a parent past num_rows_in or a length outside 0 ..
 *   max_blocks_per_seq * block_size - 1 (PA_ERR_INVALID_ARG; the row is empty), a block
 *   that position L needs outside the cache (PA_ERR_BAD_BLOCK; its entry and slot are -1,
 *   nothing is copied).
 * pa_pool_reserve / pa_pool_reorder / pa_pool_unreserve are the host's side: spare
 *   blocks are reserved ahead, the device goes on without waiting for the host, and the pool
 *   follows by the same rule once the parents are known there.
 * ------------------------------------------------------------------------- */
pa_status pa_beam_reorder(const pa_kv_cache* caches, int32_t num_layers, const int32_t* parents, int32_t num_rows,
                          const int32_t* block_table, int32_t num_rows_in, int32_t max_blocks_per_seq,
                          const int32_t* seq_lens, const int32_t* spare_blocks, int32_t* block_table_out,
                          int32_t* seq_lens_out, int64_t* slot_mapping_out, int32_t* spare_used_out,
                          int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Mixed batch dispatcher: a varlen batch (as pa_prefill_varlen) whose
 * trailing sequences have one query token each is split -- the leading
 * sequences go to the varlen tensor-core kernel, the trailing one-token run
 * to the decode kernel, which reads each length as cu_seq_lens_k[b+1] -
 * cu_seq_lens_k[b] ("Paged 어텐션": the decode path is the faster one for
 * single-query sequences, the varlen path takes the prefills).  A single
 * query sees all of its keys, causal or not, so the split computes the same
 * attention.
 *
 * host_cu_seq_lens_q: host int32 [num_seqs+1], a copy of cu_seq_lens_q (the
 *   split is decided on the host; nothing is read back from the device).
 * workspace: device scratch of pa_varlen_mixed_workspace_size(...) bytes,
 *   16-byte aligned (NULL if that is 0), for the decode kernel's partitions.
 * Everything else as pa_prefill_varlen; head_size 64 is only served when
 * every sequence is a one-token sequence.
 * ------------------------------------------------------------------------- */
size_t pa_varlen_mixed_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t head_size,
                                      int32_t max_seqlen_k, int32_t block_size);
pa_status pa_varlen_mixed(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                          const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* cu_seq_lens_q,
                          const int32_t* cu_seq_lens_k, const int32_t* host_cu_seq_lens_q, int32_t num_seqs,
                          int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t num_heads, float scale,
                          int32_t causal, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                          pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Varlen attention over packed K/V: "Paged 어텐션", Varlen 경로 -- the batch's
 * keys and values are contiguous tensors [Σk][num_kv_heads][head_size]
 * indexed by cu_seq_lens_k (no cache, no block table), queries as in
 * pa_prefill_varlen.  Same arithmetic and causal alignment as
 * pa_prefill_varlen (bottom-right; rows without a visible key give 0).
 *
 * k, v: device, total_k rows of num_kv_heads*head_size elements of dtype (F16
 *   or BF16, the same as q and out), 16-byte aligned; may be NULL when
 *   total_k == 0.  cu_seq_lens_k[b+1] must be <= total_k, otherwise
 *   PA_ERR_INVALID_ARG is reported in *dev_status and that sequence's rows are
 *   unspecified.
 * Supported: head_size 128; num_heads / num_kv_heads in {1, 2, 4, 8};
 *   num_seqs <= 6144.
 * ------------------------------------------------------------------------- */
pa_status pa_prefill_varlen_packed(void* out, const void* q, const void* k, const void* v, pa_dtype dtype,
                                   const int32_t* cu_seq_lens_q, const int32_t* cu_seq_lens_k, int32_t num_seqs,
                                   int32_t max_seqlen_q, int32_t max_seqlen_k, int64_t total_k, int32_t num_heads,
                                   int32_t num_kv_heads, int32_t head_size, float scale, int32_t causal,
                                   int32_t* dev_status, pa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Slots of new tokens from a block table (host arrays): "Как работает paged
 * attention?" 4.1 (logical block = pos / block_size, offset pos % block_size);
 * vLLM paper summary §3.  For token i of sequence seq_idx[i] at position
 * pos[i]: slot = block_table[seq][pos / block_size] * block_size
 * + pos % block_size.  An entry < 0 (unallocated) or a position past the row
 * gives slot -1.  block_table: host int32 [num_seqs][max_blocks]; seq_idx:
 * host int32 [n] in [0, num_seqs); pos: host int64 [n] >= 0; slots_out: host
 * int64 [n].  Returns PA_ERR_INVALID_ARG for a bad sequence index or position.
 * ------------------------------------------------------------------------- */
pa_status pa_slot_mapping(const int32_t* block_table, int32_t num_seqs, int32_t max_blocks,
                          int32_t block_size, const int32_t* seq_idx, const int64_t* pos, int64_t n,
                          int64_t* slots_out);

/* ---------------------------------------------------------------------------
 * Host block pool ("Как работает paged attention?" 3.2 BlockManager, 3.3,
 * 4.1, 4.2; vLLM paper summary §2-4).  Host memory only.
 *
 * The free list is FIFO: allocation takes its head, a freed block goes to
 * its tail.  free_order (nullable, a permutation of 0..num_blocks-1) sets the
 * initial order; NULL means 0, 1, 2, ...
 * pa_pool_append(seq, n): positions len .. len+n-1 get slots; a position in a
 *   logical block not yet mapped gets a new block (reference count 1).  If the
 *   last block is shared (reference count > 1) and not full, it is first
 *   replaced by a private block taken from the free list: the (old, new) pair
 *   is written to cow_pairs_out (room for 2 int32) and *n_cow_out = 1; the
 *   caller copies it with pa_copy_blocks before writing the slots.  If the
 *   free list cannot supply every block the append needs, nothing changes and
 *   PA_ERR_OOM is returned.  slots_out: host int64 [n].
 * pa_pool_fork(parent, child): the child shares all of the parent's blocks
 *   (each reference count + 1) and its length.
 * pa_pool_free_seq: each block's reference count - 1, in logical order; a
 *   block reaching 0 goes to the tail of the free list.
 * pa_pool_block_table: host int32 [n][max_blocks] rows, -1 padded, and host
 *   int32 lens_out[n] (nullable).  A sequence with more blocks than
 *   max_blocks gives PA_ERR_INVALID_ARG.
 * pa_pool_release_window(seq, window, num_sinks): gives back the blocks that no
 *   query of the sequence from position len - 1 on sees with that window and
 *   that many sinks (pa_decode_window, pa_prefill_varlen_window): those wholly
 *   past the first num_sinks positions and wholly before position len - window.
 *   Call it once the queries of the tokens appended last are the only ones left
 *   to attend (a prefill's chunk of n tokens: with window + n - 1).  Each block's
 *   reference count - 1, in logical order, a block reaching 0 goes to the tail of the
 *   free list; the sequence's table holds -1 there from then on (a fork takes the
 *   holes over; pa_decode and the other unwindowed calls report them as
 *   PA_ERR_BAD_BLOCK).  *n_released_out (nullable): how many.  window >= 1,
 *   num_sinks >= 0.
 * pa_pool_reserve(n): the next n blocks of the free list (reference count 1) become the
 *   caller's own, of no sequence, until pa_pool_reorder gives them to one or
 *   pa_pool_unreserve returns them (to the tail, in the order given; an id that is not
 *   reserved, or twice, gives PA_ERR_INVALID_ARG and changes nothing).
 * pa_pool_reorder: what pa_beam_reorder does, in the pool.  The sequences new_ids[i] take
 *   the place of the sequences old_ids (all of them end): new_ids[i] goes on from old_ids
 *   [parents[i]] with one token more, by pa_beam_reorder's rules with spare_blocks
 *   (reserved ids; those used stop being reserved, the others stay the caller's).
 *   parents[i] < 0: an empty sequence.  slots_out, spare_used_out: host [num_new],
 *   nullable.  Ids are distinct among the old and among the new; a new id is an old one or
 *   unknown.  A parent whose partly filled block another sequence holds too, a spare
 *   that is needed and not reserved (or named twice), or bad ids give PA_ERR_INVALID_ARG
 *   and change nothing.
 * Sequence ids are arbitrary int64 keys; an unknown id gives
 * PA_ERR_INVALID_ARG.
 * ------------------------------------------------------------------------- */
pa_status pa_pool_create(int64_t num_blocks, int32_t block_size, const int32_t* free_order,
                         void** pool_out);
void pa_pool_destroy(void* pool);
pa_status pa_pool_add_seq(void* pool, int64_t seq_id);
pa_status pa_pool_append(void* pool, int64_t seq_id, int32_t n_tokens, int64_t* slots_out,
                         int32_t* cow_pairs_out, int32_t* n_cow_out);
pa_status pa_pool_fork(void* pool, int64_t parent, int64_t child);
pa_status pa_pool_free_seq(void* pool, int64_t seq_id);
pa_status pa_pool_release_window(void* pool, int64_t seq_id, int32_t window, int32_t num_sinks,
                                 int32_t* n_released_out);
pa_status pa_pool_reserve(void* pool, int32_t n, int32_t* blocks_out);
pa_status pa_pool_unreserve(void* pool, const int32_t* blocks, int32_t n);
pa_status pa_pool_reorder(void* pool, const int64_t* old_ids, int32_t num_old, const int64_t* new_ids, int32_t num_new,
                          const int32_t* parents, const int32_t* spare_blocks, int64_t* slots_out,
                          int32_t* spare_used_out);
pa_status pa_pool_block_table(void* pool, const int64_t* seq_ids, int32_t n, int32_t max_blocks,
                              int32_t* table_out, int32_t* lens_out);
int64_t pa_pool_num_free(void* pool);
int32_t pa_pool_ref_count(void* pool, int64_t block);
int32_t pa_pool_seq_len(void* pool, int64_t seq_id);

/* ---------------------------------------------------------------------------
 * Test hooks for the wait timeouts.  (Not on the pages: every wait of
 * the library's kernels is bounded, so that a stalled copy ends in an error
 * status instead of a hung GPU.)
 *
 * Same arguments and host checks as pa_decode, but the launched decode's
 * producer warp issues no copy at all: no page and no query ever lands, so
 * every consumer wait runs out after the library's wait limit (2 s) with
 * nothing in flight, PA_ERR_TIMEOUT (5) is written to *dev_status, and the
 * kernel returns.  The output and workspace contents are unspecified
 * afterwards (within their stated sizes); the device stays usable.  For the
 * library's own tests; a serving path has no use for it.
 * pa_decode_window_test_wait_timeout: the same of pa_decode_window, with its arguments.
 * pa_varlen_cascade_test_wait_timeout: the same of pa_varlen_cascade's tensor-core kernel.
 * pa_prefill_test_wait_timeout: the same of pa_prefill_varlen_window (window > 0)
 * or of the causal pa_prefill_varlen (window 0): its loader warps issue no copy.
 * ------------------------------------------------------------------------- */
pa_status pa_decode_test_wait_timeout(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                                      const int32_t* block_table, int32_t max_blocks_per_seq,
                                      const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                                      int32_t num_heads, float scale, int32_t partition_size, void* workspace,
                                      size_t workspace_bytes, int32_t* dev_status, pa_stream_t stream);
pa_status pa_decode_window_test_wait_timeout(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                                             const int32_t* block_table, int32_t max_blocks_per_seq,
                                             const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                                             int32_t num_heads, float scale, int32_t window, int32_t num_sinks,
                                             int32_t partition_size, void* workspace, size_t workspace_bytes,
                                             int32_t* dev_status, pa_stream_t stream);
pa_status pa_prefill_test_wait_timeout(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                                       const int32_t* block_table, int32_t max_blocks_per_seq,
                                       const int32_t* cu_seq_lens_q, const int32_t* cu_seq_lens_k, int32_t num_seqs,
                                       int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t num_heads, float scale,
                                       int32_t window, int32_t num_sinks, int32_t* dev_status, pa_stream_t stream);

pa_status pa_varlen_cascade_test_wait_timeout(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                            const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* cu_seq_lens_q,
                            const int32_t* cu_seq_lens_k, int32_t num_seqs, int64_t total_q, int32_t max_seqlen_q,
                            int32_t max_seqlen_k, int32_t num_heads, float scale, const int32_t* cu_groups,
                            const int32_t* shared_lens, int32_t num_groups, int32_t max_group_size,
                            int32_t max_shared_len, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                            pa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_KV_H */
