/*
 * pa.h -- C ABI of the GB300 (sm_103a) paged-attention library.
 *
 * Paged attention over a block-tabled KV cache, as described on the
 * TensorSharp "Mistral 3" model page, section 11 "Batched / paged forward
 * (continuous batching)", and on the mistral.rs part of the "pure Rust
 * engines" page (paged attention, KV-cache manager, prefix cache and
 * scheduler sections).  Four operations:
 *
 *   pa_reshape_and_cache  write fresh K/V into cache slots through a slot map
 *   pa_decode             one query token per sequence, split-K over the
 *                         context, log-sum-exp reduce
 *   pa_prefill_chunk      a chunk of query tokens per sequence: causal inside
 *                         the chunk, full over the cached prefix
 *   pa_copy_blocks        whole-block copies for prefix-cache reuse
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every tensor argument is a pointer to DEVICE memory owned by the caller,
 *    dense row-major, 16-byte aligned.  The library allocates nothing, keeps
 *    no state between calls and never synchronises the device.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and runs asynchronously.
 *  - The return value is PA_OK (0) or a negative PA_ERR_* code.  Argument
 *    errors are detected on the host before anything is launched.  A failed
 *    launch returns PA_ERR_CUDA.
 *  - The first call of an attention or pa_tables_* entry point on a device raises its kernels' shared-memory limit
 *    (cudaFuncSetAttribute) and may load the library's device code into the
 *    current context; make that first call outside stream capture.  Calls
 *    from several host threads are safe (per-device setup is atomic).
 *  - Values that only the device can see (slot numbers, block ids, context
 *    lengths) are range-checked inside the kernels: an out-of-range value is
 *    never dereferenced and, if `status` is not NULL, the matching PA_DEVERR_*
 *    bit is OR-ed into the device int32 `*status`.  The offending token / copy
 *    pair is skipped.  The keys of an offending block are left out of the
 *    softmax by pa_decode_window, by pa_cross_attention for F32 caches and
 *    where it keeps its weights as pa_decode_window does; elsewhere they and
 *    their values count as zeros.  The caller clears *status and reads it
 *    after synchronising.
 *
 * Layouts (S sequences, Hq query heads, Hkv kv heads, D head dim, bs block
 * size, NB blocks in the pool; G = Hq / Hkv; query head h reads kv head h / G)
 *  - key_cache, value_cache: [NB][bs][Hkv][D], the flat
 *    [numBlocks * blockSize * numKvHeads * headDim] per-layer buffer of the
 *    TensorSharp page, section 11.  Token slot `slot` is row slot of the
 *    [NB * bs][Hkv][D] view: block slot / bs, offset slot % bs.
 *  - block_tables: int32 [S][max_blocks_per_seq]; logical token j of sequence
 *    s lives in physical block block_tables[s][j / bs] at offset j % bs.
 *    Entries past ceil(context_lens[s] / bs) are never read.
 *  - context_lens: int32 [S]; the number of keys the sequence's last query row
 *    sees, the freshly written token(s) included.
 *
 * Supported shapes: dtype F32, F16 or BF16 (query and cache share it); D in
 * {64, 128}; bs in {8, 16, 32} (the mistral.rs page's allowed block sizes);
 * Hq a multiple of Hkv with G = Hq / Hkv in {1, 2, 4, 8}; Hkv in {1, 2, 4} or
 * a multiple of 8; num_blocks * block_size < 2^31.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t; declared here so the header needs no CUDA headers. */
typedef struct CUstream_st *pa_stream_t;

typedef enum { PA_F32 = 0, PA_F16 = 1, PA_BF16 = 2 } pa_dtype;

enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = -1, /* null / misaligned pointer, negative size, bad dtype */
    PA_ERR_UNSUPPORTED = -2, /* head_dim, block_size or head grouping not built */
    PA_ERR_WORKSPACE = -3,   /* workspace missing or smaller than required */
    PA_ERR_CUDA = -4,        /* a kernel launch failed (cudaGetLastError) */
    PA_ERR_NO_BLOCKS = -5    /* KV-cache manager: not enough free blocks (nothing changed) */
};

/* Bits OR-ed into the optional device-side `*status` word. */
enum {
    PA_DEVERR_SLOT = 1,      /* slot_mapping entry >= num_blocks * block_size */
    PA_DEVERR_BLOCK_ID = 2,  /* block table / block mapping id outside [0, num_blocks) */
    PA_DEVERR_CONTEXT = 4,   /* context length < 0, > max_context_len, or beyond the block table */
    PA_DEVERR_QUERY = 8,     /* query_start_loc not monotone, or a chunk longer than its context */
    PA_DEVERR_TIMEOUT = 16,  /* a bounded wait inside a kernel gave up (internal error; the
                                kernel returned instead of hanging) */
    PA_DEVERR_AXIS = 32,     /* pa_rope_axes.pair_axis entry outside [0, num_axes) */
    PA_DEVERR_FREE_LIST = 64 /* pa_tables_*: the free list ran out, its count lies outside it, or a
                                returned block does not fit it */
};

/*
 * pa_reshape_and_cache -- write fresh keys and values into their cache slots.
 * TensorSharp "Mistral 3" page, section 11 (K/V scatter via slotMapping to
 * blockId * blockSize + offset; no per-sequence extract / inject).
 *
 *   key, value     [num_tokens][num_kv_heads][head_dim], kv_dtype (read)
 *   key_cache,
 *   value_cache    [num_blocks][block_size][num_kv_heads][head_dim] (written)
 *   slot_mapping   int64 [num_tokens]; slot < 0 skips the token (padding)
 *
 * Each written row is a bit copy.  Tokens must map to distinct slots (two
 * tokens writing one slot race).  num_tokens == 0 is a no-op.
 */
int pa_reshape_and_cache(const void *key, const void *value, void *key_cache, void *value_cache,
                         const int64_t *slot_mapping, int num_tokens, int num_kv_heads,
                         int head_dim, int block_size, int num_blocks, pa_dtype kv_dtype,
                         int32_t *status, pa_stream_t stream);

/*
 * pa_decode_workspace_size -- bytes of device workspace pa_decode needs for
 * these sizes on the current device (0 only when num_seqs == 0).  The value
 * depends on its arguments and on the device's SM count (the split of the
 * contexts is balanced over one CTA per SM); on a machine without a visible
 * device it returns an upper bound.  Returns 0 for arguments pa_decode would
 * reject.
 */
size_t pa_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                int max_context_len);

/*
 * pa_decode -- decode attention: one query token per sequence against every
 * cached key of that sequence, gathered through its block table.
 * TensorSharp "Mistral 3" page, section 11 (per-sequence paged attention over
 * the paged K/V buffer) and sections 3 / 4.1 (standard causal GQA attention,
 * Q scaled by 1/sqrt(headDim)).
 *
 *   out            [num_seqs][num_heads][head_dim], out_dtype (written)
 *   query          [num_seqs][num_heads][head_dim], kv_dtype
 *   key_cache,
 *   value_cache    [num_blocks][block_size][num_kv_heads][head_dim], kv_dtype
 *   block_tables   int32 [num_seqs][max_blocks_per_seq]
 *   context_lens   int32 [num_seqs]; max_context_len >= every entry (host bound
 *                  used to size the split of the context)
 *   scale          softmax scale applied to q.k (normally 1/sqrt(head_dim))
 *   workspace      device scratch of >= pa_decode_workspace_size(...) bytes,
 *                  16-byte aligned, owned by the caller; it needs no
 *                  initialisation (each call marks what it writes with its own
 *                  64-bit tag), its contents are clobbered, and two calls in
 *                  flight must not share it
 *
 * A call made while `stream` is being captured into a CUDA graph is replayable: the
 * merge of the split context then waits for the whole first pass instead of the
 * per-call tags (a replay repeats the captured tag), a few microseconds slower.
 *
 *   out[s][h] = sum_j softmax_j(scale * q[s][h] . k_j) v_j over j < context_lens[s];
 *   a sequence with context length 0 gets an all-zero row.
 * Accumulation is fp32; the result does not depend on the split.
 * With eight query heads per kv head, an fp16/bf16 cache and num_seqs * num_kv_heads
 * >= 0.4 x the SM count, the rows run on the tensor cores instead (the chunked-prefill
 * kernel with one-token chunks): q.k and p.v in fp32 accumulators, the softmax weights
 * rounded to the cache's type before p.v (as in pa_prefill_chunk), each (sequence, kv
 * head) in one fixed key order, so that a row does not depend on the rest of the batch
 * while the call stays on this path; the workspace is then not touched.  A row computed
 * on the two paths (a small batch and a large one) agrees within the attention tolerance,
 * not bit for bit.  One to four query heads per kv head always take the split path.
 */
int pa_decode(void *out, pa_dtype out_dtype, const void *query, const void *key_cache,
              const void *value_cache, const int32_t *block_tables, int max_blocks_per_seq,
              const int32_t *context_lens, int max_context_len, int num_seqs, int num_heads,
              int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
              pa_dtype kv_dtype, void *workspace, size_t workspace_bytes, int32_t *status,
              pa_stream_t stream);

/*
 * pa_decode_write -- pa_reshape_and_cache of one new token per sequence followed by
 * pa_decode, in one launch (the decode step of a serving loop: the TensorSharp "Mistral 3"
 * page, section 11, writes the step's K/V through slotMapping, then attends).
 *
 *   key, value     [num_seqs][num_kv_heads][head_dim], kv_dtype (device): token s is the
 *                  newest token of sequence s
 *   slot_mapping   int64 [num_seqs]: its cache slot (blockId * block_size + offset); a
 *                  negative slot writes nothing, a slot past the pool is reported
 *                  (PA_DEVERR_SLOT) and not written
 *   key_cache,
 *   value_cache    written at those slots, then read as by pa_decode
 *   (every other argument as for pa_decode)
 *
 * Precondition (the decode step of any paged KV manager): slot_mapping[s] is the slot that
 * block_tables[s] gives position context_lens[s] - 1, and no other sequence of the call
 * reads that slot (a block being appended to is never shared).  Then out and both pools
 * equal those of pa_reshape_and_cache(key, value, ..., slot_mapping, num_seqs, ...) and
 * pa_decode(...) on the same stream, bit for bit.  Otherwise the pools are written as
 * stated and out is unspecified.  The launch that streams a sequence's last keys stores
 * the token and uses it from the same copy, so no kernel boundary separates the two
 * (where pa_decode runs its rows on the tensor cores, the write is a launch of its own
 * in front of them).
 */
int pa_decode_write(void *out, pa_dtype out_dtype, const void *query, const void *key,
                    const void *value, const int64_t *slot_mapping, void *key_cache,
                    void *value_cache, const int32_t *block_tables, int max_blocks_per_seq,
                    const int32_t *context_lens, int max_context_len, int num_seqs, int num_heads,
                    int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                    pa_dtype kv_dtype, void *workspace, size_t workspace_bytes, int32_t *status,
                    pa_stream_t stream);

/*
 * pa_decode_noalloc -- pa_decode for callers that cannot allocate device
 * memory: plugin hosts and serving runtimes that own all device memory and hand
 * kernels only their tensors, hot paths where a cudaMalloc could synchronise
 * the device, and language bindings without a device allocator.  The pages
 * describe no such call; it exists only for these callers.
 *
 * Same arguments, results and error behaviour as pa_decode, without the
 * workspace: the scratch lives in one static device array of
 * PA_DECODE_NOALLOC_SCRATCH_BYTES inside the library (held by every GPU that
 * loads the library until the process exits).  A problem whose scratch
 * (pa_decode_workspace_size) exceeds it returns PA_ERR_WORKSPACE before
 * anything runs; with 152 SMs, Hq = 32, Hkv = 8 and D = 128 that allows about 350
 * sequences.  Nothing is allocated and nothing needs clearing between calls.
 *
 * Every call looks up the array's device address in the current context
 * (cudaGetSymbolAddress), so the address never goes stale across device resets
 * or contexts.  The first call in a context loads the library's device code
 * there and sets up the decode kernels: make that first call before any stream
 * capture.  All calls on a device share the one array: two calls whose kernels overlap
 * on the GPU (different streams, no ordering between them) race and corrupt
 * each other's results.
 */
#define PA_DECODE_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
int pa_decode_noalloc(void *out, pa_dtype out_dtype, const void *query, const void *key_cache,
                      const void *value_cache, const int32_t *block_tables, int max_blocks_per_seq,
                      const int32_t *context_lens, int max_context_len, int num_seqs, int num_heads,
                      int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                      pa_dtype kv_dtype, int32_t *status, pa_stream_t stream);

/*
 * pa_prefill_chunk -- chunked-prefill attention.  Sequence s owns the packed
 * query rows query_start_loc[s] .. query_start_loc[s+1]-1 (Lq_s rows, the
 * newest tokens of the sequence, whose K/V are already in the cache).  Row i
 * sits at absolute position context_lens[s] - Lq_s + i and attends keys
 * 0 .. that position: full attention over the cached prefix, causal inside
 * the chunk.  mistral.rs page, scheduling section (prompts chunked under a
 * token budget of 4096, 512 per chunk); TensorSharp page, section 11.
 *
 *   out              [num_tokens][num_heads][head_dim], out_dtype (written)
 *   query            [num_tokens][num_heads][head_dim], kv_dtype (F16 or BF16)
 *   query_start_loc  int32 [num_seqs + 1], non-decreasing, [0] = 0,
 *                    [num_seqs] = num_tokens
 *   max_query_len    >= every Lq_s (host bound used to size the grid)
 *   other arguments  as for pa_decode
 *
 * Tensor-core MMA with fp32 accumulation; the softmax weights are rounded to
 * the input dtype before the P.V product.
 */
int pa_prefill_chunk(void *out, pa_dtype out_dtype, const void *query,
                     const int32_t *query_start_loc, int num_tokens, int max_query_len,
                     const void *key_cache, const void *value_cache, const int32_t *block_tables,
                     int max_blocks_per_seq, const int32_t *context_lens, int max_context_len,
                     int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                     int num_blocks, float scale, pa_dtype kv_dtype, int32_t *status,
                     pa_stream_t stream);

/*
 * pa_copy_blocks -- copy whole cache blocks, K and V, for prefix-cache reuse
 * (mistral.rs page, block-hash prefix cache: full blocks are shared by
 * content; a copy gives a sequence its own writable copy of a shared block).
 *
 *   block_mapping  int64 [num_pairs][2] = (src, dst) block ids
 *
 * Destinations must be distinct and must not appear as sources (then the
 * result equals copying the pairs one after another); otherwise the result
 * is undefined.  num_pairs == 0 is a no-op.
 */
int pa_copy_blocks(void *key_cache, void *value_cache, const int64_t *block_mapping, int num_pairs,
                   int num_kv_heads, int head_dim, int block_size, int num_blocks,
                   pa_dtype kv_dtype, int32_t *status, pa_stream_t stream);

/*
 * Rotary position embedding fused into the cache write and the decode query load
 * (TensorSharp "Mistral 3" page, section 3 "Forward graph" and section 4.2 "RoPE - GPT-J
 * style with YaRN": RoPE rotates Q and K with the GPT-J pairing -- adjacent elements
 * (x[2i], x[2i+1]) rotate together -- at each token's absolute position, with a frequency
 * table built once at load time (YaRN-corrected when the model asks for it); Q is then
 * scaled by 1 + beta * log(1 + floor(pos / origCtx)) when origCtx > 0).
 *
 * Pair i (i < rope_dim / 2) of a row at position pos is rotated by the angle
 * pos * freqs[i]:  (x, y) -> (x cos - y sin, x sin + y cos).  The angle is formed exactly
 * (as a sum of two floats) and reduced by whole turns in fp32 (within 2.4e-7 of the exact
 * angle less those turns for |pos| < 2^24; positions beyond lose that bound), its sine and cosine
 * taken in fp32 (in all within 6e-7 for |pos| < 2^17 and freqs up to 1, 9e-7 for |pos| < 2^24,
 * as measured), the rotation done in fp32.  Elements past
 * rope_dim are not rotated.  The 1/sqrt(head_dim) factor stays the attention's `scale`
 * argument.
 */
typedef struct {
    const float *freqs;   /* device, [rope_dim / 2]: angular frequency of pair i (pa_rope_yarn_freqs) */
    int rope_dim;         /* even, 2 .. head_dim */
    float q_scale_beta;   /* beta of the position-dependent query scale */
    int q_scale_orig_ctx; /* origCtx of the query scale; 0 turns the scale off */
} pa_rope;

/*
 * pa_rope_yarn_freqs -- host: the frequency table, freqs[i] = base^(-2i / rope_dim), then
 * YaRN-corrected when yarn_scale != 1 and orig_ctx > 0 (section 4.2): with r = orig_ctx /
 * (2 pi / f), the number of turns pair i makes over the original context, a pair with
 * r > beta_fast keeps f (extrapolation), one with r < beta_slow takes f / yarn_scale
 * (interpolation), and in between f mixes linearly in r: f * (1 - g) + f / yarn_scale * g
 * with g = (beta_fast - r) / (beta_fast - beta_slow).  Computed in double, stored fp32.
 * freqs: host array of rope_dim / 2 floats.
 */
int pa_rope_yarn_freqs(float *freqs, int rope_dim, float base, float yarn_scale, int orig_ctx,
                       float beta_fast, float beta_slow);

/*
 * pa_reshape_and_cache_rope -- pa_reshape_and_cache with K rotated on the way in:
 * token t's key row is rotated at position positions[t] (int32 [num_tokens], device)
 * before it is written; values are copied as they are.  Same layouts, skip rule and errors
 * as pa_reshape_and_cache, plus PA_ERR_INVALID_ARG for a missing rope/positions/freqs, an
 * odd rope_dim or one outside 2..head_dim.
 */
int pa_reshape_and_cache_rope(const void *key, const void *value, void *key_cache, void *value_cache,
                              const int64_t *slot_mapping, const int32_t *positions, int num_tokens,
                              int num_kv_heads, int head_dim, int block_size, int num_blocks,
                              pa_dtype kv_dtype, const pa_rope *rope, int32_t *status,
                              pa_stream_t stream);

/*
 * pa_decode_rope -- pa_decode with the query rotated and scaled as it is loaded: the query
 * of sequence s sits at position context_lens[s] - 1 (the newest token), is rotated there
 * and, when q_scale_orig_ctx > 0, multiplied by 1 + q_scale_beta * log(1 + floor(pos /
 * q_scale_orig_ctx)); `query` holds the unrotated query.  Keys must already be rotated in
 * the cache (pa_reshape_and_cache_rope).  Arguments otherwise as pa_decode.
 */
int pa_decode_rope(void *out, pa_dtype out_dtype, const void *query, const void *key_cache,
                   const void *value_cache, const int32_t *block_tables, int max_blocks_per_seq,
                   const int32_t *context_lens, int max_context_len, int num_seqs, int num_heads,
                   int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                   pa_dtype kv_dtype, const pa_rope *rope, void *workspace, size_t workspace_bytes,
                   int32_t *status, pa_stream_t stream);

/*
 * Sliding-window attention with sinks.  A query at position p (its sequence's keys are at
 * positions 0, 1, ...) sees the keys j <= p with j > p - window (the newest `window` keys,
 * its own included) or j < num_sinks (the first tokens of the sequence, which stay visible).
 * window >= context length makes it plain causal attention; num_sinks = 0 leaves the bare
 * window.  Layouts, checks, errors and asynchrony are those of pa_decode / pa_prefill_chunk,
 * with two differences:
 *  - a block-table entry is read only if its block holds a key that some query row of the
 *    sequence sees: the blocks behind the window may have been freed, their entries hold
 *    anything (-1, say).  What the cache holds in slots that no row of the sequence sees is
 *    never used, not even NaN;
 *  - there is no workspace: the pieces of a split context are merged inside the launch.  A
 *    call may be captured into a CUDA graph after one eager call with its types, head
 *    dimension and head grouping on the device.
 * window < 1, num_sinks < 0 or scale <= 0 returns PA_ERR_INVALID_ARG.
 */

/*
 * pa_decode_window -- decode attention (one query token per sequence, at position
 * context_lens[s] - 1) over the window and the sinks.  Arguments as for pa_decode; F32, F16
 * and BF16 caches.  A sequence with context length 0 gets an all-zero row; a negative
 * context, or one past max_context_len or the block table, is reported and clamped, as in
 * pa_decode.  Sums are fp32.  The softmax weights are fp32 for F32 caches; for F16 and BF16 they
 * enter the products as two parts of the cache's type: within 2^-16 (BF16) or 2^-22 (F16) of
 * themselves, F16 also within 2^-32 of the row's largest.  Values that a row sees must be finite
 * (an infinite one comes out as NaN or infinity); NaN scores give NaN rows.  The split of a
 * row depends on the call's sizes (num_seqs, max_context_len, window, num_sinks, heads) alone,
 * not on the other rows' contents.
 */
int pa_decode_window(void *out, pa_dtype out_dtype, const void *query, const void *key_cache,
                     const void *value_cache, const int32_t *block_tables, int max_blocks_per_seq,
                     const int32_t *context_lens, int max_context_len, int window, int num_sinks,
                     int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                     int num_blocks, float scale, pa_dtype kv_dtype, int32_t *status,
                     pa_stream_t stream);

/*
 * pa_prefill_window -- chunked prefill under the window: row i of sequence s sits at
 * position context_lens[s] - Lq_s + i.  Arguments, invalid chunks and dtypes (F16, BF16) as
 * for pa_prefill_chunk.  Values at the positions that some row of a chunk sees must be
 * finite (a key that one row sees and another does not enters the second row's sum with
 * weight zero); NaN scores give NaN rows.  The softmax weights are rounded to the cache's type
 * (F16: but to no coarser than 2^-32 of the row's largest) before the products and the row
 * sums; the products are summed by the tensor core, which cuts off what falls below the last
 * bits of its fp32 sum (up to 2^-24 of a row's magnitude per key).  How a row's keys are split
 * depends on the call's sizes alone.
 */
int pa_prefill_window(void *out, pa_dtype out_dtype, const void *query,
                      const int32_t *query_start_loc, int num_tokens, int max_query_len,
                      const void *key_cache, const void *value_cache, const int32_t *block_tables,
                      int max_blocks_per_seq, const int32_t *context_lens, int max_context_len,
                      int window, int num_sinks, int num_seqs, int num_heads, int num_kv_heads,
                      int head_dim, int block_size, int num_blocks, float scale, pa_dtype kv_dtype,
                      int32_t *status, pa_stream_t stream);

/*
 * Rotary positions with several axes (time, height and width of images and video): every
 * rotated pair belongs to one axis and turns by that axis's position of the token.
 */
#define PA_ROPE_MAX_AXES 8
typedef struct {
    const float *freqs;       /* device, [rope_dim / 2]: angular frequency of pair i (pa_rope_yarn_freqs) */
    const int32_t *pair_axis; /* device, [rope_dim / 2]: axis of pair i, 0 .. num_axes - 1 (pa_rope_pair_axes) */
    int rope_dim;             /* even, 2 .. head_dim */
    int num_axes;             /* 1 .. PA_ROPE_MAX_AXES */
    int halves;               /* 0: pair i is elements (2i, 2i+1); 1: elements (i, i + rope_dim/2) */
} pa_rope_axes;

/*
 * pa_rope_pair_axes -- host: the axis of each of the rope_dim / 2 pairs from the number of
 * pairs of each axis (sections, which must add up to rope_dim / 2): interleaved = 0 gives
 * axis 0 the first sections[0] pairs, axis 1 the next sections[1], and so on; interleaved = 1
 * deals the pairs out in turn (0, 1, 2, 0, 1, 2, ...), passing over an axis that has all of
 * its pairs.
 */
int pa_rope_pair_axes(int32_t *pair_axis, int rope_dim, const int32_t *sections, int num_axes,
                      int interleaved);

/*
 * pa_reshape_and_cache_rope_axes -- one step's rotation and cache write in one launch:
 * queries rotated into query_out, keys rotated into their cache slots, values copied into
 * theirs.
 *
 *   query_out  [num_tokens][num_heads][head_dim], kv_dtype (written, dense); may be `query`
 *              itself when query_stride is num_heads * head_dim
 *   query      num_tokens rows [num_heads][head_dim], query_stride elements apart
 *   key, value num_tokens rows [num_kv_heads][head_dim], key_stride / value_stride apart
 *   positions  int32 [num_axes][num_tokens]: position of token t on each axis
 *   slot_mapping, caches  as for pa_reshape_and_cache (a slot < 0 writes no key and value;
 *              the token's query is rotated all the same)
 *
 * Strides are in elements, at least the row and a multiple of 16 bytes (so the three may be
 * slices of one projection's output).  query_out and the caches overlap no other tensor of
 * the call, query_out == query apart.  num_heads = 0 (query and query_out NULL) rotates and
 * writes keys only.  Pair i of token t turns by positions[pair_axis[i]][t] * freqs[i], for
 * any position and |freqs[i]| < 4: the angle is formed as a 64-bit fraction of a turn, its sine
 * and cosine are within 2.2e-7 (F32) or 1e-6 (F16, BF16), the rotation is in fp32, rounded
 * once; elements past rope_dim and values are bit copies.  A pair_axis entry outside
 * [0, num_axes) is reported (PA_DEVERR_AXIS) and its pair not rotated.
 */
int pa_reshape_and_cache_rope_axes(void *query_out, const void *query, const void *key,
                                   const void *value, void *key_cache, void *value_cache,
                                   const int64_t *slot_mapping, const int32_t *positions,
                                   int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                   int64_t query_stride, int64_t key_stride, int64_t value_stride,
                                   int block_size, int num_blocks, pa_dtype kv_dtype,
                                   const pa_rope_axes *rope, int32_t *status, pa_stream_t stream);

/*
 * The same three calls with their arguments in one record, for bindings whose foreign calls
 * pay for every argument.  A field means what the argument of its name does;
 * pa_decode_window_args reads neither query_start_loc, num_tokens nor max_query_len, and
 * pa_reshape_and_cache_rope_axes_args takes the fields of pa_rope_axes beside the others.  A
 * NULL record returns PA_ERR_INVALID_ARG.
 */
typedef struct {
    void *out;
    const void *query, *key_cache, *value_cache;
    const int32_t *query_start_loc, *block_tables, *context_lens;
    int32_t *status;
    pa_stream_t stream;
    int32_t out_dtype, kv_dtype, num_tokens, max_query_len, max_blocks_per_seq, max_context_len;
    int32_t window, num_sinks, num_seqs, num_heads, num_kv_heads, head_dim, block_size, num_blocks;
    float scale;
} pa_window_args;

typedef struct {
    void *query_out;
    const void *query, *key, *value;
    void *key_cache, *value_cache;
    const int64_t *slot_mapping;
    const int32_t *positions;
    const float *freqs;
    const int32_t *pair_axis;
    int32_t *status;
    pa_stream_t stream;
    int64_t query_stride, key_stride, value_stride;
    int32_t num_tokens, num_heads, num_kv_heads, head_dim, block_size, num_blocks, kv_dtype;
    int32_t rope_dim, num_axes, halves;
} pa_rope_axes_args;

int pa_decode_window_args(const pa_window_args *args);
int pa_prefill_window_args(const pa_window_args *args);
int pa_reshape_and_cache_rope_axes_args(const pa_rope_axes_args *args);

/*
 * pa_cross_attention -- attention of packed query rows over a sequence's whole context: the
 * states of an encoder, the patches of images, a retrieved document, written to cache slots
 * once (pa_reshape_and_cache) and read by every later row.  Nothing is causal: row r sees the
 * keys [begin_r, end_r) of its sequence's context.
 *
 *   out              [num_tokens][num_heads][head_dim], out_dtype (written)
 *   query            [num_tokens][num_heads][head_dim], kv_dtype
 *   query_start_loc  int32 [num_seqs + 1], non-decreasing: the rows of sequence s are
 *                    query_start_loc[s] .. query_start_loc[s+1]-1 (one token, a beam's rows, a
 *                    chunk).  NULL: one row each, row s of sequence s, num_tokens == num_seqs
 *                    (max_query_len is not read)
 *   max_query_len    >= every sequence's rows (host bound); a sequence with more is reported
 *                    (PA_DEVERR_QUERY) and its rows left as they were (0, like num_tokens 0: a
 *                    no-op, which looks at no sequence)
 *   key_ranges       int32 [num_tokens][2], 8-byte aligned: (begin, end) of each row, cut to
 *                    [0, context); NULL: every row sees its whole context
 *   context_lens     int32 [num_seqs]: cached keys of the sequence, 0 allowed
 *   other arguments  as for pa_decode
 *
 *   out[r][h] = sum_j softmax_j(scale * q[r][h] . k_j) v_j over begin_r <= j < end_r;
 *   a row that sees no key is all zeros.  Rows of no sequence are left as they were.
 * F32, F16 and BF16 caches, any number of rows.  scale <= 0 returns PA_ERR_INVALID_ARG.  There
 * is no workspace; a call may be captured into a CUDA graph after one eager call with its cache
 * type and head dimension on the device.  Few rows (up to eight
 * (row, query head) columns per kv head, more where the call is small) and F32 caches keep their
 * weights as pa_decode_window does; the others round them to the cache's type before the products
 * and the row sums, as pa_prefill_window does.  Which of the two runs, and how a row's keys are
 * split, depends on the call's sizes alone.  Contexts below zero, past max_context_len or past the
 * block table are reported and clamped.  A block-table entry is read only if a row's range
 * reaches its block; what the cache holds in slots that no row of the sequence sees is never used,
 * not even NaN.  Values that some row of a sequence sees must be finite (a key that one row
 * sees and another does not may enter the second row's sum with weight zero); NaN scores give
 * NaN rows.
 */
int pa_cross_attention(void *out, pa_dtype out_dtype, const void *query, const int32_t *query_start_loc,
                       int num_tokens, int max_query_len, const int32_t *key_ranges, const void *key_cache,
                       const void *value_cache, const int32_t *block_tables, int max_blocks_per_seq,
                       const int32_t *context_lens, int max_context_len, int num_seqs, int num_heads,
                       int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                       pa_dtype kv_dtype, int32_t *status, pa_stream_t stream);

/*
 * Block tables kept on the device: a step's tables, row starts, positions and slots made from
 * the sequences' lengths, so that a step loop (captured into a CUDA graph, say) grows its own
 * sequences and sends nothing from the host.  The free blocks are a stack in device memory:
 * free_blocks int32 [free_capacity], of which the first *num_free are free.  These pools share no
 * blocks between sequences (pa_kv_manager.h does, on the host).  Each call is one launch, keeps
 * nothing between calls, and its results do not depend on timing.  At most 65535 sequences;
 * block_size 8, 16 or 32.  The tensors of a call overlap only where it says so.
 *
 * pa_tables_extend -- sequence s grows from cached_lens[s] to cached_lens[s] + new_lens[s] tokens.
 *
 *   block_tables     int32 [num_seqs][max_blocks_per_seq]: the first ceil(cached / block_size)
 *                    entries of a row are its blocks (read); those of the blocks it gains are
 *                    written, the rest is left as it was
 *   context_lens     int32 [num_seqs] (written): the new lengths; may be cached_lens itself
 *   query_start_loc  int32 [num_seqs + 1] or NULL (written): prefix sums of new_lens, cut to
 *                    num_tokens
 *   positions        int32 [num_tokens] or NULL (written): position of each new token
 *   slot_mapping     int64 [num_tokens] (written): its cache slot.  Rows behind the last sequence
 *                    get position 0 and slot -1 (padding, which the cache writes skip)
 *   num_free_out     int32 [1] (written): free blocks left; may be num_free itself
 *   cached_lens,
 *   new_lens         int32 [num_seqs]; new_lens[s] = 0 leaves the sequence as it is
 *   free_blocks,
 *   num_free         the stack (read): block i taken by the call, in the order of the sequences
 *                    and of their tables, is free_blocks[*num_free - 1 - i]
 *
 * A sequence that finds too few blocks left (PA_DEVERR_FREE_LIST; no later sequence gets any
 * either), would not fit its table row or has a negative length (PA_DEVERR_CONTEXT), or whose
 * rows end past num_tokens (PA_DEVERR_QUERY) is not served: it keeps its length (a negative one is
 * written as 0) and table, and its rows get position 0 and slot -1.  The caller sees the reported bit
 * and runs the step again with what it can serve.  A negative new length is reported
 * (PA_DEVERR_QUERY) and taken as 0; a *num_free outside [0, free_capacity] is reported
 * (PA_DEVERR_FREE_LIST) and taken as the nearer end, by pa_tables_trim too.
 * A block id outside [0, num_blocks) is reported (PA_DEVERR_BLOCK_ID); its tokens get slot -1.
 */
int pa_tables_extend(int32_t *block_tables, int max_blocks_per_seq, int32_t *context_lens, int32_t *query_start_loc,
                     int32_t *positions, int64_t *slot_mapping, int num_tokens, int32_t *num_free_out,
                     const int32_t *cached_lens, const int32_t *new_lens, int num_seqs, const int32_t *free_blocks,
                     const int32_t *num_free, int free_capacity, int block_size, int num_blocks, int32_t *status,
                     pa_stream_t stream);

/*
 * pa_tables_trim -- sequence s shrinks from cached_lens[s] to keep_lens[s] tokens (0: it has ended;
 * a few fewer: drafted tokens were rejected).  The blocks it no longer needs, those from
 * ceil(keep / block_size) on, go onto the stack, sequence by sequence, each sequence's last block
 * first (so that a pa_tables_extend of one trimmed sequence gives it the same blocks again).
 * free_blocks is written from *num_free on, context_lens (may be cached_lens itself) gets the
 * kept lengths, num_free_out (may be num_free itself) the new count; block_tables is only read.
 * A keep length outside [0, cached] or a cached length past the table row is reported
 * (PA_DEVERR_CONTEXT) and its sequence left as it is (a negative cached length is written as 0).
 * Blocks past the end of the list are reported (PA_DEVERR_FREE_LIST) and dropped, block ids outside
 * [0, num_blocks) reported (PA_DEVERR_BLOCK_ID) and listed as they are.
 */
int pa_tables_trim(int32_t *free_blocks, int free_capacity, int32_t *context_lens, int32_t *num_free_out,
                   const int32_t *block_tables, int max_blocks_per_seq, const int32_t *cached_lens,
                   const int32_t *keep_lens, int num_seqs, const int32_t *num_free, int block_size, int num_blocks,
                   int32_t *status, pa_stream_t stream);

/*
 * The same three calls with their arguments in one record (see pa_window_args).  In
 * pa_tables_args, lens is new_lens or keep_lens; pa_tables_trim_args reads neither
 * query_start_loc, positions, slot_mapping nor num_tokens.
 */
typedef struct {
    void *out;
    const void *query, *key_cache, *value_cache;
    const int32_t *query_start_loc, *key_ranges, *block_tables, *context_lens;
    int32_t *status;
    pa_stream_t stream;
    int32_t out_dtype, kv_dtype, num_tokens, max_query_len, max_blocks_per_seq, max_context_len;
    int32_t num_seqs, num_heads, num_kv_heads, head_dim, block_size, num_blocks;
    float scale;
} pa_cross_args;

typedef struct {
    int32_t *block_tables, *context_lens, *query_start_loc, *positions;
    int64_t *slot_mapping;
    int32_t *free_blocks, *num_free_out;
    const int32_t *cached_lens, *lens, *num_free;
    int32_t *status;
    pa_stream_t stream;
    int32_t num_seqs, max_blocks_per_seq, num_tokens, free_capacity, block_size, num_blocks;
} pa_tables_args;

int pa_cross_attention_args(const pa_cross_args *args);
int pa_tables_extend_args(const pa_tables_args *args);
int pa_tables_trim_args(const pa_tables_args *args);

/* Static description of a PA_* return code. */
const char *pa_status_string(int code);

/* Library version as major * 10000 + minor * 100 + patch. */
int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
