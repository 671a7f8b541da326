/*
 * pagedattn.h -- C ABI of the GB300 (sm_103a) paged-attention decode library.
 *
 * The KV cache is one pool of fixed-size physical blocks (16 or 32 tokens);
 * each sequence's block table maps its logical token blocks to physical block
 * ids, and the attention kernel looks the table up itself (itimpress.au
 * "PagedAttention, speculative decoding, MoE and Blackwell", section 1;
 * yangyu.win blog #54 section 2.2; learn.tanhdev.com "Part 8: Inference
 * optimization with vLLM", section on executing the kernel math in CUDA).
 *
 * Conventions for every entry point:
 *  - Pointers named as device pointers must point to memory of the pool's
 *    device, 16-byte aligned, owned by the caller (the library never frees
 *    them). The library owns only what pa_pool_create allocated.
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *    stream). Work is enqueued asynchronously; no call synchronises except
 *    pa_pool_check.
 *  - Argument errors are detected on the host and returned before anything is
 *    launched. Data errors that only the device can see (a block id outside the
 *    pool, a context length the table cannot hold, a slot outside the pool) are
 *    checked on the device: the access is skipped or clamped and a sticky bit
 *    is set in the pool's status word, read back by pa_pool_check.
 *
 * Layouts (row-major, element = one 16-bit fp16 or bf16 value):
 *   K pool, V pool   [num_blocks, num_kv_heads, block_size, head_dim]
 *   new k, v         [num_tokens, num_kv_heads, head_dim]
 *   q, out           [num_seqs, q_len, num_q_heads, head_dim]
 *   block_tables     int32 [num_seqs, block_table_stride]
 *   context_lens     int32 [num_seqs], counting the q_len newest tokens
 *   slot_mapping     int64 [num_tokens], slot = block * block_size + offset
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_status {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,    /* bad pointer, size, alignment or geometry; nothing launched */
    PA_ERR_UNSUPPORTED = 2,    /* valid but not built (e.g. head_dim not in {64, 128}) */
    PA_ERR_CUDA = 3,           /* a CUDA runtime or driver call failed */
    PA_ERR_OOM = 4,            /* pa_pool_create could not allocate; too few free blocks (pa_allocator_*, pa_step_tables) */
    PA_ERR_DEVICE_BOUNDS = 5,  /* pa_pool_check: a kernel saw an out-of-range block id, slot or length */
    PA_ERR_TIMEOUT = 6         /* pa_pool_check: a kernel gave up waiting on a copy (bounded wait) */
} pa_status;

typedef enum pa_dtype { PA_FP16 = 0, PA_BF16 = 1 } pa_dtype;

/*
 * How K and V are stored in the pool.
 *  PA_KV_16BIT     in the model dtype: each cache is [num_blocks, Hkv, bs, head_dim] 16-bit values.
 *  PA_KV_FP8_E4M3  FP8 E4M3 codes with one float32 scale per (slot, head): each cache is one buffer
 *                  of num_blocks*Hkv*bs*head_dim code bytes followed by num_blocks*Hkv*bs float32
 *                  scales ([num_blocks, Hkv, bs]). pa_cache_write quantises: scale = amax|row| / 448
 *                  (1 for an all-zero row), code = e4m3(x / scale), nearest even, saturated; decode
 *                  uses code * scale. head_dim 128 only. (yangyu.win blog #54 section 4 and the
 *                  quantisation section of learn.tanhdev.com part 8: FP8 E4M3 halves the KV cache.)
 */
typedef enum pa_kv_format { PA_KV_16BIT = 0, PA_KV_FP8_E4M3 = 1 } pa_kv_format;

typedef struct pa_pool pa_pool;

/*
 * Geometry of one KV pool and the limits the pool's workspace is sized for.
 * A pool describes one attention layer's cache. Layers with the same geometry
 * may share one pool object and pass their own caches to pa_cache_write and
 * pa_decode.
 */
typedef struct pa_pool_config {
    int32_t num_blocks;        /* physical blocks in the pool (> 0) */
    int32_t block_size;        /* tokens per block: 16 or 32 */
    int32_t num_kv_heads;      /* KV heads (> 0) */
    int32_t head_dim;          /* 64 or 128 */
    int32_t dtype;             /* pa_dtype of K, V, q and out */
    int32_t device;            /* CUDA device ordinal */
    int32_t partition_tokens;  /* context partition length for the split pass; 0 = 512.
                                  Must be a positive multiple of block_size. */
    int32_t max_seqs;          /* largest num_seqs passed to pa_decode */
    int32_t max_q_heads;       /* largest num_q_heads */
    int32_t max_q_len;         /* largest q_len (1..8) */
    int32_t max_context_len;   /* largest context length (sizes the split workspace) */
    void *k_cache;             /* device pointer to a caller-owned K pool, or NULL to allocate */
    void *v_cache;             /* same for V */
    int32_t kv_format;         /* pa_kv_format (0 = 16-bit in the model dtype) */
} pa_pool_config;

/*
 * Create a pool: validates the geometry, allocates the caches when the config
 * passes NULL (left uninitialised), the split workspace and the status word on
 * `device`. On success *out owns them until pa_destroy.
 * Errors: PA_ERR_INVALID_ARG (geometry), PA_ERR_UNSUPPORTED, PA_ERR_OOM, PA_ERR_CUDA.
 */
pa_status pa_pool_create(const pa_pool_config *config, pa_pool **out);

/* Release everything the pool allocated (not caller-owned caches). NULL is a no-op. */
void pa_destroy(pa_pool *pool);

/* The pool's own K and V caches (device pointers; the ones passed in or allocated) and their bytes each
   (for FP8 pools: codes plus scales). */
pa_status pa_pool_caches(const pa_pool *pool, void **k_cache, void **v_cache, uint64_t *bytes_each);

/*
 * Cache write (scatter): for each token i with slot s = slot_mapping[i] >= 0
 * and each KV head h, copy k[i][h][:] to K[s / block_size][h][s % block_size][:]
 * and v likewise. Raw 16-bit words are copied without conversion (FP8 pools:
 * each row is quantised with its own scale, see pa_kv_format); negative
 * slots are skipped (padding). Slots beyond the pool are skipped and flagged
 * (PA_ERR_DEVICE_BOUNDS). Two tokens with one slot: which one lands is unspecified.
 * (A sequence growing past a block boundary receives a new physical block:
 * yangyu.win blog #54, section 5 question 2.)
 *   k, v            device, [num_tokens, num_kv_heads, head_dim]
 *   slot_mapping    device, int64 [num_tokens]
 *   k_cache/v_cache device pools to write, or NULL for the pool's own
 */
pa_status pa_cache_write(pa_pool *pool, const void *k, const void *v, const int64_t *slot_mapping,
                         int32_t num_tokens, void *k_cache, void *v_cache, void *stream);

/*
 * Paged attention decode. For sequence b, query row qi (0 <= qi < q_len) and
 * query head h (KV head g = h / (num_q_heads / num_kv_heads)):
 *   the row sits at position p = context_lens[b] - q_len + qi and attends to
 *   tokens t = 0..p, token t read from physical block block_tables[b][t / bs]
 *   at offset t % bs;
 *   out[b][qi][h] = sum_t softmax_t(scale * q[b][qi][h] . K_t) * V_t
 * (learn.tanhdev.com part 8: A_i = softmax(q_i K^T / sqrt(d_k)) computed block
 * by block with an online softmax, o_i = sum_j sum_t a_{i,j,t} v_{(j,t)}).
 * q_len > 1 verifies q_len speculative draft tokens in one pass with a causal
 * mask (itimpress.au section 1; yangyu.win section 2.4). Several tables may
 * name the same physical blocks (a shared copy-on-write prefix); no special
 * case is needed. Contexts longer than the pool's partition_tokens are cut into
 * partitions whose (max, sum, weighted V) are combined by a log-sum-exp merge
 * (maths.nthquan ch. 17 "Scaling and deployment", section on sequence
 * parallelism: local attention per segment, then a reduction); the merge uses
 * the pool's workspace and a second kernel on the same stream.
 * Accumulation is fp32; out is rounded to nearest even. Results are
 * deterministic run to run. Concurrent pa_decode calls on one pool must be
 * ordered (they share the workspace).
 *   q                     device [num_seqs, q_len, num_q_heads, head_dim]
 *   k_cache, v_cache      device pools, or NULL for the pool's own
 *   block_tables          device int32 [num_seqs, block_table_stride]; entries at or
 *                         beyond ceil(context_lens[b] / bs) are never read
 *   context_lens          device int32 [num_seqs]; q_len <= context_lens[b] <= stride * bs
 *   num_q_heads           a multiple of num_kv_heads; (num_q_heads / num_kv_heads) * q_len <= 32
 *   scale                 softmax scale (1/sqrt(head_dim) in the pages' formula)
 *   out                   device [num_seqs, q_len, num_q_heads, head_dim]
 */
pa_status pa_decode(pa_pool *pool, const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *block_tables, int32_t block_table_stride, const int32_t *context_lens,
                    int32_t num_seqs, int32_t num_q_heads, int32_t q_len, float scale, void *out,
                    void *stream);

/*
 * Paged decode for a batch whose sequences share a prefix (copy-on-write
 * blocks named by every table: yangyu.win blog #54, section 5 question 2;
 * itimpress.au section 1). Computes exactly pa_decode's result; the shared
 * part is evaluated once for the whole batch: every query row of every
 * sequence attends to each prefix partition on the 5th-generation tensor
 * cores (one pass over the prefix's K/V instead of one per sequence), the
 * decode kernel covers each sequence's own tokens, and the log-sum-exp merge
 * combines the partitions (maths.nthquan ch. 17 "Sequence parallelism").
 * Preconditions, checked on the device (violations are flagged,
 * PA_ERR_DEVICE_BOUNDS at pa_pool_check, outputs then unspecified):
 *   block_tables[b][i] == block_tables[0][i] for i < prefix_tokens / block_size;
 *   context_lens[b] - q_len >= prefix_tokens (every query row follows the prefix).
 * Host-checked: 16-bit pool, head_dim 128, the pool's partition_tokens a
 * multiple of 128, prefix_tokens a positive multiple of partition_tokens and
 * below the launch's longest context, scale > 0; all other arguments as
 * pa_decode (which this call replaces; it uses the pool's workspace).
 */
pa_status pa_decode_shared_prefix(pa_pool *pool, const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *block_tables, int32_t block_table_stride,
                                  const int32_t *context_lens, int32_t num_seqs, int32_t num_q_heads,
                                  int32_t q_len, float scale, int32_t prefix_tokens, void *out,
                                  void *stream);

/*
 * Chunked prefill: attention for a chunk of q_len new tokens per sequence, the
 * chunk's K and V already written to the pool (pa_cache_write). A long prompt
 * is processed in chunks (yangyu.win blog #54, section 4 "Chunked Prefill":
 * an 8,000-token prompt as 512-token chunks); chunk row qi sits at position
 * context_lens[b] - q_len + qi and attends causally to tokens 0..that position,
 * which is exactly pa_decode's definition with a large q_len (learn.tanhdev.com
 * part 8: A_i = softmax(q_i K^T / sqrt(d_k)), o_i = sum a v). The products run
 * on the 5th-generation tensor cores (tcgen05.mma, fp32 accumulators in tensor
 * memory); the softmax is fp32; out is rounded to nearest even.
 * Requires a 16-bit pool with head_dim 128 (PA_ERR_UNSUPPORTED otherwise).
 * Uses no workspace: concurrent calls on one pool are allowed.
 *   q              device [num_seqs, q_len, num_q_heads, 128]
 *   k_cache, v_cache  device pools, or NULL for the pool's own
 *   block_tables   device int32 [num_seqs, block_table_stride]
 *   context_lens   device int32 [num_seqs]; q_len <= context_lens[b] <= stride * bs
 *                  (violations are flagged, PA_ERR_DEVICE_BOUNDS at pa_pool_check)
 *   q_len          1 .. PA_PREFILL_MAX_Q_LEN; num_q_heads a multiple of num_kv_heads
 *   scale          softmax scale, finite and > 0 (1/sqrt(head_dim) in the pages' formula)
 *   out            device [num_seqs, q_len, num_q_heads, 128]
 */
#define PA_PREFILL_MAX_Q_LEN 8192
pa_status pa_prefill(pa_pool *pool, const void *q, const void *k_cache, const void *v_cache,
                     const int32_t *block_tables, int32_t block_table_stride, const int32_t *context_lens,
                     int32_t num_seqs, int32_t num_q_heads, int32_t q_len, float scale, void *out,
                     void *stream);

/*
 * Rotary frequencies of a model, laid out on the device once: pa_rope_append
 * turns dimension pair i of a row at position p by the angle p * inv_freq[i].
 *   inv_freq      host, rot_dim / 2 frequencies in radians per position, of either sign, magnitude
 *                 at most PA_ROPE_MAX_FREQ
 *   rot_dim       rotated dimensions of a head, a multiple of 16 (16 .. 128); dimensions
 *                 from rot_dim on pass through
 *   interleaved   0: pair i is dimensions (i, i + rot_dim / 2); 1: (2i, 2i + 1)
 *   scale         factor on every cosine and sine (1 for a plain rotation), finite
 * The frequencies are kept as turns per position in 64-bit fixed point, so the
 * angle is exact to p * 2^-64 turns (plus the frequency's own rounding, 2^-64
 * turns per position) at any 32-bit position.
 * Synchronises the device. A rope is kept for as long as calls with it, or
 * graphs that captured them, may still run.
 * Errors: PA_ERR_INVALID_ARG, PA_ERR_OOM, PA_ERR_CUDA.
 */
#define PA_ROPE_MAX_FREQ 1000000
typedef struct pa_rope pa_rope;
pa_status pa_rope_create(const double *inv_freq, int32_t rot_dim, int32_t interleaved, float scale, int32_t device,
                         pa_rope **out);
void pa_rope_destroy(pa_rope *rope);

/*
 * Rotate and append: for each token i, the q and k rows are rotated by
 * positions[i]; rotated q goes to q_out, rotated k and v to the pool at
 * slot_mapping[i], as pa_cache_write would put them (negative slots are
 * skipped, q is still rotated; slots beyond the pool are skipped and flagged,
 * PA_ERR_DEVICE_BOUNDS; two tokens with one slot: which one lands is
 * unspecified). Rotation is fp32, rounded once to the model type; an FP8 pool's
 * k codes are quantised from the fp32 values (scale 1 also where amax / 448 is
 * below the smallest fp32 number).
 *   q, k, v       device rows [heads, head_dim] of the pool's dtype, 16-byte aligned; token i's
 *                 starts i * stride elements behind the first (strides: multiples of 8, at least
 *                 heads * head_dim), so the three may be slices of one projection's output
 *   positions     device int32 [num_tokens], any sign
 *   slot_mapping  device int64 [num_tokens]
 *   num_q_heads   0 .. 65536; 0 appends without a q (q and q_out are then ignored);
 *                 num_q_heads + 2 num_kv_heads at most 262144 (PA_ERR_UNSUPPORTED)
 *   q_out         device rows, q_out_stride as above; may be q itself with the same stride,
 *                 must not overlap the rows of q, k and v otherwise (PA_ERR_INVALID_ARG, also where
 *                 rows of different strides lie in between one another)
 *   k_cache/v_cache  device pools to write, or NULL for the pool's own
 * The rope's rot_dim is at most the pool's head_dim, and its device the pool's.
 */
pa_status pa_rope_append(pa_pool *pool, const pa_rope *rope, const void *q, int64_t q_stride, const void *k,
                         int64_t k_stride, const void *v, int64_t v_stride, const int32_t *positions,
                         const int64_t *slot_mapping, int32_t num_tokens, int32_t num_q_heads, void *q_out,
                         int64_t q_out_stride, void *k_cache, void *v_cache, void *stream);

/*
 * Causal attention of packed prompts: num_seqs sequences with different numbers
 * of new tokens, rows cu_q[b] .. cu_q[b+1] of q belonging to sequence b, their K
 * and V already in the pool (pa_rope_append or pa_cache_write). Row i of
 * sequence b's n_b sits at position context_lens[b] - n_b + i and attends to
 * tokens 0..that position through the block table: whole prompts
 * (context_lens[b] = n_b), prompts with a cached prefix, chunks and single
 * tokens may be mixed. Values at positions a row does not see (later tokens,
 * unwritten slots) do not reach it, whatever their words are.
 *   q, out         device [num_tokens, num_q_heads, head_dim], not overlapping (PA_ERR_INVALID_ARG)
 *   cu_q           device int32 [num_seqs + 1], 0 <= cu_q[b] <= cu_q[b+1] <= num_tokens;
 *                  rows before cu_q[0] and from cu_q[num_seqs] on are left as they are in out
 *   block_tables   device int32 [num_seqs, block_table_stride]; entries at or beyond
 *                  ceil(context_lens[b] / bs) are never read
 *   context_lens   device int32 [num_seqs]; n_b <= context_lens[b] <= stride * bs, and at most
 *                  PA_PACKED_MAX_CONTEXT
 *   num_q_heads    a multiple of num_kv_heads, at most 128 per KV head
 *   scale          softmax scale, finite and > 0
 *   workspace      device, 16-byte aligned, at least pa_prefill_packed_workspace() bytes (0 where the
 *                  tables hold short contexts only: NULL will do), written by this call alone while
 *                  it runs
 * Violations in cu_q, block_tables or context_lens are clamped and flagged
 * (PA_ERR_DEVICE_BOUNDS at pa_pool_check); the sequence's outputs are then
 * unspecified, where cu_q decreases every sequence's. 16-bit pools, head_dim 64
 * or 128, at most PA_PACKED_MAX_SEQS sequences, num_tokens * num_q_heads below
 * 2^31 (PA_ERR_UNSUPPORTED otherwise). Nothing of the pool is written, so calls
 * with workspaces of their own may run at the same time. Results are
 * deterministic run to run. Contexts are cut along the keys, so that several
 * blocks share one, only where num_tokens rows are little work (below about
 * 2400 of 32 / 8 heads); rows of padding count there.
 */
#define PA_PACKED_MAX_SEQS 2048
#define PA_PACKED_MAX_CONTEXT (1 << 29)
pa_status pa_prefill_packed_workspace(const pa_pool *pool, int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                                      int32_t block_table_stride, uint64_t *bytes);
pa_status pa_prefill_packed(pa_pool *pool, const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *cu_q, const int32_t *block_tables, int32_t block_table_stride,
                            const int32_t *context_lens, int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                            float scale, void *workspace, uint64_t workspace_bytes, void *out, void *stream);

/*
 * The tables of a serving step, made on the device from the requests' lengths:
 * what pa_allocator_append does on the host for one sequence, for all of them
 * by one call that a captured graph can repeat. In this order:
 *   every sequence b is cut back to kept = min(context_lens[b], keep_lens[b])
 *   tokens (0: its request has ended; rejected drafts; NULL: nothing is cut), the
 *   blocks that it no longer needs go back on the free stack;
 *   it is given new_lens[b] tokens and takes the blocks that they need:
 *   context_lens[b] = kept + new_lens[b];
 *   the new tokens, sequence after sequence, get rows cu_q[b] .. cu_q[b+1] of
 *   positions and slot_mapping (as pa_rope_append and pa_cache_write take them;
 *   cu_q as pa_prefill_packed does); the rows behind them position 0, slot -1.
 * free_blocks[0 .. *num_free) is the free stack, its top last. Blocks are taken
 * in the order of sequences and their blocks; returned ones are put back so that
 * the first of them ends on top: cutting back a step's tokens and taking as many
 * again gives the same blocks. Entries of a table row at or beyond the
 * sequence's blocks, and of the stack at or beyond *num_free, are left over.
 * Every block has one owner: blocks that several tables share are the host
 * allocator's (pa_allocator_*).
 * A negative length, a sequence longer than its table row (or 2^29 tokens),
 * more new tokens than num_tokens, or *num_free outside what the pool's blocks
 * allow is flagged (PA_ERR_DEVICE_BOUNDS at pa_pool_check), more blocks than are
 * free is flagged as PA_ERR_OOM: tables, lengths and the stack's blocks are then
 * left as they are, and the step has no tokens (cu_q all 0, positions 0, slots -1).
 * So is a step that would return a block id outside the pool (PA_ERR_DEVICE_BOUNDS).
 * Another one outside the pool is flagged, its tokens' slots are -1.
 */
#define PA_TABLES_MAX_SEQS 8192
#define PA_TABLES_MAX_TOKENS 536870912
typedef struct pa_tables_args {
    int32_t num_seqs;            /* 0 .. PA_TABLES_MAX_SEQS */
    int32_t num_tokens;          /* rows of positions and slot_mapping, 0 .. PA_TABLES_MAX_TOKENS */
    int32_t block_table_stride;  /* entries of a table row, >= 1 */
    const int32_t *new_lens;     /* device [num_seqs], >= 0 */
    const int32_t *keep_lens;    /* device [num_seqs], >= 0, or NULL */
    int32_t *context_lens;       /* device [num_seqs], in and out; may be new_lens or keep_lens as well */
    int32_t *block_tables;       /* device [num_seqs, block_table_stride], in and out */
    int32_t *free_blocks;        /* device [num_blocks], in and out */
    int32_t *num_free;           /* device [1], in and out */
    int32_t *cu_q;               /* device [num_seqs + 1], out */
    int32_t *positions;          /* device [num_tokens], out */
    int64_t *slot_mapping;       /* device [num_tokens], out */
} pa_tables_args;                /* arrays that are written overlap no other one but as stated (PA_ERR_INVALID_ARG) */
pa_status pa_step_tables(pa_pool *pool, const pa_tables_args *args, void *stream);

/*
 * Sparse decoding: attention over the blocks that a cheap score selects for each
 * query, instead of the whole context. Three calls beside the cache:
 * pa_key_bounds keeps, for each block and KV head, bounds of its keys;
 * pa_select_blocks scores a sequence's blocks by them and lists the best;
 * pa_decode_selected attends to the listed blocks.
 *
 * The bounds of a block and KV head: codes hi[d], lo[d] (int8) and a step, with
 * hi * step and lo * step the largest and smallest key in each dimension,
 * rounded to the nearest multiple (even of two); step is the smallest power of
 * two with |hi|, |lo| <= 127 (0 for keys of zeros). Keys are the pool's values
 * in fp32 (FP8 pools: code * scale). A NaN or infinite key makes the step +inf:
 * its block is always wanted. One buffer: codes int8
 * [num_blocks, Hkv, 2, head_dim] (hi, then lo), then steps float32
 * [num_blocks, Hkv]; pa_key_bounds_size() bytes, owned by the caller, one for
 * each cache.
 */
pa_status pa_key_bounds_size(const pa_pool *pool, uint64_t *bytes);

/*
 * Bounds of the blocks that hold the newest tokens: sequence b's newest
 * cu_q[b+1] - cu_q[b] tokens end at context_lens[b] (as for pa_prefill_packed;
 * their K is in the pool already); the bounds of every block that holds one of
 * them are made anew from all its tokens before context_lens[b]. Other blocks'
 * bounds are left as they are: a block filled without such a call (by
 * pa_copy_blocks, say) keeps those that it had, until its next token or a call that
 * counts its tokens among the newest (as many as the context holds, new or not).
 * 16-bit and FP8 pools.
 *   k_cache        device pool, or NULL for the pool's own
 *   cu_q           device int32 [num_seqs + 1], 0 <= cu_q[b] <= cu_q[b+1] <= num_tokens
 *   block_tables   device int32 [num_seqs, block_table_stride]
 *   context_lens   device int32 [num_seqs], at most stride * bs and 2^29
 *   num_seqs       0 .. PA_TABLES_MAX_SEQS
 *   bounds         device, 32-byte aligned, pa_key_bounds_size() bytes
 * Lengths and block ids that do not fit are flagged (PA_ERR_DEVICE_BOUNDS at
 * pa_pool_check), the sequence or block is skipped, where cu_q decreases
 * possibly every sequence. Where two sequences name one block with different
 * fillings, its codes and step may be a mixture of both, the bounds of neither: one
 * of them makes them anew before they are used.
 */
pa_status pa_key_bounds(pa_pool *pool, const void *k_cache, const int32_t *cu_q, const int32_t *block_tables,
                        int32_t block_table_stride, const int32_t *context_lens, int32_t num_tokens, int32_t num_seqs,
                        void *bounds, void *stream);

/*
 * Selection: for each sequence and KV head, the `budget` blocks with the largest
 * scores, ascending, -1 behind them where the context has fewer; the first
 * num_first and the last num_last blocks of the context are always among them.
 * The score of a block is the largest, over the query rows that read the KV head
 * (q_len rows of num_q_heads / num_kv_heads heads), of
 *   s * step * (sum of c[d] * hi[d] where c[d] > 0 and of c[d] * lo[d] where c[d] < 0)
 * with the row as whole numbers c and a step s, made from q as the bounds' codes
 * are from the keys: the largest product that a key within the bounds could
 * have with it. Sums are of whole numbers and steps are powers of two, so
 * scores are exact (in fp32's range); of equal scores the lowest block comes
 * first. A row of q with a NaN or an infinity does not count.
 *   q              device [num_seqs, q_len, num_q_heads, head_dim] of the pool's dtype
 *   bounds         of a cache (pa_key_bounds)
 *   block_tables   device int32 [num_seqs, block_table_stride], at most PA_SELECT_MAX_BLOCKS entries a row
 *   context_lens   device int32 [num_seqs], counting the q_len newest tokens; 0: a row of padding
 *   num_q_heads    a multiple of num_kv_heads; (num_q_heads / num_kv_heads) * q_len <= 32
 *   budget         1 .. PA_SELECT_MAX_BUDGET, at least num_first + num_last
 *   num_last       at least the blocks that q_len tokens may lie in, ceil((q_len - 1) / bs) + 1
 *   selected       device int32 [num_seqs, num_kv_heads, budget], no part of the inputs
 * Lengths and block ids that do not fit are flagged (PA_ERR_DEVICE_BOUNDS at
 * pa_pool_check); such a block scores lowest, such a length is clamped. No
 * workspace: concurrent calls on one pool are allowed, as for pa_decode_selected.
 */
#define PA_SELECT_MAX_BUDGET 4096
#define PA_SELECT_MAX_BLOCKS 262144
pa_status pa_select_blocks(pa_pool *pool, const void *q, const void *bounds, const int32_t *block_tables,
                           int32_t block_table_stride, const int32_t *context_lens, int32_t num_seqs,
                           int32_t num_q_heads, int32_t q_len, int32_t budget, int32_t num_first, int32_t num_last,
                           int32_t *selected, void *stream);

/*
 * pa_decode over listed blocks only: row (b, qi) sits at position
 * context_lens[b] - q_len + qi and attends to the tokens at or before it in the
 * blocks selected[b][h / (num_q_heads / num_kv_heads)][0 .. budget). The list is
 * pa_select_blocks's or any other, in any order; negative entries are skipped, a
 * block listed twice counts twice. A row that sees no listed token gives zeros
 * (so does a context of 0); one whose scores are all -inf gives NaN. An infinity
 * among the values that a row sees gives it that infinity. Values at positions a
 * row does not see do not reach it, whatever their words are. Softmax and sums are
 * fp32; weights go into the product with V as two parts of 16 bits (off by 2^-16 of
 * themselves at most), in FP8 pools with bf16 outputs as one (2^-11, where the output
 * keeps 2^-8), whatever the V scales are as long as they are at most 2^90 and those
 * of a list lie within 2^100 of each other (or are 0). Deterministic run to run.
 * 16-bit pools with heads of 64 or 128 and FP8 pools.
 *   q, out         device [num_seqs, q_len, num_q_heads, head_dim], not overlapping
 *   selected       device int32 [num_seqs, num_kv_heads, budget]; budget 1 .. PA_SELECT_MAX_BUDGET
 *   scale          softmax scale; finite, and so times log2(e)
 * the others as pa_select_blocks. Entries beyond the context, lengths and block
 * ids that do not fit are flagged (PA_ERR_DEVICE_BOUNDS at pa_pool_check); such
 * an entry is skipped, such a length is clamped.
 */
pa_status pa_decode_selected(pa_pool *pool, const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *selected, int32_t budget, const int32_t *block_tables,
                             int32_t block_table_stride, const int32_t *context_lens, int32_t num_seqs,
                             int32_t num_q_heads, int32_t q_len, float scale, void *out, void *stream);

/*
 * Synchronise the device, read and clear the pool's status word.
 * Returns PA_OK, PA_ERR_DEVICE_BOUNDS, PA_ERR_TIMEOUT, PA_ERR_OOM (pa_step_tables:
 * a step needed more blocks than were free) or PA_ERR_CUDA. Of a step without
 * blocks beside one of the first two, the next call tells.
 */
pa_status pa_pool_check(pa_pool *pool, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Block manager (host side) and copy-on-write.
 *
 * The pool's physical blocks are handed out from one shared free pool; a
 * block named by several block tables (a shared prompt, parallel samples)
 * carries a reference count; before a sequence writes into a block it shares,
 * the block is copied to a private one (copy-on-write). (yangyu.win blog #54,
 * section 5 question 2; itimpress.au section 1.) The allocator is plain host
 * memory and host code, thread-safe, and never touches the GPU; the copy is
 * pa_copy_blocks. A failed call changes nothing.
 */
typedef struct pa_block_allocator pa_block_allocator;

/* An allocator of num_blocks blocks of block_size tokens, all free. */
pa_status pa_allocator_create(int32_t num_blocks, int32_t block_size, pa_block_allocator **out);
void pa_allocator_destroy(pa_block_allocator *allocator);

/* Free blocks left; the reference count of one block (0 = free). -1 on a bad argument. */
int32_t pa_allocator_num_free(pa_block_allocator *allocator);
int32_t pa_allocator_ref_count(pa_block_allocator *allocator, int32_t block_id);

/* Take n free blocks (reference count 1 each) into ids[n]; PA_ERR_OOM if fewer are free. */
pa_status pa_allocator_alloc(pa_block_allocator *allocator, int32_t n, int32_t *ids);

/* One more reference to each listed live block (a new table shares them). */
pa_status pa_allocator_fork(pa_block_allocator *allocator, const int32_t *ids, int32_t n);

/* Drop one reference per listed id (an id may repeat); blocks reaching 0 return to the free pool. */
pa_status pa_allocator_free(pa_block_allocator *allocator, const int32_t *ids, int32_t n);

/*
 * Copy-on-write before writing into block_id: if it is shared (count > 1), one
 * reference is dropped, a free block is taken into *out_id and *copy = 1 (the
 * caller copies block_id -> *out_id with pa_copy_blocks before writing);
 * otherwise *out_id = block_id and *copy = 0.
 */
pa_status pa_allocator_cow(pa_block_allocator *allocator, int32_t block_id, int32_t *out_id, int32_t *copy);

/*
 * Append n_new tokens to a sequence of *len tokens whose block-table row
 * (host int32 [stride]) holds ceil(*len / block_size) live blocks: takes a new
 * block each time a token crosses a block boundary, copy-on-writes the partly
 * filled last block if it is shared (then copy_pair = {old, new} and
 * *n_copies = 1, else 0), writes each new token's slot
 * (block * block_size + offset) to slots[n_new] (host int64), and advances *len.
 */
pa_status pa_allocator_append(pa_block_allocator *allocator, int32_t *table_row, int32_t stride, int32_t *len,
                              int32_t n_new, int64_t *slots, int32_t *copy_pair, int32_t *n_copies);

/*
 * Copy whole blocks on the device: for i < n, block pairs[2i] -> block
 * pairs[2i+1] of both caches (every KV head), raw words. pairs is a device
 * int32 [n][2]; destinations must be distinct and not sources of another pair.
 * Ids outside the pool are skipped and flagged (PA_ERR_DEVICE_BOUNDS).
 * k_cache/v_cache NULL = the pool's own.
 */
pa_status pa_copy_blocks(pa_pool *pool, const int32_t *pairs, int32_t n, void *k_cache, void *v_cache, void *stream);

/*
 * Speculative rejection sampling after the target model verified num_draft
 * draft tokens in one pass (yangyu.win blog #54, section 5 question 3;
 * maths.nthquan ch. 17 "Speculative decoding"). For each sequence b, draft
 * x_i is kept while u_i * q_i(x_i) < p_i(x_i) (fp32; i.e. with probability
 * min(1, p/q)); the first rejected position is resampled from
 * max(0, p_i - q_i) renormalised (from p_i if that has no mass) and later
 * drafts are dropped; if all are kept, one more token is drawn from
 * p_num_draft. Draws use the inverse CDF at v_b, summed as float pairs
 * (about 44 significant bits); a drawn token always has positive weight.
 *   p      device fp32 [num_seqs, num_draft + 1, vocab]  target distributions
 *   q      device fp32 [num_seqs, num_draft, vocab]      draft distributions
 *   draft  device int32 [num_seqs, num_draft]            a token outside the vocabulary counts as rejected
 *   u      device fp32 [num_seqs, num_draft]  uniforms in [0, 1) for the accept tests
 *   v      device fp32 [num_seqs]              uniforms in [0, 1) for the final draw
 *   out    device int32 [num_seqs, num_draft + 1]  kept drafts, then the drawn token, then -1
 *   n_out  device int32 [num_seqs]             tokens emitted (kept drafts + 1); 0 if the rows
 *          could not be read (a bounded wait on a copy ran out), out[b] then holds no drawn token
 * num_draft <= 64. No pool is needed.
 */
pa_status pa_spec_verify(const float *p, const float *q, const int32_t *draft, const float *u, const float *v,
                         int32_t num_seqs, int32_t num_draft, int64_t vocab, int32_t *out, int32_t *n_out,
                         void *stream);

/*
 * Penalties for repeated tokens, biases and grammar masks on logits
 * (pa_adjust_logits), and the token distribution of the result
 * (pa_token_probs), in the form pa_spec_verify takes as p. Row j of sequence b
 * (rows_per_seq rows each; row j of a verify follows drafts 0..j-1), token t,
 * in single fp32 steps in this order:
 *   count = occurrences of t in history[b][prompt_lens[b]..history_lens[b]) and draft[b][0..j)
 *   seen  = count > 0, or t occurs in history[b][0..prompt_lens[b])
 *   x = logit;  if seen: x = x > 0 ? x / repetition[b] : x * repetition[b]
 *   x = x - frequency[b] * count;  if count > 0: x = x - presence[b]
 *   x = x + bias of t;  if t's mask bit is 0: x = -inf
 *   pa_adjust_logits: out = x
 *   pa_token_probs:   out = exp((x - max x) / temperature[b]) / sum; temperature 0: 1 at the largest
 *                     x (the lowest index of equals), 0 elsewhere
 * A row whose mask leaves nothing (or only -inf) gives all -inf, all 0 as
 * probabilities (no mass: pa_spec_verify then draws no token). What a masked
 * logit holds does not matter; a NaN that is not masked makes its row of
 * probabilities NaN, and so does a +inf at a temperature above 0.
 * Every list pointer may be NULL (and its count 0): that step is then left out.
 */
typedef enum pa_logits_dtype { PA_LOGITS_FP16 = 0, PA_LOGITS_BF16 = 1, PA_LOGITS_FP32 = 2 } pa_logits_dtype;

typedef struct pa_logits_args {
    const void *logits;        /* device; row (b, j) starts at b * seq_stride + j * row_stride elements */
    int32_t dtype;             /* pa_logits_dtype */
    int32_t num_seqs;          /* >= 0 */
    int32_t rows_per_seq;      /* 1 .. PA_LOGITS_MAX_ROWS (num_draft + 1 for a verify); num_seqs * rows_per_seq < 2^24 */
    int32_t num_bias;          /* entries of a bias row, 0 .. PA_LOGITS_MAX_BIAS */
    int64_t vocab;             /* 1 .. PA_LOGITS_MAX_VOCAB */
    int64_t seq_stride, row_stride;   /* elements, >= 0; rows need not be aligned beyond an element */
    const int32_t *history;    /* device [num_seqs, history_stride]: prompt tokens, then outputs */
    int64_t history_stride;    /* 0 .. PA_LOGITS_MAX_HISTORY */
    const int32_t *history_lens;  /* device [num_seqs], clamped to 0 .. history_stride; needed with history */
    const int32_t *prompt_lens;   /* device [num_seqs]; NULL = 0 (every history token is an output) */
    const int32_t *draft;      /* device [num_seqs, rows_per_seq - 1] */
    const float *repetition;   /* device [num_seqs], > 0; 1 = none */
    const float *presence;     /* device [num_seqs]; 0 = none */
    const float *frequency;    /* device [num_seqs]; 0 = none */
    const int32_t *bias_tokens;   /* device [num_seqs, num_bias]; the last entry naming a token counts */
    const float *bias_values;  /* device [num_seqs, num_bias] */
    const int32_t *mask;       /* device [num_seqs, rows_per_seq, ceil(vocab / 32)]: bit t % 32 of word
                                  t / 32 allows token t */
    const float *temperature;  /* device [num_seqs], >= 0 (pa_token_probs; ignored by pa_adjust_logits);
                                  a negative or NaN one makes its rows NaN */
    float *out;                /* device fp32 [num_seqs, rows_per_seq, vocab]; may be logits itself (fp32,
                                  same strides), must not lie between the first and the last
                                  logit otherwise (PA_ERR_INVALID_ARG), nor overlap the lists */
} pa_logits_args;

/* Token ids outside the vocabulary (in history, draft or bias_tokens; -1 as padding) are ignored. No pool
   is needed; work is launched on the current device. PA_ERR_INVALID_ARG / PA_ERR_UNSUPPORTED (sizes above
   the limits) before anything is launched. */
#define PA_LOGITS_MAX_VOCAB 393216
#define PA_LOGITS_MAX_HISTORY 1000000
#define PA_LOGITS_MAX_BIAS 2000
#define PA_LOGITS_MAX_ROWS 4096
pa_status pa_adjust_logits(const pa_logits_args *args, void *stream);
pa_status pa_token_probs(const pa_logits_args *args, void *stream);

/*
 * Self-test of failure detection. Every wait of the kernels' copy pipelines is
 * bounded: after a time limit the kernel records PA_ERR_TIMEOUT in the pool's
 * status word and returns instead of spinning. This launches one warp that
 * waits, through the same bounded wait, on a barrier that nothing completes;
 * after limit_ns (at most 10 s) it records the timeout and returns, leaving
 * the context usable. pa_pool_check then returns PA_ERR_TIMEOUT.
 */
pa_status pa_pool_selftest_wait(pa_pool *pool, uint64_t limit_ns, void *stream);

/* Number of kernels pa_decode launches for these arguments (1, or 2 with the merge); -1 on bad args. */
int32_t pa_decode_launches(const pa_pool *pool, int32_t block_table_stride, int32_t num_seqs,
                           int32_t num_q_heads, int32_t q_len);

/*
 * Allocation-free decode.
 *
 * Some callers cannot allocate device memory: a plugin inside a host runtime
 * that owns every device allocation through its own allocator and memory
 * budget, or a latency-critical loop that must not make cudaMalloc's
 * synchronising call. Such a caller cannot create a pool, because
 * pa_pool_create allocates the split workspace. This entry point takes the
 * pool geometry directly and keeps its scratch (a status word, two work
 * counters and the split workspace) in one static device array of PA_NOALLOC_SCRATCH_BYTES, which
 * every GPU that runs it holds from its first call until the process exits.
 * The pages have no counterpart to this entry point; it computes what
 * pa_decode computes, with the same decode and merge kernels.
 *
 *  - Inputs and outputs are the caller's, with pa_decode's layouts and meaning;
 *    num_blocks .. dtype and partition_tokens (0 = 512) are as in pa_pool_config.
 *  - Scratch needed: 256 bytes (the status word and the counters with which
 *    the tensor-core kernel's CTAs share out their items; each launch leaves
 *    them at zero), plus, when P =
 *    ceil(block_table_stride * block_size / partition_tokens) > 1,
 *    num_seqs * q_len * num_q_heads * P * head_dim * 4 bytes (rounded up to
 *    256) and num_seqs * q_len * num_q_heads * P * 8. A larger request returns
 *    PA_ERR_INVALID_ARG before anything is launched.
 *  - Calls no cudaMalloc, cudaFree or other allocating routine.
 *  - The first call in a device's context, made with that device current,
 *    looks up the array's device address (again after the context is reset);
 *    make that first call before any stream capture.
 *  - Every call shares the one array and leaves its contents behind. Each call
 *    clears the status word (cudaMemsetAsync) and writes every partition slot
 *    before reading it; calls that overlap on the GPU (e.g. on two streams)
 *    race on the array and must be ordered by the caller.
 *  - There is no status word to read back. Instead, when the kernels flag
 *    anything -- a copy wait that ran out (its outputs would be left unwritten)
 *    or an out-of-range block id or context length (clamped, so the kernel
 *    does not fault) -- the call's last kernel fills the whole of `out` with
 *    NaN, so a failed call never returns stale or partial results as numbers.
 */
#define PA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

pa_status pa_decode_noalloc(const void *q, const void *k_cache, const void *v_cache, int32_t num_blocks,
                            int32_t block_size, int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                            const int32_t *block_tables, int32_t block_table_stride, const int32_t *context_lens,
                            int32_t num_seqs, int32_t num_q_heads, int32_t q_len, float scale,
                            int32_t partition_tokens, void *out, void *stream);

/* A static, human-readable name of a status code. */
const char *pa_status_string(pa_status status);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
