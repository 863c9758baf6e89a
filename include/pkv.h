/*
 * pkv.h -- paged KV-cache decode step with RoPE for one GPU (sm_103a), C ABI.
 *
 * The operation, in the words of the source pages (restated):
 *   For every sequence in a decode batch, rotate the new token's query and key
 *   with RoPE at the token's absolute position, store its key and value in a
 *   shared pool of BF16 pages (16 tokens per page, one block table per
 *   sequence and layer), then let every query head attend over its own
 *   sequence's cached pages with a softmax accumulated online in FP32, never
 *   gathering a contiguous prefix and never storing the scores.
 *   ("Hours of YouTube and 85 handtyped pages of notes on LLM Inference –
 *   Start here": the shared BF16 KV page pool item, the batched decode item
 *   and the direct paged decode attention item. The RoPE equations are those
 *   of "手写LLM推理引擎：Tokenizer、Transformer与Detokenizer三段式实现"
 *   section 3.2, read with rotate-half pairing.)
 *
 * Conventions shared by every entry point:
 *  - The return value is 0 on success or a negative errno value, as in the C
 *    engine of "llmc — 从零写一个大模型推理引擎（配套代码）" (introduction):
 *      -EINVAL  bad argument (null pointer, bad shape, misaligned storage,
 *               workspace too small, ...); nothing is launched.
 *      -ENOSPC  the storage given to kv_pool_create holds no page.
 *      -EIO     a CUDA runtime call failed; pkv_last_cuda_error() returns the
 *               cudaError_t value of the calling thread's last failure.
 *  - Tensor arguments are device pointers that the caller owns and keeps
 *    alive until the work queued on `stream` has finished. The library frees
 *    none of them and allocates no device memory except the pool's 4-byte
 *    error word (kv_pool_create).
 *  - `stream` is a cudaStream_t passed as void* (NULL: the legacy default
 *    stream). Every call only enqueues work on it; nothing synchronises except
 *    pkv_get_error.
 *  - A call runs on the current device, which must be the one that was current
 *    when the pool was created. The calls that take pkv_scoring,
 *    paged_tables_build, paged_rope_append, paged_tables_fork and
 *    paged_pages_compact return -EINVAL where it is not.
 *  - Checks that need device data (lengths, page ids) are made by the
 *    kernels. A failed check skips the affected sequence or page and sets a
 *    bit (PKV_ERR_*) in the pool's error word; no kernel traps.
 *  - Fixed geometry: head_dim 64, page_size 16 tokens, bf16 cache.
 *
 * Pool layout (the contract between the append and the decode, and what the
 * test oracle indexes independently): physical page p is a contiguous block of
 * num_kv_heads * 2 * 16 * 64 bf16 values; the element for (page p, kv head h,
 * kind K=0 / V=1, slot s, dim d) is at bf16 offset
 *     (((p * num_kv_heads + h) * 2 + kind) * 16 + s) * 64 + d.
 * One kv head's keys and values for one page are one contiguous 4 KiB block.
 *
 * Sequence conventions: seq_lens[b] is the attention length AFTER the append
 * (cached tokens + the new one); the new token goes to cache index
 * seq_lens[b] - 1, i.e. slot (seq_lens[b]-1) % 16 of page
 * block_tables[b * max_blocks + (seq_lens[b]-1) / 16]; positions[b] is the
 * RoPE position it is rotated at. block_tables is the table of ONE layer,
 * row-major [batch][max_blocks]; entries past ceil(seq_lens[b]/16) are never
 * read. Query head i reads kv head i / (num_q_heads / num_kv_heads).
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_HEAD_DIM 64
#define PKV_PAGE_SIZE 16
/* Largest query-head group (num_q_heads / num_kv_heads) the decode serves. */
#define PKV_MAX_GROUP 8

/* Bits of the pool's device error word. */
#define PKV_ERR_SEQ_LEN 0x1  /* seq_lens[b] < 1 or > max_blocks*16: sequence skipped, its output rows zeroed */
#define PKV_ERR_PAGE_ID 0x2  /* block-table entry outside [0, num_pages): that page skipped */
#define PKV_ERR_TIMEOUT 0x4  /* a bounded wait (a copy into shared memory, or another CTA's partial) gave up; results incomplete */
#define PKV_ERR_SPLITS  0x8  /* a row needed more than max_splits partial results: row skipped */
#define PKV_ERR_POSITION 0x10 /* a RoPE position outside the RoPE table's rows: token skipped, its rows zeroed */
#define PKV_ERR_NO_PAGES 0x20 /* a step needs more free pages than its list holds: the sequence gets none, its tokens no slot */
#define PKV_ERR_PARENT 0x40 /* a parent that is no sequence: the child is left empty */
#define PKV_ERR_FREE_LIST 0x80 /* a list of free pages has no room for what is given back: those pages stay out of it */

typedef struct pkv_pool pkv_pool_t;

/*
 * Wrap caller-owned device storage as a page pool. ("Hours of YouTube …",
 * shared BF16 KV page pool item: one pool of physical pages, shared by all
 * sequences and layers, each page 16 tokens of K and V.)
 *   storage        device pointer, 16-byte aligned (-EINVAL otherwise)
 *   storage_bytes  size of storage; num_pages = storage_bytes / page bytes
 *                  (-ENOSPC if that is 0)
 *   num_kv_heads   1 .. 256
 *   head_dim       must be 64;  page_size  must be 16
 * On success *pool receives a handle; the storage is neither cleared nor
 * owned. Allocates the 4-byte device error word (zeroed) on the current
 * device, which must stay current for every call that uses the pool.
 */
int kv_pool_create(pkv_pool_t **pool, void *storage, size_t storage_bytes, int num_kv_heads,
                   int head_dim, int page_size);

/* Free the handle and its error word (not the storage). NULL is accepted. */
int kv_pool_destroy(pkv_pool_t *pool);

/* Number of physical pages, or -EINVAL for a NULL pool. */
int kv_pool_num_pages(const pkv_pool_t *pool);

/* Bytes of one physical page (0 for an unsupported geometry). Host only. */
size_t kv_pool_page_bytes(int num_kv_heads, int head_dim, int page_size);

/*
 * Bound of the one wait in the decode that depends on another CTA: the CTA
 * that merges a (sequence, kv head) segment split across CTAs looks at the
 * other CTAs' partial results, each look one round trip to L2, and after
 * `looks` looks without finding them all it gives up: PKV_ERR_TIMEOUT is set,
 * that segment's output rows are left unwritten and its workspace slots stay
 * written (zero the workspace again before the next call). The default,
 * 2^20 looks, is a second or more, where the partials arrive within
 * microseconds; 0 makes every such merger give up at once (a way to exercise
 * the timeout path without any wait). The setting belongs to the pool handle
 * and is read when a decode is launched (a captured CUDA graph keeps the
 * value it was captured with). *previous, if not NULL, receives the old value.
 * Host only; no device work. (Failure handling of this library, not on the
 * pages.)
 */
int kv_pool_set_merge_wait_limit(pkv_pool_t *pool, uint32_t looks, uint32_t *previous);

/*
 * RoPE + append for one layer. ("Hours of YouTube …", shared BF16 KV page pool
 * item: decode appends the new token at its absolute RoPE position;
 * "手写LLM推理引擎…" section 3.2: the rotation, inverse frequency
 * rope_theta^(-2j/64), pairs (j, j+32).)
 *   q             bf16 [batch][num_q_heads][64]
 *   k, v          bf16 [batch][num_kv_heads][64]
 *   q_rot         fp32 [batch][num_q_heads][64] out: the rotated query
 *   block_tables  int32 [batch][max_blocks], this layer
 *   seq_lens      int32 [batch], length after the append (>= 1)
 *   positions     int32 [batch], RoPE position of the new token
 *   rope_theta    RoPE base (> 0, finite)
 * The stored key is the bf16 rounding (nearest, ties to even) of the fp64
 * rotation by the correctly rounded fp64 cos and sin of the angle (as in
 * paged_rope_cos_sin): two rounded products and one rounded sum or
 * difference. v is copied bit for bit. q_rot is fp32, not rounded to bf16.
 * A sequence with a bad length or page id gets its q_rot written but nothing
 * stored in the pool (error bit set). batch == 0 is a no-op.
 * num_q_heads must be a multiple of the pool's num_kv_heads.
 */
int paged_kv_append_rope(pkv_pool_t *pool, const void *q, const void *k, const void *v,
                         float *q_rot, const int32_t *block_tables, int max_blocks,
                         const int32_t *seq_lens, const int32_t *positions, int batch,
                         int num_q_heads, double rope_theta, void *stream);

/*
 * Device bytes of workspace paged_gqa_decode needs for these sizes on the
 * current device (0 for invalid sizes). pages_per_split: as for
 * paged_gqa_decode (0 = automatic).
 */
size_t paged_gqa_decode_workspace_bytes(int batch, int num_q_heads, int num_kv_heads,
                                        int max_blocks, int pages_per_split);

/*
 * Paged GQA decode attention for one layer, split-KV with a log-sum-exp
 * merge, in one kernel launch on `stream`: the kernel merges the pieces of
 * the (sequence, kv head) segments it split, in shared memory where the
 * pieces ran in one CTA and through the workspace where they did not. ("Hours of YouTube …", direct paged decode attention
 * item: each query head streams its sequence's cached pages and accumulates
 * softmax-weighted values online in FP32, with no gathered prefix and no
 * stored scores. The split-KV form and its merge are flash-decoding, not on
 * the pages.)
 *   q_rot        fp32 [batch][num_q_heads][64], as written by paged_kv_append_rope
 *   out          fp32 [batch][num_q_heads][64]
 *   block_tables int32 [batch][max_blocks];  seq_lens int32 [batch] (>= 1)
 *   scale        softmax scale applied to q.k (typically 1/8)
 *   pages_per_split  0: balance all (sequence, kv head, page) work items
 *                evenly over the persistent grid; > 0: cut the work into
 *                ranges of this many pages (used to force splits in tests).
 *                Small values can give a CTA several rounds of ranges; a
 *                CTA that merges a split segment then waits for CTAs of an
 *                earlier round, so run such calls with the GPU to itself
 *                (otherwise the bounded wait may end in PKV_ERR_TIMEOUT).
 *   workspace    device memory of at least paged_gqa_decode_workspace_bytes(),
 *                256-byte aligned, ZERO-FILLED before its first use. It holds
 *                the partial results of segments split between CTAs, and a
 *                zero word means "not written in this call"; every call puts
 *                the words it wrote back to zero, so a workspace is zeroed
 *                once, when it is allocated. With pages_per_split = 0 it
 *                also holds the step's plan (paged_decode_plan), if any. (After a call that set
 *                PKV_ERR_TIMEOUT, zero it again: a CTA that gave up waiting
 *                for a neighbour's partial leaves its slots as they are; see
 *                kv_pool_set_merge_wait_limit.)
 *                Calls that share a workspace must not overlap on the GPU.
 * Constraints: num_q_heads = g * num_kv_heads with 1 <= g <= PKV_MAX_GROUP.
 * Rows of a sequence with a bad length are written as zeros.
 */
int paged_gqa_decode(const pkv_pool_t *pool, const float *q_rot, float *out,
                     const int32_t *block_tables, int max_blocks, const int32_t *seq_lens,
                     int batch, int num_q_heads, float scale, int pages_per_split,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * The work plan of a decode step, written into the decode workspace. The
 * decode cuts the (sequence, kv head, page) work items of a launch into
 * ranges, one per warp, from the sequence lengths alone; the lengths are the
 * same in every layer of a step, so this call works the partition out once
 * (the page prefix sums and every range's first item) and each later
 * paged_decode_step (positions given) or paged_gqa_decode (positions NULL)
 * on the same workspace, with the same batch, lengths and shapes, reads it
 * instead of recomputing it in every CTA. A decode checks the plan against
 * its own lengths and launch shape and works the partition out itself when
 * they differ (a stale or missing plan costs time, never correctness).
 * Arguments as for paged_decode_step; pages_per_split is 0 (the automatic
 * partition). Batches above 2048 sequences are not planned (returns 0).
 * Launches one small kernel on `stream`, without programmatic dependent
 * launch, so a decode launched after it starts only once the plan is in
 * memory. (Not on the pages: a scheduling aid of this library.)
 */
int paged_decode_plan(const pkv_pool_t *pool, const int32_t *seq_lens, const int32_t *positions,
                      int rope_positions, int batch, int num_q_heads, int max_blocks,
                      void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of a RoPE table of `rows` rows. */
#define PKV_ROPE_TABLE_BYTES(rows) ((size_t)(rows) * 1024u)

/*
 * RoPE cos/sin table: row r holds, for each frequency j < 32, the cos and sin
 * of the angle positions[r] * rope_theta^(-2j/64): the product rounded once
 * to fp64, then its cos and sin correctly rounded to fp64 (the fp64 values
 * nearest to the true ones, evaluated in double-double with a rounding test;
 * every angle of positions below 2^17 at bases 1e4, 5e5 and 1e6 is decided,
 * and elsewhere an undecided value, of probability about 2^-37, is within
 * half an ulp plus 2^-90 relative). Layout of the PKV_ROPE_TABLE_BYTES(rows)
 * bytes:
 *   float[rows][32][4]  {cos_hi, cos_lo, sin_hi, sin_lo}: cos_hi = cos
 *                       rounded to fp32, cos_lo = (cos - cos_hi) rounded to
 *                       fp32 (so cos_hi + cos_lo is within 2^-48 |cos|), the
 *                       same for sin; then
 *   double[rows][32][2] {cos, sin}.
 *   positions  int32 [rows];  table  out, 16-byte aligned
 * The evaluation is a chain of about 200 dependent fp64 operations per value,
 * which on this GPU takes about 13 us whatever the number of rows: the table
 * is meant to be built once (paged_rope_table_build), not per step.
 */
int paged_rope_cos_sin(const int32_t *positions, int rows, double rope_theta, void *table,
                       void *stream);

/*
 * The RoPE table of every position 0 .. num_positions - 1 (row p = position p),
 * as paged_rope_cos_sin builds it. ("手写LLM推理引擎…" section 3.2 precomputes
 * the cos/sin of every position up to the context length once, instead of
 * per use.) paged_decode_step and paged_prefill read the row of each token's
 * position from it. table: PKV_ROPE_TABLE_BYTES(num_positions) bytes,
 * 16-byte aligned. num_positions >= 1.
 */
int paged_rope_table_build(double rope_theta, int num_positions, void *table, void *stream);

/*
 * The whole decode step of one layer in one call: paged_kv_append_rope
 * followed by paged_gqa_decode, fused. ("Hours of YouTube …", batched decode
 * item: per layer, the new token of every sequence is rotated and appended,
 * then attention reads the sequence's pages; "手写LLM推理引擎…" section 4.2
 * proposes folding RoPE into the attention kernel to save launches.) The
 * decode warp that owns a sequence's last page rotates and stores the new
 * key and value (the same bytes paged_kv_append_rope stores: the rotation is
 * rounded to bf16 exactly as fp64 arithmetic on the same fp64 cos/sin rounds
 * it), and each warp rotates the query rows it uses (in fp32).
 *   q            bf16 [batch][num_q_heads][64];  k, v bf16 [batch][num_kv_heads][64]
 *   rope_table   a RoPE table of rope_positions rows, row p for position p
 *                (paged_rope_table_build), built once for the model's theta
 *   positions    int32 [batch], RoPE position of each new token; a position
 *                outside [0, rope_positions) skips the sequence (nothing
 *                appended, its rows zeroed) and sets PKV_ERR_POSITION
 *   q_rot        fp32 [batch][num_q_heads][64] out, or NULL: the rotated query
 *                (rows of sequences with a bad length or position are zeroed)
 *   out          fp32 [batch][num_q_heads][64]
 *   other arguments as for paged_gqa_decode; the workspace is sized by
 *   paged_gqa_decode_workspace_bytes().
 * A sequence whose new-token page id is bad gets no append and no attention
 * over that page (error bit set).
 * Launch order: the kernels are launched with programmatic dependent launch.
 * This call reads seq_lens, positions, block_tables and the pool's existing
 * pages before it waits for the kernel that precedes it in `stream`. That
 * kernel must therefore not write them if it lets its dependents start early
 * (griddepcontrol.launch_dependents / cudaTriggerProgrammaticLaunchCompletion).
 * A kernel that does not trigger early, a memcpy, or this library's own
 * kernels (which never write another layer's pages) are fine. q, k, v, the
 * RoPE table and all outputs are accessed only after that wait.
 */
int paged_decode_step(pkv_pool_t *pool, const void *q, const void *k, const void *v,
                      const void *rope_table, int rope_positions, const int32_t *positions,
                      float *q_rot, float *out, const int32_t *block_tables, int max_blocks,
                      const int32_t *seq_lens, int batch, int num_q_heads, float scale,
                      int pages_per_split, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Device bytes of workspace paged_prefill needs for total_tokens chunk tokens
 * over batch sequences with max_blocks-entry block tables (0 for invalid
 * sizes: a negative count, batch < 1 or max_blocks < 1).
 */
size_t paged_prefill_workspace_bytes(int total_tokens, int batch, int max_blocks);

/*
 * Chunked causal prefill into the pool. ("Hours of YouTube …": prefill fills
 * the prompt pages, the dense causal prefill item; RoPE per "手写LLM推理引擎…"
 * section 3.2.) Sequence b holds start_pos[b] cached tokens and brings the
 * chunk of tokens cu_tokens[b] .. cu_tokens[b+1]-1 (rows of q, k, v, q_rot and
 * out) at positions start_pos[b], start_pos[b]+1, ...:
 *   - every chunk token's k is rotated and stored, with its v, at its position
 *     in its sequence's pages, with the bytes paged_kv_append_rope would store
 *     for a decode token at that position;
 *   - q_rot is its rotated q;
 *   - out is the attention of each of its query heads over the sequence's
 *     first start_pos[b] + t + 1 tokens (causal: the cached ones, the chunk's
 *     earlier tokens and itself), as paged_gqa_decode computes it.
 *   q            bf16 [total_tokens][num_q_heads][64];  k, v bf16 [total_tokens][num_kv_heads][64]
 *   q_rot, out   fp32 [total_tokens][num_q_heads][64] out
 *                (q, v, q_rot, out and rope_table 16-byte aligned: -EINVAL otherwise)
 *   block_tables int32 [batch][max_blocks], the pages of every token up to
 *                start_pos[b] + chunk length assigned;  cu_tokens int32 [batch+1]
 *                (cu_tokens[0] = 0, non-decreasing, cu_tokens[batch] = total_tokens);
 *                start_pos int32 [batch] (>= 0)
 *   rope_table   a RoPE table of rope_positions rows, row p for position p
 *                (paged_rope_table_build), built once for the model's theta
 *   workspace    device memory of at least paged_prefill_workspace_bytes(),
 *                256-byte aligned, contents irrelevant
 * Launches three kernels on `stream`: a preparation (each chunk token's
 * sequence and position, and the tile plan), the append (every chunk token
 * stored as a decode token would be, with the same certified key rounding,
 * the cos and sin read from the table row of its position), and a
 * flash-attention kernel (launched to overlap the append's end, through
 * programmatic dependent launch; it lets no later kernel start early) on the tcgen05 tensor cores, one CTA per (sequence,
 * kv head, tile of up to 128 (token, query head) rows) that streams the
 * sequence's pages once per tile. Tokens of a malformed chunk (cu_tokens
 * decreasing, a negative start, or a position past max_blocks*16) are not
 * stored, their rows are zeroed and PKV_ERR_SEQ_LEN is set; tokens at a
 * position past the table's rows are treated the same way with
 * PKV_ERR_POSITION.
 */
int paged_prefill(pkv_pool_t *pool, const void *q, const void *k, const void *v, float *q_rot,
                  float *out, const int32_t *block_tables, int max_blocks,
                  const int32_t *cu_tokens, const int32_t *start_pos, int batch, int total_tokens,
                  int num_q_heads, const void *rope_table, int rope_positions, float scale,
                  void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of the fixed device array paged_gqa_decode_no_alloc uses as workspace. */
#define PKV_NO_ALLOC_SCRATCH_BYTES (8u << 20)

/*
 * paged_gqa_decode for callers that cannot allocate device memory. The source
 * pages have no counterpart: this entry point exists because some callers may
 * not call cudaMalloc -- code running under a host framework whose memory
 * manager owns all device memory (a direct cudaMalloc there would synchronise
 * the device and escape the manager's accounting), or a plugin that a runtime
 * only hands its input and output buffers. It takes no workspace: the decode's
 * scratch lives in a fixed array of PKV_NO_ALLOC_SCRATCH_BYTES inside this
 * library, which every GPU that loads the library holds until the process
 * exits. It calls no allocation routine.
 *   Arguments, layouts and results are those of paged_gqa_decode.
 *   Returns -E2BIG when these sizes need more scratch than the array holds
 *   (paged_gqa_decode_workspace_bytes() > PKV_NO_ALLOC_SCRATCH_BYTES). With
 *   pages_per_split = 0 the need is two partial slots of (64 + 2) * group
 *   floats per warp of the persistent grid, 2 * SMs * CTAs per SM * warps
 *   per CTA * slot bytes, plus a plan area of about 8 bytes per sequence
 *   (22 KB at 2048); with groups of 8 on a 152-SM GPU (one CTA of 10 warps
 *   per SM) that is 6.2 MiB, so a GPU with 30% more SMs would get -E2BIG
 *   for groups of 8.
 *   The first call on each device looks up the array's device address (with
 *   that device current) and keeps it for the process; make that first call
 *   before any stream capture. The address does not survive a reset of the
 *   device's primary context (cudaDeviceReset): do not call this entry point
 *   after one.
 *   Each call first clears, on `stream`, the bytes of the array it will use
 *   (a cudaMemsetAsync, which allocates nothing), so the zero state the
 *   decode needs holds even after a call that ended with PKV_ERR_TIMEOUT.
 *   (This also clears any plan, so this entry point always works out its
 *   partition itself.)
 *   All calls share the one array: calls that overlap on the GPU (other
 *   streams, other threads) race and give wrong results; order them on one
 *   stream.
 */
int paged_gqa_decode_no_alloc(const pkv_pool_t *pool, const float *q_rot, float *out,
                              const int32_t *block_tables, int max_blocks,
                              const int32_t *seq_lens, int batch, int num_q_heads, float scale,
                              int pages_per_split, void *stream);

/*
 * The same decode, but every (sequence, query head) row leaves its split
 * results for paged_kv_split_combine instead of merging them:
 *   o_part     fp32 [batch*num_q_heads][max_splits][64]: split j's normalised output
 *   lse_part   fp32 [batch*num_q_heads][max_splits]: split j's log-sum-exp of the
 *              scaled scores (natural log)
 *   num_splits int32 [batch*num_q_heads]: number of splits of the row
 * pages_per_split must be > 0; max_splits must be at least
 * max_blocks / pages_per_split + 2 (integer division), else -EINVAL.
 */
int paged_gqa_decode_partials(const pkv_pool_t *pool, const float *q_rot,
                              const int32_t *block_tables, int max_blocks,
                              const int32_t *seq_lens, int batch, int num_q_heads, float scale,
                              int pages_per_split, float *o_part, float *lse_part,
                              int32_t *num_splits, int max_splits, void *stream);

/*
 * Log-sum-exp merge of split results (flash-decoding; not on the pages):
 * for each row r, with M = max_j lse[r][j] over j < num_splits[r] and
 * w_j = exp(lse[r][j] - M): out[r] = sum_j w_j o[r][j] / sum_j w_j.
 *   o_part [rows][max_splits][head_dim], lse_part [rows][max_splits],
 *   num_splits [rows] (rows with a count outside [1, max_splits], or whose
 *   every lse is -inf, are written as zeros), out [rows][head_dim] fp32.
 *   head_dim 1 .. 1024.
 */
int paged_kv_split_combine(const float *o_part, const float *lse_part, const int32_t *num_splits,
                           float *out, int rows, int max_splits, int head_dim, void *stream);

/* Largest batch paged_tables_build serves. */
#define PKV_TABLES_MAX_BATCH 8192

/*
 * A step's block tables, slot maps and positions, built on the GPU from the
 * requests' lengths and a list of free pages. Sequence b holds start_pos[b]
 * cached tokens and brings new_tokens[b] (0 or more; 1 for a decode, a chunk
 * for a prefill). With have = ceil(start/16), need = ceil((start+new)/16) -
 * have and base_b the sum of need over the sequences before b, block have + i
 * (i < need) of (layer l, sequence b) becomes
 *     free_pages[*free_head + base_b * num_layers + l * need + i],
 * and the step's token t (sequence b, the (t - cu_tokens[b])-th it brings, at
 * position p = start + t - cu_tokens[b]) gets, in layer l, slot
 * block_tables[l][b][p / 16] * 16 + p % 16 of the pool.
 *   start_pos, new_tokens  int32 [batch], batch <= PKV_TABLES_MAX_BATCH
 *   free_pages   int32 [num_free]: ids of free pages, used from entry
 *                *free_head on
 *   free_head    int32 [1], 0 <= *free_head <= num_free;  free_head_out int32
 *                [1] out: the next unused entry.
 *   block_tables int32 [num_layers][batch][max_blocks], in and out: the new
 *                blocks' entries are written, the others kept
 *   cu_tokens    int32 [batch+1] out: first token of each sequence, the last
 *                one the step's token count, capacity or not (counts stop at
 *                2^30 - 1)
 *   seq_lens     int32 [batch] out: tokens after the step (start + new, or
 *                start where the sequence is not served)
 *   positions    int32 [capacity] out;  slot_map int32 [num_layers][capacity]
 *                out: position 0 and slot -1 for entries past the step's
 *                tokens and for tokens of a sequence that is not served.
 *                capacity < 2^29.
 * No array that is written (free_head_out, block_tables, cu_tokens, seq_lens,
 * positions, slot_map) may overlap another one of the call (-EINVAL): lengths
 * and head are read by the whole grid while the new ones are written, so pass
 * one step's seq_lens and free_head_out as the next one's inputs instead of
 * updating them in place.
 * A sequence is not served, and takes no pages, when a length is negative,
 * start + new passes max_blocks*16 or its tokens end past capacity
 * (PKV_ERR_SEQ_LEN), or when it needs pages and the list does not hold those
 * of all sequences up to and including it (PKV_ERR_NO_PAGES; sequences are
 * served in order). A page id outside the pool is stored as -1, its tokens
 * get slot -1 (PKV_ERR_PAGE_ID). One launch. (Not on the pages: their engine
 * keeps the tables on the host, as pkv_sched.h does.)
 */
int paged_tables_build(pkv_pool_t *pool, const int32_t *start_pos, const int32_t *new_tokens,
                       int batch, int num_layers, const int32_t *free_pages, int num_free,
                       const int32_t *free_head, int32_t *free_head_out, int32_t *block_tables,
                       int max_blocks, int32_t *cu_tokens, int32_t *seq_lens, int32_t *positions,
                       int32_t *slot_map, int capacity, void *stream);

/* Device bytes of workspace that paged_tables_fork and paged_pages_compact need
 * for this pool (0 for a NULL pool). Host only. */
size_t paged_pages_workspace_bytes(const pkv_pool_t *pool);

/*
 * Sequences that go on from others: beams reordered after a step, a prompt that
 * was filled once and is answered several times, requests that are dropped. Child
 * b goes on from sequence parents[b] (-1: an empty sequence). Pages are shared by
 * reference: shares[p] is the number of holders of page p beyond its first, 0 for
 * a page held once and for one that is free (so paged_tables_build need not know).
 * In every layer
 *   - a child's table row has its parent's full pages. A part-filled last page
 *     stays with the parent's first child; every other child gets the next page
 *     of the list, into which the filled slots are copied (the k-th child that
 *     gets one takes entry *free_head + k * num_layers + l in layer l);
 *   - shares changes by the parent's children less one for each of its full
 *     pages, and by -1 for the part-filled page of a parent without children;
 *   - a page that has lost its last holder is given back: those pages go to the
 *     entries before the list's next one, in ascending order.
 *   parents      int32 [children];  seq_lens int32 [batch], tokens of each
 *                sequence.  children, batch <= PKV_TABLES_MAX_BATCH
 *   block_tables int32 [num_layers][batch][max_blocks]; num_layers <= 4096,
 *                max_blocks <= 2^23, children * num_layers * num_kv_heads < 2^30.
 *                A part-filled page must have one holder
 *                (this call and paged_tables_build leave it so). Entries of -1
 *                (given back before) are passed on.
 *   shares       int32 [pages of the pool]
 *   free_pages   int32 [num_free];  free_head int32 [1], 0 <= *free_head <= num_free
 *   block_tables_out int32 [num_layers][children][max_blocks] out, -1 past a
 *                child's pages;  seq_lens_out int32 [children] out;  shares_out,
 *                free_pages_out, free_head_out out, shaped as their inputs
 *   workspace    device memory of workspace_bytes, at least
 *                paged_pages_workspace_bytes(), 256-byte aligned, ZERO-FILLED
 *                before its first use and before one with another
 *                workspace_bytes; every call leaves it ready for the next one of
 *                either operation, on any pool that it is large enough for. Calls
 *                that share a workspace must not overlap on the GPU.
 * No array that is written, the workspace and the pool's storage among them, may
 * overlap another one of the call (-EINVAL): pass one call's outputs as the
 * next one's inputs.
 * A child is left empty (length 0, a row of -1, not counted among its parent's
 * children) where parents[b] is no sequence (PKV_ERR_PARENT), its parent's length
 * is negative or past max_blocks*16 (PKV_ERR_SEQ_LEN; that parent's pages stay as
 * they are), or the list does not hold the pages of all children up to and
 * including it (PKV_ERR_NO_PAGES). Pages given back that find no room before the
 * list's next entry are left out of it (PKV_ERR_FREE_LIST). A page id outside the
 * pool is passed over, in the new tables as -1 (PKV_ERR_PAGE_ID). At most three launches.
 * (Not on the pages.)
 */
int paged_tables_fork(pkv_pool_t *pool, const int32_t *parents, int children, const int32_t *seq_lens,
                      int batch, int num_layers, const int32_t *block_tables, int max_blocks,
                      const int32_t *shares, const int32_t *free_pages, int num_free,
                      const int32_t *free_head, int32_t *block_tables_out, int32_t *seq_lens_out,
                      int32_t *shares_out, int32_t *free_pages_out, int32_t *free_head_out,
                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * Held pages moved to the front of the pool, so that what is free is at its end.
 * With U the number of pages that the tables hold (entries up to ceil(seq_lens /
 * 16), each page once), the k-th held page with an id of U or more, in ascending
 * order, moves to the k-th page with an id below U that the list holds (from
 * entry *free_head on); a page that is neither held nor listed is never touched.
 * Tables and shares follow; in the list the page that was left takes the entry of
 * the page that was moved into, so *free_head stays as it is.
 *   used         int32 [1] out: U. When every page of the pool is held or listed,
 *                no page from U on is held after the call.
 *   block_tables_out int32 [num_layers][batch][max_blocks] out, -1 past a
 *                sequence's pages;  shares_out, free_pages_out out, shaped as
 *                their inputs
 *   other arguments, overlaps and page ids outside the pool: as for
 *   paged_tables_fork. A sequence of a bad length holds nothing and gets a row of
 *   -1 (PKV_ERR_SEQ_LEN); with a bad *free_head nothing moves (PKV_ERR_NO_PAGES).
 * At most four launches. (Not on the pages.)
 */
int paged_pages_compact(pkv_pool_t *pool, const int32_t *seq_lens, int batch, int num_layers,
                        const int32_t *block_tables, int max_blocks, const int32_t *shares,
                        const int32_t *free_pages, int num_free, const int32_t *free_head,
                        int32_t *block_tables_out, int32_t *shares_out, int32_t *free_pages_out,
                        int32_t *used, void *workspace, size_t workspace_bytes, void *stream);

/*
 * A RoPE table (layout of paged_rope_cos_sin) of positions 0 ..
 * num_positions - 1 for given frequencies: entry j < num_freqs of row p holds
 * magnitude times the cos and sin of fl64(p * inv_freq[j]), the product by
 * magnitude rounded once more to fp64 (exact for 1); entries from num_freqs on
 * have angle 0. With inv_freq[j] = theta^(-2j/64), 32 frequencies and
 * magnitude 1 it is the table of paged_rope_table_build. Scaled rotary
 * positions (interpolated, by wavelength band, with an attention factor) are
 * such frequencies and magnitudes.
 *   inv_freq  HOST pointer, double [num_freqs], finite, every angle below 2^52;
 *             1 <= num_freqs <= 32
 *   magnitude finite
 */
int paged_rope_table_build_freqs(const double *inv_freq, int num_freqs, double magnitude,
                                 int num_positions, void *table, void *stream);

/*
 * RoPE of a step's q and k in either pairing, of all or part of the head,
 * with the append of k and v, for one layer. Pair j < rot_dim/2 of a head is
 * dims (j, j + rot_dim/2), or (2j, 2j+1) when interleaved != 0; it is rotated
 * by entry j of the table row of the token's position. Dims from rot_dim on
 * are passed through.
 *   q, k, v    bf16 [tokens][heads][64], 16-byte aligned; token t's heads start
 *              at element t * q_stride (k_stride, v_stride), so that they may
 *              be slices of one projection's output. Strides are multiples
 *              of 8 elements, at least heads * 64.
 *   q_rot      fp32 [tokens][num_q_heads][64] out, 16-byte aligned
 *   slot_map   int32 [tokens], this layer's slots (paged_tables_build): page *
 *              16 + slot. A token with a negative slot is rotated, not stored.
 *   positions  int32 [tokens], rows of rope_table
 *   rot_dim    8, 16, .. 64
 * The stored key is rounded to bf16 once, exactly as paged_kv_append_rope
 * rounds it (with rot_dim 64, half pairs and an unscaled table the bytes are
 * the same); v is copied bit for bit. A position outside the table's rows
 * skips the token (its q_rot rows zeroed, nothing stored, PKV_ERR_POSITION);
 * a slot past the pool is not stored to (PKV_ERR_PAGE_ID).
 */
int paged_rope_append(pkv_pool_t *pool, const void *q, long long q_stride, const void *k,
                      long long k_stride, const void *v, long long v_stride, float *q_rot,
                      const int32_t *slot_map, const int32_t *positions, int tokens,
                      int num_q_heads, const void *rope_table, int rope_positions, int rot_dim,
                      int interleaved, void *stream);

/*
 * How attention scores are made and which keys a query sees. With query
 * position i and key position j of one sequence, the score is
 *     s = scale * q.k;  s = softcap * tanh(s / softcap) if softcap > 0;
 *     s = s - alibi_slopes[head] * |i - j| if alibi_slopes,
 * and key j is seen when it is in the sequence and j <= i (or j is in the
 * sequence's prefix), j > i - window if window > 0, and j is not before the
 * first key the query may see. A query that sees no key gets a zero row.
 */
typedef struct pkv_scoring {
  float scale;               /* softmax scale, finite */
  float softcap;             /* 0: scores are not capped; otherwise > 0, at most 1e30 and at least 1e-20 |scale| */
  const float *alibi_slopes; /* fp32 [num_q_heads] on the device, or NULL */
  int window;                /* 0: no window; otherwise the last `window` positions, itself included */
} pkv_scoring_t;

/* Types of an attention output or of logits. */
#define PKV_BF16 0
#define PKV_F32 1

/*
 * paged_gqa_decode with pkv_scoring scores: attention of one token a sequence,
 * at position seq_lens[b] - 1, over its cached pages. Pages before the first
 * key that a sequence sees are neither read nor looked up (they may have been
 * given back).
 *   first_keys   int32 [batch] or NULL: first key position each sequence sees
 *                (the start of its document, or of what is kept)
 *   out          [batch][num_q_heads][64] of out_type (PKV_BF16: the fp32
 *                result rounded once), 16-byte aligned
 *   other arguments as for paged_gqa_decode (the automatic partition; the
 *   workspace is sized with pages_per_split = 0; little work may leave it
 *   untouched). max_blocks <= 2^23.
 */
int paged_gqa_decode_scored(const pkv_pool_t *pool, const float *q_rot, void *out, int out_type,
                            const int32_t *block_tables, int max_blocks, const int32_t *seq_lens,
                            const int32_t *first_keys, int batch, int num_q_heads,
                            const pkv_scoring_t *scoring, void *workspace, size_t workspace_bytes,
                            void *stream);

/* Largest batch, and most blocks of a table, that paged_gqa_decode_shared serves. */
#define PKV_SHARED_MAX_BATCH 1024
#define PKV_SHARED_MAX_BLOCKS (1 << 18)

/* Device bytes of workspace paged_gqa_decode_shared needs on the current device
 * (0 for invalid sizes). */
size_t paged_gqa_decode_shared_workspace_bytes(int batch, int num_q_heads, int num_kv_heads);

/*
 * paged_gqa_decode_scored for sequences that share their first pages (beams of a
 * prompt, samples, requests behind one system prompt: paged_tables_fork makes
 * them): the pages that a group shares are read once for the group. Sequences
 * cu_groups[g] .. cu_groups[g+1] - 1 are a group whose tables agree in their first
 * shared_lens[g] / 16 entries (whole pages; as far as its shortest member goes);
 * these may be looked up in any member's table. That the tables agree is not
 * checked. A sequence that no group holds shares nothing.
 *   cu_groups    int32 [groups + 1], non-decreasing, 0 .. batch;  shared_lens int32
 *                [groups], in tokens;  0 <= groups <= batch
 *   q_rot        fp32 [batch][num_q_heads][64], 16-byte aligned
 *   out          [batch][num_q_heads][64] of out_type, 16-byte aligned. With
 *                PKV_BF16 the softmax weights of pages that are read once for a
 *                group are rounded to bf16 (and summed as rounded); all others,
 *                and with PKV_F32 these too, keep 16 bits.
 *   block_tables int32 [batch][max_blocks];  seq_lens int32 [batch] (>= 1).
 *                batch <= PKV_SHARED_MAX_BATCH, max_blocks <= PKV_SHARED_MAX_BLOCKS
 *   workspace    device memory of at least
 *                paged_gqa_decode_shared_workspace_bytes(), 256-byte aligned,
 *                contents irrelevant. Calls that share a workspace must not overlap
 *                on the GPU.
 * Neither out nor the workspace may overlap another array of the call or the
 * pool's storage (-EINVAL).
 * Rows of a sequence with a bad length are zeroed (PKV_ERR_SEQ_LEN; its group goes
 * on without it). With cu_groups that decrease or leave 0 .. batch nothing is
 * shared (PKV_ERR_SEQ_LEN): the result is that of paged_gqa_decode_scored, read
 * the long way, as it is for little work, where the groups are not looked at.
 * Keys of a bad page are skipped (PKV_ERR_PAGE_ID). Pages before the first key
 * that a tile of rows sees (128 / group members) are neither read nor looked up.
 * A value that is not finite reaches the rows that see its key and no others (with
 * a window, rows that it may have reached are worked out again from their own keys,
 * which takes long). At most two launches. (Not on the pages.)
 */
int paged_gqa_decode_shared(const pkv_pool_t *pool, const float *q_rot, void *out, int out_type,
                            const int32_t *block_tables, int max_blocks, const int32_t *seq_lens,
                            int batch, int num_q_heads, const int32_t *cu_groups,
                            const int32_t *shared_lens, int groups, const pkv_scoring_t *scoring,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * The attention of paged_prefill with pkv_scoring scores, over pages that
 * already hold the chunk's keys and values (paged_rope_append). Token t of
 * sequence b's chunk is at position start_pos[b] + t; the sequence ends with
 * its chunk.
 *   q_rot        fp32 [total_tokens][num_q_heads][64], 16-byte aligned
 *   out          [total_tokens][num_q_heads][64] of out_type, 16-byte aligned.
 *                With PKV_BF16 the softmax weights are rounded to bf16 as well
 *                (and summed as rounded); with PKV_F32 they keep 16 bits.
 *   prefix_lens  int32 [batch] or NULL: keys below prefix_lens[b] are seen by
 *                queries before them too (a prefix that attends both ways)
 *   doc_starts   int32 [total_tokens] or NULL: first key position each chunk
 *                token sees (the start of its document)
 *   block_tables, cu_tokens, start_pos, workspace: as for paged_prefill
 *   (the workspace is sized by paged_prefill_workspace_bytes).
 * Rows of tokens past the block table's end, or of a sequence with a negative
 * start, are zeroed (PKV_ERR_SEQ_LEN); rows of no chunk are not written; a bad
 * page's keys are skipped (PKV_ERR_PAGE_ID).
 * Pages before the first key that a tile of rows sees (of at most 128 / group
 * tokens) are neither read nor looked up.
 * A value that is not finite can reach the rows of neighbouring tokens of its
 * sequence (of one tile) that do not see it; slots before the first key that a
 * tile's rows see, and past the last one, may hold anything. Two launches.
 */
int paged_gqa_prefill_scored(const pkv_pool_t *pool, const float *q_rot, void *out, int out_type,
                             const int32_t *block_tables, int max_blocks, const int32_t *cu_tokens,
                             const int32_t *start_pos, const int32_t *prefix_lens,
                             const int32_t *doc_starts, int batch, int total_tokens,
                             int num_q_heads, const pkv_scoring_t *scoring, void *workspace,
                             size_t workspace_bytes, void *stream);

/* Largest number of alternatives token_logprobs gives. */
#define PKV_MAX_TOP 32

/* Device bytes of workspace token_logprobs needs (0 for invalid sizes): the
 * same for all sizes, so that one workspace serves calls of any. */
size_t token_logprobs_workspace_bytes(int rows, int vocab, int top);

/*
 * Log-probabilities of given tokens, with the entropy of each row's
 * distribution and its most likely tokens. With y = scale * logits[r] and
 * lse = log sum_v exp(y_v):
 *   logprobs[r]        = y_{targets[r]} - lse (NaN for a target outside
 *                        [0, vocab))
 *   entropy[r]         = -sum_v p_v log p_v, p_v = exp(y_v - lse), in nats
 *   top_ids[r][i]      the i-th largest logit's token, the lower id first
 *                        among equals;  top_logprobs[r][i] its log-probability
 *   logits   bf16 or fp32 (logits_type) [rows][vocab], row r at element
 *            r * row_stride; any alignment of the element
 *   scale    1 / temperature, 1e-6 .. 1e6
 *   targets  int32 [rows] with logprobs fp32 [rows], or both NULL
 *   entropy  fp32 [rows] or NULL
 *   top      0 .. min(PKV_MAX_TOP, vocab); top_ids int32 [rows][top] and
 *            top_logprobs fp32 [rows][top] (NULL when top is 0)
 *   workspace  device memory of at least token_logprobs_workspace_bytes(),
 *            256-byte aligned, ZERO-FILLED before its first use (each call
 *            leaves what it needs to be zero at zero, unless it ends with
 *            PKV_ERR_TIMEOUT). Calls that share a workspace must not overlap
 *            on the GPU.
 * A logit of -inf is a token of probability 0. A row that holds +inf or NaN,
 * or only -inf, has no distribution: its logprobs, entropy and top_logprobs
 * are NaN; top_ids still follow the order of its logits, NaN taken as -inf.
 */
int token_logprobs(const void *logits, int logits_type, long long row_stride, int rows, int vocab,
                   float scale, const int32_t *targets, int top, float *logprobs, float *entropy,
                   int32_t *top_ids, float *top_logprobs, void *workspace, size_t workspace_bytes,
                   void *stream);

/*
 * token_logprobs has no pool; its error word is in the workspace. A wait that
 * gives up sets PKV_ERR_TIMEOUT there. That call's results are incomplete: what was
 * not worked out is NaN, with top_ids 0. So is every row of later calls on the
 * workspace, until the word is reset.
 *   token_logprobs_get_error       synchronises and reads the word; reset != 0
 *                                  makes the workspace as new
 *   token_logprobs_set_wait_limit  bound of a wait in polls, for later calls of
 *                                  the process; 0 gives up at once. The
 *                                  default (previous, if not NULL, gets the
 *                                  bound that was set) is far above what a copy
 *                                  takes.
 */
int token_logprobs_get_error(void *workspace, int *bits, int reset);
int token_logprobs_set_wait_limit(uint32_t polls, uint32_t *previous);

/* Most beams of a request, and most requests, that token_beam_select serves. */
#define PKV_MAX_BEAMS 32
#define PKV_MAX_BEAM_REQUESTS 65536

/* Device bytes of workspace token_beam_select needs (0 for invalid sizes). One
 * workspace serves calls of these sizes and of fewer beams in all. */
size_t token_beam_select_workspace_bytes(int requests, int beams, int vocab, int select);

/*
 * Beam search's selection: the best continuations of every request over its
 * beams and the vocabulary. Row r = request * beams + w of the logits is beam w
 * of a request. With y = scale * logits[r] and lse = log sum_v exp(y_v), beam w
 * and token v are a candidate of value scores[r] + y_v - lse; a beam that has
 * finished is one candidate, itself: pad_token, of value scores[r]. Candidates
 * rank by weights[r] * value (value without weights: a weight is a length
 * penalty, for instance), largest first, of equal ranks the lower beam, then the
 * larger logit, then the lower token.
 *   logits     bf16 or fp32 (logits_type) [requests * beams][vocab], row r at
 *              element r * row_stride; any alignment of the element. Rows of
 *              finished beams are not read.
 *   scale      1 / temperature, 1e-6 .. 1e6
 *   scores     fp32 [requests][beams], the beams' log-probabilities so far
 *   finished   int32 [requests][beams] or NULL: not 0 where a beam has ended
 *   weights    fp32 [requests][beams] or NULL: positive, finite
 *   pad_token  0 .. vocab - 1
 *   select     1 .. PKV_MAX_TOP continuations wanted of each request
 *   parents    int32 [requests][select] out: the rows they go on from, as
 *              paged_tables_fork takes them;  tokens int32 [requests][select]
 *              out;  new_scores fp32 [requests][select] out: their values (worked
 *              out in 64 bits from sums in 32, rounded once)
 *   workspace  device memory of at least token_beam_select_workspace_bytes(),
 *              256-byte aligned, ZERO-FILLED before its first use (each call
 *              leaves what it needs to be zero at zero, unless it ends with
 *              PKV_ERR_TIMEOUT). Calls that share a workspace must not overlap
 *              on the GPU.
 * No output, the workspace among them, may overlap another array of the call
 * (-EINVAL). Where a request has fewer
 * candidates than are wanted, the rest has parent -1, pad_token and score -inf.
 * A logit of -inf is a token of probability 0. A beam whose score is not finite,
 * or whose row holds +inf or NaN or only -inf, has candidates of value -inf: its
 * first tokens. (Not on the pages.)
 *   token_beam_select_get_error  as token_logprobs_get_error; what a call that
 *                                gave up a wait did not work out has parent -1 and
 *                                score NaN. token_logprobs_set_wait_limit bounds
 *                                these waits too.
 */
int token_beam_select(const void *logits, int logits_type, long long row_stride, int requests,
                      int beams, int vocab, double scale, const float *scores,
                      const int32_t *finished, const float *weights, int pad_token, int select,
                      int32_t *parents, int32_t *tokens, float *new_scores, void *workspace,
                      size_t workspace_bytes, void *stream);
int token_beam_select_get_error(void *workspace, int *bits, int reset);


/*
 * Read the pool's device error word (PKV_ERR_* bits) into *bits; with reset
 * != 0 also clear it. Synchronises the device.
 */
int pkv_get_error(pkv_pool_t *pool, int *bits, int reset);

/* cudaError_t value of the calling thread's last CUDA failure (0 if none). */
int pkv_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
