/*
 * pagedattn.h -- C ABI of the GB300 (sm_103a) paged-KV-cache kernels.
 *
 * The KV cache lives in a pool of fixed 16-token blocks allocated once by the
 * caller; each sequence reaches its blocks through a block table (logical
 * block -> physical block), so attention reads K/V indirectly, exactly as an
 * MMU maps pages to frames ("PagedAttention：vLLM 系统论文" reading notes,
 * section 核心思想, block-pool figure and the OS-paging table; default block
 * of 16 tokens also in the vLLM deep notes, section "PagedAttention：操作系统
 * 启发的设计").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All pointers are DEVICE pointers, owned by the caller, 16-byte aligned.
 *    The library never allocates, frees or synchronises; every call only
 *    enqueues kernels on `stream` (a cudaStream_t passed as void*; NULL is the
 *    legacy default stream) and returns.
 *  - dtype: PA_DTYPE_F16 or PA_DTYPE_BF16, the type of q, out and both pools.
 *    Accumulation is fp32.
 *  - Pool layout ("HND"): k_cache, v_cache = [num_blocks][num_kv_heads]
 *    [block_size][head_dim], row-major.  Token t of sequence s lives in
 *    physical block block_tables[s][t / block_size] at offset
 *    t % block_size; slot numbers are block * block_size + offset.
 *  - block_size must be 16; head_dim 64 or 128; num_heads a multiple of
 *    num_kv_heads with a group G = num_heads / num_kv_heads of 1..16.  Query
 *    head h reads kv head h / G (grouped-query attention: several query heads
 *    share one K/V head, ICML tutorial notes, section "Attention 简化与 KV Cache
 *    优化").
 *  - Every call returns a pa_status.  Scalars and pointers are checked on the
 *    host before anything is enqueued.  Device arrays are not read on the
 *    host; kernels bounds-check every block id, slot and length they use,
 *    skip the offending access and record a PA_DEVERR_* bit that
 *    pa_get_device_error() returns.  No kernel traps.
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PAGEDATTN_VERSION 1

enum pa_status {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size or count */
    PA_ERR_UNSUPPORTED = 2,   /* head_dim, block_size, group or dtype not built */
    PA_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required */
    PA_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed */
    PA_ERR_DEVICE = 5         /* a kernel recorded an error (see pa_get_device_error) */
};

enum pa_dtype { PA_DTYPE_F16 = 0, PA_DTYPE_BF16 = 1 };

/* bits recorded by kernels; read and cleared with pa_get_device_error() */
#define PA_DEVERR_SLOT_RANGE   0x1u  /* reshape_and_cache: slot >= num_blocks*block_size */
#define PA_DEVERR_BLOCK_RANGE  0x2u  /* copy_blocks: src or dst outside [0, num_blocks) */
#define PA_DEVERR_TABLE_RANGE  0x4u  /* decode/gather: table entry outside [0, num_blocks) */
#define PA_DEVERR_SEQLEN_RANGE 0x8u  /* seq_len < 0 or > max_blocks_per_seq*block_size */
#define PA_DEVERR_TIMEOUT      0x10u /* a bounded wait on a copy expired */
#define PA_DEVERR_APPEND_SLOT  0x20u /* decode_append: slot is not the last position's */
#define PA_DEVERR_QUERY_RANGE  0x40u /* prefill: chunk < 0, > seq_len or > max_query_len;
                                      * block_bounds: start outside [0, seq_len], or
                                      * not -1 with seq_len 0 */
#define PA_DEVERR_POSITION_RANGE 0x80u /* rotation: position >= max_position */

/* PAGEDATTN_VERSION of the loaded library. */
int pa_version(void);

/* Static, human-readable name of a pa_status. */
const char *pa_status_string(int status);

/*
 * Library plumbing, no passage of the pages behind it: bytes of device
 * workspace pa_decode needs for these sizes (0 when none).  partition_size
 * selects the split-K mode exactly as in pa_decode.  The value depends on the
 * current device's SM count for the split modes.  It takes max_blocks_per_seq
 * (the block-table row length, which bounds every sequence's length) rather
 * than a maximum sequence length, because that is the figure pa_decode itself
 * receives.
 */
size_t pa_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                int head_dim, int max_blocks_per_seq,
                                int partition_size);

/*
 * Paged decode attention, one query token per sequence.
 *
 * For every sequence s and query head h:
 *     out[s][h] = sum_t softmax_t(scale * q[s][h] . k_t) v_t,   t < seq_lens[s]
 * with k_t, v_t read through block_tables (the block-table figure of the vLLM
 * reading notes: attention addresses non-contiguous KV through the table).
 * The result is the exact softmax attention; scores are never materialised
 * (online softmax with running max and sum, vLLM deep notes, section
 * "核心思想：Tiling + Online Softmax").  A sequence of length 0 yields zeros.
 *
 *   out          [num_seqs][num_heads][head_dim]        dtype, written
 *   q            [num_seqs][num_heads][head_dim]        dtype
 *   k_cache, v_cache  pool, layout above                dtype
 *   block_tables [num_seqs][max_blocks_per_seq] int32;  entries past a
 *                sequence's ceil(len/16) blocks are never read
 *   seq_lens     [num_seqs] int32, 0 <= len <= max_blocks_per_seq * 16
 *   scale        multiplies q.k (typically 1/sqrt(head_dim))
 *
 * Split-K along the sequence (FlashDecoding, ICML tutorial notes, section
 * "内核优化"), chosen by partition_size:
 *   -1  no split: one warp reduces each (sequence, kv head) run whole;
 *    0  balanced split: the grid is sized to the GPU and every warp gets the
 *       same number of 16-token tiles; runs cut by a tile-range boundary are
 *       finished by a log-sum-exp merge.  A batch whose tables are at most
 *       kWholeMaxBlocks = 8 blocks wide and whose (sequence, kv head) runs
 *       number at most four per SM is decoded as with -1 instead (every run
 *       short and on a warp of its own: no merge to wait for);
 *   >0  fixed partitions of partition_size tokens (a multiple of 16); each
 *       partition's partial result is merged with the log-sum-exp rule
 *           M = max_p m_p,  w_p = l_p exp(m_p - M),  o = sum_p w_p o_p / sum_p w_p.
 *       The partials are left at the start of the workspace, fp32, as three
 *       arrays each starting at a 256-byte boundary:
 *           m [num_seqs][num_heads][P_max]  max of the partition's scaled scores
 *           l [num_seqs][num_heads][P_max]  sum_t exp(score_t - m)
 *           o [num_seqs][num_heads][P_max][head_dim]  normalised partial output
 *       P_max = ceil(max_blocks_per_seq * 16 / partition_size); entries of
 *       partitions past a sequence's end, and of sequences that fit one
 *       partition, are not written.  Scratch of the split follows them.
 *
 * A split decode is the decode kernel plus one merge kernel (fixed mode with
 * more than one partition: two).  They are programmatic dependent launches:
 * each may be scheduled while the kernel before it on the stream drains, and
 * touches no global memory until that kernel has completed.
 *
 * workspace: device buffer of at least pa_decode_workspace_size(...) bytes,
 * 256-byte aligned, caller-owned; its contents need no initialisation.  Calls
 * that share a workspace must be ordered on one stream.  The split modes
 * always need one; with no split (-1) a workspace is needed only for batches
 * of more than 2048 sequences, whose per-sequence lengths and tile prefix
 * two small kernels build there first (smaller batches keep them in shared
 * memory).  A batch has no size limit beyond 32-bit tile indices
 * (num_seqs * max_blocks_per_seq * num_kv_heads < 2^31).
 */
int pa_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
              const int32_t *block_tables, const int32_t *seq_lens,
              int num_seqs, int num_heads, int num_kv_heads, int head_dim,
              int block_size, int max_blocks_per_seq, int num_blocks,
              float scale, int dtype, int partition_size,
              void *workspace, size_t workspace_bytes, void *stream);

/*
 * Differential attention, one query token per sequence: every head takes the
 * difference of two softmax maps over the same values.  The pages describe no
 * such operator; it reads the pool the plain decode reads, with two queries in
 * a head's q row and two keys in a pool row, head_dim / 2 channels each, side
 * by side (H = head_dim / 2):
 *     s1_t = scale * q[:H].k_t[:H],   s2_t = scale * q[H:].k_t[H:]
 *     y    = sum_t softmax_t(s1) v_t - lambda[h] * sum_t softmax_t(s2) v_t
 *     out  = out_scale * y * norm_weight / sqrt(mean y^2 + norm_eps)
 * or out = out_scale * y if norm_weight is NULL; the mean is over the head's
 * head_dim channels.  A model's learned vectors give lambda once, when its weights
 * are loaded.  fp32 throughout (the weights of the softmax enter the product
 * with V as two 16-bit terms each, in groups of more than 8 heads rounded to
 * dtype), one rounding at the end.  A sequence of
 * length 0 yields zeros.  Keys and values of live tokens must be finite; slots
 * past a sequence's end may hold anything.  out overlaps no input (out == q is
 * refused).
 *
 *   lambda       [num_heads] fp32
 *   norm_weight  [head_dim] dtype, 16-byte aligned, or NULL
 *   norm_eps     finite, >= 0; out_scale finite
 *   scale        typically 1/sqrt(head_dim / 2)
 *   workspace    at least pa_diff_decode_workspace_size(...) bytes, else as pa_decode
 * Other arguments, the groups of 1..16 heads per kv head, the split (that of
 * partition_size 0), launches and errors as pa_decode.
 */
size_t pa_diff_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                     int max_blocks_per_seq);

int pa_diff_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
                   const int32_t *block_tables, const int32_t *seq_lens, const float *lambda,
                   const void *norm_weight, int num_seqs, int num_heads, int num_kv_heads,
                   int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                   float scale, float norm_eps, float out_scale, int dtype, void *workspace,
                   size_t workspace_bytes, void *stream);

/*
 * Chunked-prefill attention over the paged pool: the newest tokens of each
 * sequence (a prompt chunk) attend causally to everything before them and to
 * one another.  Long prompts are cut into chunks that share steps with
 * decodes (vLLM deep notes, section "调度优化：Continuous / Chunked /
 * Disaggregated", part Chunked Prefill; forum summary, section
 * "Sarathi-Serve：Chunked-Prefill技术"); the chunks of a step are packed
 * back to back into one flat batch of rows, as in continuous batching (the
 * same section of the deep notes).
 *
 * Sequence s has seq_lens[s] = L tokens in the pool, its newest
 * c = query_start[s+1] - query_start[s] tokens being the chunk (their K/V
 * are written first, e.g. by pa_reshape_and_cache).  Query row i of the
 * chunk is at position L - c + i and its output is
 *     out[query_start[s] + i, h, :] = sum_{t <= L-c+i} softmax_t(scale q.k_t) v_t
 * with kv head h / (num_heads / num_kv_heads) and k_t, v_t gathered through
 * the block table as in pa_decode.
 *
 *   out, q        [total_q][num_heads][head_dim] dtype, 16-byte aligned;
 *                 total_q = query_start[num_seqs]
 *   query_start   [num_seqs + 1] int32, non-decreasing, query_start[0] = 0
 *   seq_lens      [num_seqs] int32, chunk <= len <= max_blocks_per_seq * 16
 *   max_query_len host copy of the longest chunk: it sizes the grid
 *   scale         > 0
 *   other arguments as in pa_decode.
 * Rows are computed on the fifth-generation tensor cores (S = Q.K^T and
 * O += P.V with fp32 accumulators in tensor memory); P is rounded to dtype
 * before P.V.  A chunk longer than its sequence is skipped and sets
 * PA_DEVERR_QUERY_RANGE; so does one longer than max_query_len, of which
 * only the last max_query_len-ish rows (whole 256-row tiles) are computed.
 * Table entries outside the pool set PA_DEVERR_TABLE_RANGE (block 0 is read
 * instead).
 *
 * workspace (optional, 256-byte aligned, caller-owned, no initialisation
 * needed): at least pa_prefill_workspace_size(...) bytes.  With it a small
 * planning kernel first orders the (sequence, query tile) work: longest
 * first when the batch's K/V fits in L2, so the grid ends on short work (the
 * greedy longest-first schedule); otherwise sequence by sequence, each
 * sequence's kv heads one after the other with all of its query tiles, so
 * that the blocks running together share one head's K/V through L2.
 * Without it (NULL) the work runs in a fixed order.  Results are
 * bit-identical either way.  Calls sharing a workspace must be ordered on
 * one stream.  PA_ERR_WORKSPACE if it is too small or misaligned.
 */
size_t pa_prefill_workspace_size(int num_seqs, int max_query_len, int num_heads,
                                 int num_kv_heads);

int pa_prefill(void *out, const void *q, const void *k_cache, const void *v_cache,
               const int32_t *block_tables, const int32_t *seq_lens, const int32_t *query_start,
               int num_seqs, int max_query_len, int num_heads, int num_kv_heads, int head_dim,
               int block_size, int max_blocks_per_seq, int num_blocks, float scale, int dtype,
               void *workspace, size_t workspace_bytes, void *stream);

/*
 * pa_prefill as differential attention: the formulas, lambda, norm_weight,
 * norm_eps and out_scale of pa_diff_decode, the chunks, the causal mask, the
 * work order and the other arguments of pa_prefill (groups up to 128 heads,
 * scale > 0).  The softmax weights are rounded to dtype before the product
 * with V.  Rows of out past query_start[num_seqs] are left as they were.  A few
 * query tiles against a long table are spread over the SMs by their keys; over
 * how many, and with it the last bit of a result, follows from the sizes
 * passed and the sequence's length, not from the run.
 */
size_t pa_diff_prefill_workspace_size(int num_seqs, int max_query_len, int num_heads,
                                      int num_kv_heads);

int pa_diff_prefill(void *out, const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *block_tables, const int32_t *seq_lens,
                    const int32_t *query_start, const float *lambda, const void *norm_weight,
                    int num_seqs, int max_query_len, int num_heads, int num_kv_heads, int head_dim,
                    int block_size, int max_blocks_per_seq, int num_blocks, float scale,
                    float norm_eps, float out_scale, int dtype, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * One decode step with the new tokens appended on the way: the result equals
 *     pa_reshape_and_cache(k_new, v_new, k_cache, v_cache, slot_mapping,
 *                          num_seqs, ...)
 * followed by pa_decode(...), in one launch (plus the merge).  Token s is the
 * newest token of sequence s: slot_mapping[s] must be the slot of position
 * seq_lens[s] - 1 (through block_tables), or negative when sequence s gets
 * no token.  The warp that owns that position's tile takes the row from
 * k_new / v_new directly and writes it to the pool, so no other read of the
 * slot happens in the call.  A slot that is not the last position's is not
 * written and sets PA_DEVERR_APPEND_SLOT.  The block that receives a token
 * must not be read by another sequence in the same call (copy-on-write
 * guarantees this: a shared block is copied before it is written).
 *
 *   k_new, v_new  [num_seqs][num_kv_heads][head_dim]  dtype
 *   slot_mapping  [num_seqs] int64
 * Other arguments as pa_decode; k_cache, v_cache are written.
 */
int pa_decode_append(void *out, const void *q, void *k_cache, void *v_cache,
                     const int32_t *block_tables, const int32_t *seq_lens,
                     const void *k_new, const void *v_new, const int64_t *slot_mapping,
                     int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                     int block_size, int max_blocks_per_seq, int num_blocks,
                     float scale, int dtype, int partition_size,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * One decode step of a batch whose sequences come in groups that share a
 * prompt prefix: parallel samples of one prompt keep the prompt's blocks
 * shared by reference (block sharing with copy-on-write, section
 * 系统实现要点 and the page-sharing row of the OS-paging table in the vLLM
 * reading notes).  The result equals pa_decode (or pa_decode_append when
 * k_new, v_new and slot_mapping are given) up to rounding, but each group's
 * shared prefix is read once for the whole group instead of once per
 * sequence: every query column (sample, head) of a group and kv head
 * attends over the prefix together with the others, the prefix's tiles
 * read once through the group's first table (in blocks of up to 64 columns,
 * a long prefix in key chunks); each sequence's own tokens past the prefix
 * are decoded in one decode launch (the tables from the first block past
 * the prefix on, lengths less prefix_len); the partial results
 * of every (sequence, head) are combined with the log-sum-exp rule of the
 * split-K merge.
 *
 *   group_size   sequences [g*group_size, (g+1)*group_size) form group g;
 *                num_seqs must be a multiple of it
 *   prefix_len   tokens of the shared prefix, a multiple of 16, > 0; the
 *                first prefix_len/16 entries of the tables of a group's
 *                sequences must name the same blocks (not checked: the prefix
 *                is read through the group's first table), and every sequence
 *                must be longer than prefix_len when tokens are appended (the
 *                new token must lie past the shared prefix, as copy-on-write
 *                guarantees)
 *   k_new, v_new, slot_mapping  as in pa_decode_append, or all NULL
 *   workspace    at least pa_decode_shared_prefix_workspace_size(...) bytes,
 *                256-byte aligned, caller-owned, no initialisation needed
 * Other arguments as pa_decode.  Launches: the prefix attention (which also
 * writes the suffix lengths), the suffix decode and the final merge (which
 * also folds the pieces of the suffix runs the decode's split cut), all
 * programmatic dependent launches.  A sequence shorter than prefix_len sets
 * PA_DEVERR_SEQLEN_RANGE.
 */
size_t pa_decode_shared_prefix_workspace_size(int num_seqs, int group_size, int prefix_len,
                                              int num_heads, int num_kv_heads, int head_dim,
                                              int max_blocks_per_seq);

int pa_decode_shared_prefix(void *out, const void *q, void *k_cache, void *v_cache,
                            const int32_t *block_tables, const int32_t *seq_lens,
                            const void *k_new, const void *v_new, const int64_t *slot_mapping,
                            int num_seqs, int group_size, int prefix_len, int num_heads,
                            int num_kv_heads, int head_dim, int block_size,
                            int max_blocks_per_seq, int num_blocks, float scale, int dtype,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * pa_decode without a workspace argument, for callers that cannot allocate
 * device memory: an engine that gives (nearly) all free HBM to its KV block
 * pool at start-up and forbids allocations afterwards, a plugin whose host
 * framework hands it only inputs and outputs, or code running where
 * cudaMalloc is not allowed.  The pages describe no such entry point; it has
 * no counterpart there.
 *
 * Same arguments, result and split as pa_decode with partition_size = 0
 * (balanced split).  The split-K scratch is a fixed device array of
 * PA_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads the
 * library holds until the process exits; this call allocates nothing.
 *   - Sizes whose scratch would exceed PA_NOALLOC_SCRATCH_BYTES (see
 *     pa_decode_workspace_size(..., partition_size = 0)) return
 *     PA_ERR_WORKSPACE.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture on the device.
 *   - All calls on a device share the one array and it keeps what the last
 *     call left in it: calls that can overlap on the GPU (different streams,
 *     no ordering between them) race and corrupt each other's results.  Order
 *     them on one stream.
 */
#define PA_NOALLOC_SCRATCH_BYTES (16u << 20)

int pa_decode_noalloc(void *out, const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *block_tables, const int32_t *seq_lens,
                      int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                      int block_size, int max_blocks_per_seq, int num_blocks,
                      float scale, int dtype, void *stream);

/*
 * Write each new token's K and V into its pool slot: for token i with
 * slot = slot_mapping[i] >= 0, for every kv head h,
 *     k_cache[slot / 16][h][slot % 16][:] = k_new[i][h][:]   (same for V).
 * Blocks are handed out on demand, only when a sequence produces a token
 * that needs a new one, and fill up one token per decode step (forum summary
 * of the notes repository, section 虚拟内存的启示, design point 2; the
 * demand-paging row of the OS-paging table in the vLLM reading notes).
 * Negative slots mark padding tokens and are skipped.  Raw 16-bit copies:
 * bit-exact, NaN payloads preserved.
 *
 *   k_new, v_new  [num_tokens][num_kv_heads][head_dim]  dtype
 *   slot_mapping  [num_tokens] int64
 * Slots >= num_blocks*16 are skipped and set PA_DEVERR_SLOT_RANGE.  Two tokens
 * naming the same slot race (one of them wins).
 */
int pa_reshape_and_cache(const void *k_new, const void *v_new,
                         void *k_cache, void *v_cache,
                         const int64_t *slot_mapping, int num_tokens,
                         int num_kv_heads, int head_dim, int block_size,
                         int num_blocks, int dtype, void *stream);

/*
 * New tokens made ready for attention in one pass: queries and keys normalised
 * per head (optional) and rotated by their positions, and the keys and values
 * written into their pool slots.  The pages describe the pool write alone
 * (pa_reshape_and_cache); normalising and rotating before it are what models
 * do between their projections and the attention.
 *
 * Per token and per segment x of d = head_dim / num_maps channels (a head, or
 * each of its num_maps equal parts: differential attention keeps two keys in
 * a head, see pa_diff_decode):
 *     y_c = x_c * w_c / sqrt(mean_c x_c^2 + eps)    w = q_norm (k_norm); no norm if NULL
 *     y'_a = y_a cos - y_b sin,  y'_b = y_b cos + y_a sin    for each pair (a, b)
 * with pairs (i, i + rotary_dim/2), or (2i, 2i + 1) if interleaved is
 * non-zero, i < rotary_dim / 2; channels past rotary_dim are not rotated.
 * cos and sin are cos_sin[position][i] and cos_sin[position][rotary_dim/2 + i].
 * Everything is computed in fp32 and rounded to dtype once.  Then
 *     q_out[t] = q',  k_cache[slot / 16][h][slot % 16] = k',  v_cache[...] = v
 * (v as raw bits).
 *
 *   q         [num_tokens][num_heads][head_dim]     dtype; tokens q_stride elements apart
 *   k_new, v_new [num_tokens][num_kv_heads][head_dim] dtype; k_stride, v_stride
 *             (so all three may be slices of one projection's output).  A stride is
 *             a multiple of 8 and at least the row's size; with one token any is taken
 *   q_out     [num_tokens][num_heads][head_dim], q_out_stride; may be q itself (the
 *             same pointer and stride), no other overlap
 *   cos_sin   [max_position][rotary_dim] fp32
 *   positions [num_tokens] int32; slot_mapping [num_tokens] int64
 *   q_norm, k_norm [head_dim / num_maps] dtype, or NULL
 *   num_maps  1 or 2; rotary_dim a multiple of 16, 16..head_dim / num_maps
 *   eps       finite, >= 0
 * A token with a negative slot or position is padding: nothing of it is
 * written, its q_out row stays as it was.  A position >= max_position sets
 * PA_DEVERR_POSITION_RANGE, a slot >= num_blocks*16 PA_DEVERR_SLOT_RANGE; both
 * skip the token whole.  Two tokens naming the same slot race.  The kernel is
 * a programmatic dependent launch, as the decode's are.
 */
int pa_rope_and_cache(void *q_out, const void *q, const void *k_new, const void *v_new,
                      void *k_cache, void *v_cache, const int64_t *slot_mapping,
                      const int32_t *positions, const float *cos_sin, const void *q_norm,
                      const void *k_norm, int num_tokens, int num_heads, int num_kv_heads,
                      int head_dim, int num_maps, int block_size, int num_blocks,
                      int max_position, int rotary_dim, int interleaved, float eps,
                      int64_t q_stride, int64_t k_stride, int64_t v_stride,
                      int64_t q_out_stride, int dtype, void *stream);

/*
 * The same normalisation and rotation without the pool: q_out = q', k_out = k',
 * for the entry points that append the new tokens themselves
 * (pa_decode_append, pa_decode_shared_prefix).  k_out may be k itself, as q_out
 * may be q.  Arguments as pa_rope_and_cache; a negative position marks padding.
 */
int pa_qk_norm_rope(void *q_out, void *k_out, const void *q, const void *k,
                    const int32_t *positions, const float *cos_sin, const void *q_norm,
                    const void *k_norm, int num_tokens, int num_heads, int num_kv_heads,
                    int head_dim, int num_maps, int max_position, int rotary_dim,
                    int interleaved, float eps, int64_t q_stride, int64_t k_stride,
                    int64_t q_out_stride, int64_t k_out_stride, int dtype, void *stream);

/*
 * The four calls above with their arguments in one struct, for language bindings
 * that pay for every argument (27 of them through ctypes 2.3 us, one 0.4).  The
 * fields are those calls' arguments of the same names; `size` is the struct's
 * size, anything else is PA_ERR_INVALID_ARG.  The struct is read during the
 * call alone.  Doubles are rounded to float.
 *
 * pa_rope_args: k and v are pa_rope_and_cache's k_new and v_new; it does not
 * look at k_out and k_out_stride, nor pa_qk_norm_rope at v, k_cache, v_cache,
 * slot_mapping, v_stride, block_size and num_blocks.  pa_diff_args:
 * pa_diff_decode does not look at query_start and max_query_len.
 */
struct pa_rope_args {
    uint64_t size;
    void *q_out, *k_out;
    const void *q, *k, *v;
    void *k_cache, *v_cache;
    const int64_t *slot_mapping;
    const int32_t *positions;
    const float *cos_sin;
    const void *q_norm, *k_norm;
    void *stream;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    double eps;
    int32_t num_tokens, num_heads, num_kv_heads, head_dim, num_maps, block_size, num_blocks,
        max_position, rotary_dim, interleaved, dtype;
};

struct pa_diff_args {
    uint64_t size;
    void *out;
    const void *q, *k_cache, *v_cache;
    const int32_t *block_tables, *seq_lens, *query_start;
    const float *lambda;
    const void *norm_weight;
    void *workspace, *stream;
    uint64_t workspace_bytes;
    double scale, norm_eps, out_scale;
    int32_t num_seqs, max_query_len, num_heads, num_kv_heads, head_dim, block_size,
        max_blocks_per_seq, num_blocks, dtype;
};

int pa_rope_and_cache_args(const struct pa_rope_args *args);
int pa_qk_norm_rope_args(const struct pa_rope_args *args);
int pa_diff_decode_args(const struct pa_diff_args *args);
int pa_diff_prefill_args(const struct pa_diff_args *args);

/*
 * Long contexts: reading only the blocks that matter to a query, and keeping only
 * the tokens that matter.  The pages describe neither; both work on the pool and the
 * tables of the calls above.  All six take one struct, whose `size` is its own
 * (anything else is PA_ERR_INVALID_ARG) and which is read during the call alone;
 * each call looks at the fields that its comment names, besides num_seqs,
 * num_kv_heads, head_dim, block_size, num_blocks, dtype and stream.  Doubles are
 * rounded to float.  Pointers and sizes are checked as in pa_decode; workspaces are
 * those of pa_decode (256-byte aligned, caller-owned, no initialisation, calls
 * that share one ordered on one stream).  Kernels are programmatic dependent
 * launches.  A length outside [0, max_blocks_per_seq * 16] sets
 * PA_DEVERR_SEQLEN_RANGE and a table entry outside the pool
 * PA_DEVERR_TABLE_RANGE, with what each call then does.
 */
struct pa_sparse_args {
    uint64_t size;
    void *out;
    float *mass;
    const void *q;
    void *k_cache, *v_cache, *bounds;
    const int32_t *block_tables, *seq_lens, *query_start, *starts, *new_lens;
    int32_t *tiles, *tile_lens;
    void *workspace, *stream;
    uint64_t workspace_bytes;
    double scale, decay;
    int32_t num_seqs, num_queries, max_query_len, num_heads, num_kv_heads, head_dim, block_size,
        max_blocks_per_seq, num_blocks, keep, keep_first, keep_last, dtype, reserved;
};

/*
 * The bounds of blocks' keys: for every block b that holds positions starts[s] ..
 * seq_lens[s] - 1 of a sequence, every kv head h and channel c,
 *     bounds[b][h][0][c] = min_t k[b][h][t][c],  bounds[b][h][1][c] = max_t k[b][h][t][c]
 * over the block's live tokens (all of them, also those before starts[s]).  Exact;
 * a NaN among the keys makes the channel's bounds NaN.  After a decode step starts is
 * seq_lens - 1 (-1 where a sequence has no token), after a prompt chunk the chunk's first
 * position; NULL is 0.
 *
 *   bounds [num_blocks][num_kv_heads][2][head_dim] dtype, written; k_cache,
 *   block_tables, seq_lens, starts [num_seqs] int32 or NULL, max_blocks_per_seq
 * A start outside [0, seq_len], but for the -1 of an empty sequence, sets
 * PA_DEVERR_QUERY_RANGE and counts as the nearer end.  Lengths are clamped, bad table
 * entries skipped.  A block that sequences of one call hold to different lengths, which
 * forks and appends never leave, gets each minimum and each maximum from any of them: no
 * bounds of the longer ones, for which pa_select_blocks may then leave out blocks that
 * matter.
 */
int pa_block_bounds(const struct pa_sparse_args *args);

/*
 * The blocks a query token should read.  A block's score for kv head h is the
 * largest q.k that its bounds allow to any of the group's heads,
 *     score_j = max_g sum_c max(q_gc * min_jc, q_gc * max_jc),
 * so a block that holds a large score ranks before those that cannot.  Of a
 * sequence's n = ceil(seq_len / 16) blocks each head keeps `keep`: the keep_first
 * first, the keep_last last, and of the rest those with the largest scores, ties to
 * the lowest position; all of them if n <= keep.  The choice is that of exact sums
 * (blocks whose 32-bit scores are too close to tell apart are summed again with
 * 46 bits; products below 2^-100 may count as zero).  Blocks whose score is not
 * finite (an infinity or NaN among the bounds or queries) rank first.
 *
 *   tiles     [num_seqs][num_kv_heads][keep] int32, written: the kept blocks in the
 *             order of their positions, as pool tiles block * num_kv_heads + h;
 *             -1 past the last
 *   tile_lens [num_seqs][num_kv_heads] int32, written: tokens those hold
 *   q         [num_seqs][num_heads][head_dim]; groups of 1..16
 *   bounds    as pa_block_bounds leaves them; block_tables, seq_lens,
 *             max_blocks_per_seq
 *   keep > 0, keep_first >= 0, keep_last >= 1 (the last block may be partly
 *             filled), keep_first + keep_last <= keep
 * Lengths are clamped; a bad table entry counts as block 0.
 */
size_t pa_select_blocks_workspace_size(int num_seqs, int num_kv_heads, int max_blocks_per_seq);
int pa_select_blocks(const struct pa_sparse_args *args);

/*
 * pa_decode (partition_size 0) over the listed tiles alone, each kv head its own:
 * query head h of sequence s attends to tokens 0 .. tile_lens[s][h / G] - 1 of the
 * tiles tiles[s][h / G][..], 16 tokens a tile.  Lists need not come from
 * pa_select_blocks: any tile may be named, and one named twice counts twice.
 *   out, q, k_cache, v_cache, tiles, tile_lens, keep, scale; out may not be q
 * 0 <= tile_lens <= keep * 16 (else PA_DEVERR_SEQLEN_RANGE, clamped); entries past
 * ceil(tile_lens / 16) are not read, others outside
 * [0, num_blocks * num_kv_heads) set PA_DEVERR_TABLE_RANGE and read tile 0.
 */
size_t pa_sparse_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                       int head_dim, int keep);
int pa_sparse_decode(const struct pa_sparse_args *args);

/*
 * pa_decode (partition_size 0) that also keeps account of the softmax weights:
 *     mass[s][h][t] = decay * mass[s][h][t] + sum_g softmax_t(scale * q_g . k_t)
 * over the heads g of kv head h, for t < seq_lens[s].  The newest token, t =
 * seq_lens[s] - 1, has no weight from before: its old entry is not read, nor is
 * any with decay 0.  Entries past the length are left as they were.  Masses are
 * fp32 throughout, no atomics.  Keys of live tokens must be finite.
 *   out, q, k_cache, v_cache, block_tables, seq_lens, max_blocks_per_seq, scale,
 *   mass [num_seqs][num_kv_heads][max_blocks_per_seq * 16] fp32, decay (finite);
 *   out may not be q.  A sequence's masses lie in its row of the batch and are as wide as
 *   the tables: where a sequence gets another row, or the tables another width, the
 *   caller copies them over (and a fork's from its parent's row).  The workspace holds the
 *   scores: 4 bytes for each query head (an odd group one more) and position of the tables,
 *   of as many sequences as four gigabytes hold, but one at least: a larger batch is taken
 *   in parts, one after the other.  Shapes that the call refuses have size 0.
 * Errors as pa_decode.
 */
size_t pa_decode_mass_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                     int max_blocks_per_seq);
int pa_decode_mass(const struct pa_sparse_args *args);

/*
 * The weights that a prompt chunk's queries give, without their outputs:
 *     mass[s][h][t] = decay * mass[s][h][t] + sum_{i, g} softmax_t(scale * q_ig . k_t)
 * over the chunk's rows i and the heads g of kv head h, causal as in pa_prefill (a
 * row at position p sees t <= p).  The chunk's own tokens have no weight from before.
 * Chunk after chunk it accumulates a prompt's weights; on a prompt's last rows alone
 * (q and query_start of those, decay 0) it says which tokens the end of the prompt
 * looks at.  Sequences without rows are left as they were.  Keys of live tokens must
 * be finite.
 *   mass, q [num_queries][num_heads][head_dim], k_cache, block_tables, seq_lens,
 *   query_start [num_seqs + 1] int32, max_query_len, max_blocks_per_seq, scale > 0,
 *   decay; groups of 1..128
 * A chunk that is negative, longer than its sequence or than max_query_len (it may be
 * taken all the same up to the next 2 * (128 / group) rows), or whose rows lie outside q
 * sets PA_DEVERR_QUERY_RANGE; that, or a bad length, leaves the sequence as it was.
 * Bad table entries read block 0.  A workspace of a longer max_query_len serves shorter
 * ones too (its own, where chunks have few rows, lets the keys be read only once).  It holds
 * 8 bytes for each 2 * (128 / group) tokens of a chunk and place of the tables of a kv head, of
 * as many of those as a gigabyte holds, but one at least: a longer max_query_len (as far as
 * the tables reach) is taken in parts, one after the other, whether chunks have rows there or
 * not.  Shapes that the call refuses have size 0.
 */
size_t pa_prefill_mass_workspace_size(int num_seqs, int max_query_len, int num_heads,
                                      int num_kv_heads, int max_blocks_per_seq);
int pa_prefill_mass(const struct pa_sparse_args *args);

/*
 * Eviction: each sequence longer than new_lens[s] = B is cut to B tokens in place.
 * Each kv head for itself keeps the keep_last last tokens (at most B), the
 * keep_first first ones (at most what is left) and of the rest those with the largest
 * mass, ties to the lowest slot, a NaN before all.  The last ones keep their
 * order at slots B - keep_last .. B - 1; the others keep their slots, but for those
 * that lie past the last ones' new place: they move, in ascending order, to the slots
 * before it that dropped tokens leave, in ascending order.  (Attention of a later
 * token does not depend on the order of the keys before it; what was rotated into
 * a key stays with it.)  mass moves along.  Slots from B on are left as they were, as
 * are sequences of at most B tokens.  The caller goes on with min(seq_len, B) tokens, and
 * may give back the blocks past them (pa_bm_shorten); pa_block_bounds of the sequence are
 * out of date.
 *   k_cache, v_cache, mass (written), block_tables, seq_lens, new_lens [num_seqs]
 *   int32, max_blocks_per_seq, keep_first >= 0, keep_last >= 0
 * The blocks that hold the first B tokens must be the sequence's own (pa_bm_own_blocks and
 * pa_copy_blocks first); those past them are only read.  A negative new_len, a bad length or
 * table entry leaves the sequence as it was.
 */
size_t pa_evict_workspace_size(int num_seqs, int num_kv_heads, int max_blocks_per_seq);
int pa_evict(const struct pa_sparse_args *args);

/*
 * Copy-on-write of shared blocks: for every pair i,
 *     k_cache[dst] = k_cache[src], v_cache[dst] = v_cache[src]
 * whole blocks (every kv head and slot), with (src, dst) =
 * block_mapping[i][0], block_mapping[i][1].  Blocks shared by reference
 * count are copied before a sequence writes into them (block sharing for
 * parallel sampling and beam search, the page-sharing row of the OS-paging
 * table and section 系统实现要点 of the vLLM reading notes; reference counts
 * and copy-on-write in the vLLM deep notes, section "PagedAttention：操作系统
 * 启发的设计").
 *
 *   block_mapping [num_pairs][2] int64
 * No dst may appear twice or equal any src (not checked: such pairs race).
 * Pairs naming a block outside the pool are skipped and set
 * PA_DEVERR_BLOCK_RANGE.  Raw 16-bit copies, bit-exact.
 */
int pa_copy_blocks(void *k_cache, void *v_cache, const int64_t *block_mapping,
                   int num_pairs, int num_kv_heads, int head_dim, int block_size,
                   int num_blocks, int dtype, void *stream);

/*
 * Swap blocks between two pools, for preemption: for every pair i,
 *     dst_k[dst] = src_k[src], dst_v[dst] = src_v[src]
 * whole blocks, (src, dst) = block_mapping[i][0], block_mapping[i][1].  One
 * side is the GPU pool, the other a pool of the same layout in page-locked
 * host memory (cudaHostAlloc / cudaHostRegister): blocks of a preempted
 * sequence move to host memory and back instead of being recomputed (the
 * swap row of the OS-paging table and section 系统实现要点 of the vLLM
 * reading notes).  The copy is one kernel reading and writing both pools
 * directly; on GB300 host memory is reached over NVLink-C2C.
 *
 *   src_num_blocks, dst_num_blocks  pool sizes in blocks
 *   block_mapping  [num_pairs][2] int64, device or page-locked host memory
 * Pools must be device memory, managed memory or page-locked host memory;
 * anything else (pageable host memory) returns PA_ERR_INVALID_ARG.  Pairs
 * naming a block outside its pool are skipped and set PA_DEVERR_BLOCK_RANGE.
 * No dst may appear twice (not checked).  Bit-exact.
 */
int pa_swap_blocks(void *dst_k, void *dst_v, const void *src_k, const void *src_v,
                   const int64_t *block_mapping, int num_pairs, int num_kv_heads,
                   int head_dim, int block_size, int src_num_blocks, int dst_num_blocks,
                   int dtype, void *stream);

/*
 * Debug/test export: materialise each sequence's K and V contiguously,
 * read through its block table (the same indirection the decode uses):
 *     k_out[s][h][t][:] = k_cache[block_tables[s][t/16]][h][t%16][:],  t < seq_lens[s]
 *   k_out, v_out  [num_seqs][num_kv_heads][max_blocks_per_seq*16][head_dim];
 *   positions t >= seq_lens[s] are not written.  Bit-exact copies.
 */
int pa_gather_kv(void *k_out, void *v_out, const void *k_cache, const void *v_cache,
                 const int32_t *block_tables, const int32_t *seq_lens,
                 int num_seqs, int num_kv_heads, int head_dim, int block_size,
                 int max_blocks_per_seq, int num_blocks, int dtype, void *stream);

/*
 * Library plumbing, no passage of the pages behind it.  Check the tables a
 * decode would read: counts, into *bad_count (a device uint32 the caller
 * zeroes), the entries block_tables[s][b] with
 * b < ceil(seq_lens[s]/16) outside [0, num_blocks), plus the sequences whose
 * length is outside [0, max_blocks_per_seq*16].
 */
int pa_validate_tables(const int32_t *block_tables, const int32_t *seq_lens,
                       int num_seqs, int max_blocks_per_seq, int num_blocks,
                       int block_size, uint32_t *bad_count, void *stream);

/*
 * Test export for the failure path every copy wait shares: a kernel arms an
 * mbarrier for bytes no copy will deliver and waits with a limit of
 * limit_us microseconds (1..1e6).  The wait must give up, set
 * PA_DEVERR_TIMEOUT and let the kernel finish, leaving the context usable.
 */
int pa_selftest_bounded_wait(int limit_us, void *stream);

/*
 * Library plumbing, no passage of the pages behind it.  Synchronise `stream`,
 * return in *bits the PA_DEVERR_* bits kernels on the current device have
 * recorded since the last clear, and clear them when `clear` is non-zero.
 * Returns PA_ERR_DEVICE when bits is non-zero.  An expired bounded wait is
 * one of those bits (PA_DEVERR_TIMEOUT) rather than a status of its own: the
 * kernel that gave up has long returned when the host asks, and it may have
 * recorded other bits too.
 */
int pa_get_device_error(void *stream, uint32_t *bits, int clear);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
