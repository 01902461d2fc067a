/*
 * topk_b200.h -- C ABI of the B200 (sm_100a) bucketed approximate top-k library.
 *
 * Method: "Approximate Top-k for Increased Parallelism" (Key, Ribar, Cattaneo,
 * Hudlass-Galley, Orr; arXiv 2412.04358), pith.science review page, section
 * "What carries the argument" and Fig. 2: a row of n scores is split into b
 * interleaved buckets (element i goes to bucket i mod b, "The reading"), an
 * exact top-k_b is kept per bucket (Stage 1), and when the b*k_b candidates
 * exceed k a final exact top-k keeps the k best (Stage 2).
 *
 * Common conventions
 *   - Every pointer argument named *_dev is CUDA device memory owned by the
 *     caller; the library keeps no pointer after the call returns.
 *   - Matrices are row-major and contiguous: row r of an [rows x n] array
 *     starts at element r*n.
 *   - Total order: a larger value ranks first; equal values (IEEE equality, so
 *     -0.0 ties +0.0) rank by lower index; NaN ranks above +inf and all NaNs
 *     are equal.
 *   - Outputs out_vals[rows*k] / out_idx[rows*k] hold, per row, the selected
 *     elements best-first.  When fewer than k elements are selected (fewer
 *     candidates than k, or n < k), the remaining slots hold -inf and -1.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream).  Argument errors are detected on the host before any
 *     work is queued; nothing throws across the ABI.
 *   - The workspace (when required) is caller-owned device memory of at least
 *     topk_workspace_bytes(...) bytes that MUST be zero-filled before its first
 *     use.  Every call leaves it zero-filled again when it completes on the GPU,
 *     so one workspace can be reused for any later call.  Calls that overlap on
 *     the GPU (different streams) must not share a workspace.
 *   - Device-side waits are bounded in time; a wait that expires records a
 *     code readable with topk_device_status() and the kernel returns early.
 */
#ifndef TOPK_B200_H
#define TOPK_B200_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TOPK_OK = 0,          /* queued successfully */
    TOPK_EINVAL = 1,      /* bad argument: null pointer, size < 1, k_b outside [1,4], n >= 2^31 */
    TOPK_EUNSUPPORTED = 2,/* valid but outside what this build implements (see each call) */
    TOPK_ECUDA = 3,       /* a CUDA call or kernel launch failed */
    TOPK_EWORKSPACE = 4,  /* workspace missing or smaller than topk_workspace_bytes() */
    TOPK_ESCRATCH = 5     /* topk_bucketed_noalloc: the call needs more scratch than the
                             library's built-in buffer holds (TOPK_NOALLOC_SCRATCH_BYTES) */
} topk_status;

typedef enum {
    TOPK_OP_BUCKETED = 0,
    TOPK_OP_EXACT = 1,
    TOPK_OP_SCORE = 2,
    TOPK_OP_BUCKETED_BF16 = 3
} topk_op;

/* Bytes of workspace a call of `op` with these sizes needs on the current
 * device (0 when none).  Unused arguments are ignored (d for BUCKETED/EXACT,
 * b and kb for EXACT).  Returns 0 as well for invalid sizes. */
size_t topk_workspace_bytes(int op, int64_t rows, int64_t n, int k, int b, int kb, int d);

/* Two-stage bucketed approximate top-k ("What carries the argument"; Fig. 2).
 *   scores_dev  [rows x n] float32 scores.
 *   k           number of outputs per row, 1 <= k <= 16384.
 *   b           number of interleaved buckets, 1 <= b <= 1024.
 *   kb          candidates kept per bucket, 1 <= kb <= 4 (register queues).
 *   out_vals_dev[rows x k] float32: the selected scores (input bits unchanged).
 *   out_idx_dev [rows x k] int32: their column indices.
 * The result equals the CPU definition bit for bit.  Fast path: n % 4 == 0,
 * scores 16-byte aligned and b dividing 1024; other shapes take a slower
 * general path.  Returns TOPK_EUNSUPPORTED for b > 1024 or k > 16384. */
int topk_bucketed(const float *scores_dev, int64_t rows, int64_t n, int k, int b, int kb,
                  float *out_vals_dev, int32_t *out_idx_dev, void *workspace_dev,
                  size_t workspace_bytes, void *stream);

/* topk_bucketed on bfloat16 score rows: the same selection on half the bytes
 * (the page compares the two precisions in Fig. 10, "Bandwidth comparison for
 * bfloat16 values").
 *   scores_dev   [rows x n] bf16 (raw 16-bit patterns).
 *   out_vals_dev [rows x k] bf16: the selected scores, input bits unchanged
 *                (padding slots hold -inf, 0xFF80).
 * bf16 values are ordered as the floats they represent, with the same total
 * order (ties by lowest index, -0 ties +0, NaN above +inf).  Fast path: n % 8
 * == 0, 16-byte aligned rows, b dividing 1024.  Workspace:
 * topk_workspace_bytes(TOPK_OP_BUCKETED_BF16, ...); other arguments and
 * errors as topk_bucketed. */
int topk_bucketed_bf16(const uint16_t *scores_dev, int64_t rows, int64_t n, int k, int b, int kb,
                       uint16_t *out_vals_dev, int32_t *out_idx_dev, void *workspace_dev,
                       size_t workspace_bytes, void *stream);

/* Exact top-k of every row under the total order above: the baseline the
 * page compares against (Fig. 1, "exact top-k implementations") and the
 * Stage-2 primitive.  1 <= k <= 16384 (else TOPK_EUNSUPPORTED).  No workspace:
 * pass NULL / 0. */
int topk_exact(const float *scores_dev, int64_t rows, int64_t n, int k, float *out_vals_dev,
               int32_t *out_idx_dev, void *workspace_dev, size_t workspace_bytes, void *stream);

/* Bucketed top-k over candidate lists: the merge step of a row cut into
 * column slices (several CTAs, or several GPUs that each hold part of a
 * vocabulary or an entity table).  The bucket of a pair is its GLOBAL index
 * modulo b, as for a single pass over the whole row ("What carries the
 * argument"; bucket = i mod b per "The reading"); each bucket keeps its top
 * kb pairs and the final exact top-k keeps the k best, with the total order
 * above.  When part p's lists are topk_bucketed of columns
 * [part_offset[p], part_offset[p] + n_p) of the same rows (local indices),
 * the result equals topk_bucketed of the whole rows bit for bit.
 *   vals_dev [parts x rows x m] float32 and idx_dev [parts x rows x m] int32:
 *                per part and row, m (value, index) pairs; index -1 marks an
 *                empty slot (as topk_bucketed pads).  Indices of one row must
 *                be distinct after the offsets are added.
 *   parts        1 <= parts <= 64 (else TOPK_EUNSUPPORTED).
 *   part_offset  HOST array [parts] added to every index of that part; NULL
 *                means all zero.  0 <= part_offset[p] < n_total.
 *   n_total      length of the whole rows, 1 <= n_total < 2^31.  A pair whose
 *                global index is >= n_total is skipped and sets
 *                TOPK_DEV_BAD_INDEX in the device status.
 *   k, b, kb     as in topk_bucketed; out_vals_dev / out_idx_dev [rows x k]
 *                best-first with global indices and the input value bits,
 *                padded with -inf / -1.
 * No workspace.  Asynchronous on `stream`. */
int topk_bucketed_merge(const float *vals_dev, const int32_t *idx_dev, int parts, int64_t rows,
                        int m, const int64_t *part_offset, int64_t n_total, int k, int b, int kb,
                        float *out_vals_dev, int32_t *out_idx_dev, void *stream);

/* Exact re-ranking of a candidate index set ("Recall Before You Rank",
 * abstract: the supports retrieved for similar earlier queries are reused as
 * candidates and scored exactly against the current query before the top-K
 * is kept).  For row r: score_i = sum_t q[r][t] * K_r[i][t] (bf16 inputs,
 * fp32 accumulation, no 1/sqrt(d)) for every DISTINCT index 0 <= i < n among
 * cand_idx[r][0..c); the k best (score, index) pairs under the total order
 * above, best-first, padded with -inf / -1.
 *   q_dev, K_dev, d, n, k_batch_stride  as in score_topk (d 128 or 256;
 *                16-byte aligned; k_batch_stride a multiple of 8).
 *   cand_idx_dev [rows x c] int32 candidate indices: -1 marks an empty slot,
 *                repeats are scored once, an index >= n is skipped and sets
 *                TOPK_DEV_BAD_INDEX.  1 <= c <= 4096 (else TOPK_EUNSUPPORTED).
 *   out_scores_dev  nullable [rows x c] float32: the fp32 score of each slot
 *                (-inf for empty, repeated or skipped slots), for checking.
 * Values are the fp32 scores (zero as +0.0, NaN as 0x7FFFFFFF).  No
 * workspace.  Asynchronous on `stream`. */
int score_rerank(const uint16_t *q_dev, int64_t rows, int d, const uint16_t *K_dev, int64_t n,
                 int64_t k_batch_stride, const int32_t *cand_idx_dev, int c, int k,
                 float *out_vals_dev, int32_t *out_idx_dev, float *out_scores_dev, void *stream);

/* Sampling tail of top-k vocabulary sampling (the review page's "Core claim"
 * and Fig. 4, left: vocabulary sampling keeps the top k of n logits).  The
 * pages leave the tail implicit; this is plain top-k sampling.  For each row
 * of selected pairs (best-first, as the selection calls write them), index
 * idx[i] is drawn with probability w_i / sum_j w_j, w_i = exp((v_i - v_0)/T),
 * by inverse CDF with the caller's uniform u[r] in [0, 1): the first i whose
 * running sum of w exceeds u[r] * sum w (else, from rounding, the last entry
 * of positive weight).  Padding (index -1) and -inf values weigh 0.  A row
 * whose best value is NaN or +inf draws idx[0]; a row with no candidate
 * draws -1.  Weights and sums are fp32.
 *   vals_dev, idx_dev  [rows x k] selected values / indices (device).
 *   temperature        T > 0 with 1/T finite (else TOPK_EINVAL).
 *   u_dev              [rows] float32 uniforms in [0, 1), supplied by the
 *                      caller (the library draws no random numbers).
 *   token_dev          [rows] int32 output.
 * No workspace.  Asynchronous on `stream`. */
int topk_sample_rows(const float *vals_dev, const int32_t *idx_dev, int64_t rows, int k,
                     float temperature, const float *u_dev, int32_t *token_dev, void *stream);

/* topk_bucketed with the draw of topk_sample_rows fused into it: the CTA
 * that finishes a row's selection draws that row's token right away, so the
 * selection and the sampling tail of vocabulary sampling take one kernel.
 * Arguments as in those two calls (float32 logits); out_vals_dev /
 * out_idx_dev receive the selection, token_dev the draws. */
int topk_sample(const float *logits_dev, int64_t rows, int64_t n, int k, int b, int kb,
                float temperature, const float *u_dev, int32_t *token_dev, float *out_vals_dev,
                int32_t *out_idx_dev, void *workspace_dev, size_t workspace_bytes, void *stream);

/* topk_sample on bfloat16 logits (raw 16-bit patterns): the selection of
 * topk_bucketed_bf16 with the same fused draw; a bf16 logit widens to fp32
 * exactly before the softmax.  out_vals_dev receives bf16 bits. */
int topk_sample_bf16(const uint16_t *logits_dev, int64_t rows, int64_t n, int k, int b, int kb,
                     float temperature, const float *u_dev, int32_t *token_dev,
                     uint16_t *out_vals_dev, int32_t *out_idx_dev, void *workspace_dev,
                     size_t workspace_bytes, void *stream);

/* Fused selector: score[r][i] = sum_t q[r][t] * K_r[i][t] (bf16 inputs, fp32
 * accumulation; no 1/sqrt(d) scaling), then topk_bucketed on each row of
 * scores -- the sparse-attention selector that scores the current query
 * against the whole key cache before a global top-K ("Recall Before You Rank"
 * abstract; STARC page, Fig. 3: q in R^{1 x d_h}, K in R^{L x d_h}).  The
 * score matrix is not materialised.
 *   q_dev        [rows x d] bf16 (raw 16-bit patterns), 16-byte aligned.
 *   K_dev        bf16 keys; row r uses K_r = K_dev + r*k_batch_stride
 *                elements, an [n x d] row-major matrix.  k_batch_stride = 0
 *                shares one key matrix between all rows.  16-byte aligned.
 *   d            128 or 256 (else TOPK_EUNSUPPORTED).
 *   k, b, kb     as in topk_bucketed, with b dividing 1024 (else
 *                TOPK_EUNSUPPORTED).
 *   out_scores_dev  nullable [rows x n] float32: when given, receives the
 *                fp32 scores the selection ran on (for checking).
 * Output values are the fp32 scores (a zero score is returned as +0.0 and a
 * NaN score as the quiet NaN 0x7FFFFFFF). */
int score_topk(const uint16_t *q_dev, int64_t rows, int d, const uint16_t *K_dev, int64_t n,
               int64_t k_batch_stride, int k, int b, int kb, float *out_vals_dev,
               int32_t *out_idx_dev, float *out_scores_dev, void *workspace_dev,
               size_t workspace_bytes, void *stream);

/* Allocation-free form of topk_bucketed.  The paper has no counterpart: this
 * entry point exists for callers that must not allocate device memory at call
 * time -- for example a serving loop in which a cudaMalloc could synchronise
 * the device and stall every other stream, a host framework whose memory
 * accounting forbids allocations it did not make itself, or a plugin that may
 * only allocate while it is being set up.  Such callers pass inputs and
 * outputs as for topk_bucketed, but no workspace: the scratch memory the
 * kernel needs for rows split across CTAs lives in one static device buffer
 * of TOPK_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads
 * the library holds until the process exits.
 *   - Nothing is allocated and no allocating routine is called: no cudaMalloc,
 *     cudaFree or library allocator.
 *   - The first call on a device looks up that device's address of the buffer
 *     (with the device current); make that first call before any stream
 *     capture begins on the device.  The address is kept per device and
 *     context: after a device reset the first call in the new context looks
 *     it up again, with the same rule on capture.
 *   - A call whose scratch need exceeds the buffer returns TOPK_ESCRATCH and
 *     queues nothing; topk_workspace_bytes(TOPK_OP_BUCKETED, ...) tells the
 *     need in advance.
 *   - Every call on a device shares the one buffer and it keeps the previous
 *     call's contents; the part that must start at zero is cleared on
 *     `stream` at the start of each call.  Calls that overlap on the GPU
 *     (different streams, no ordering between them) race on the buffer and
 *     give wrong results: order them, or use topk_bucketed with one workspace
 *     per stream.
 * Results are identical to topk_bucketed's. */
#define TOPK_NOALLOC_SCRATCH_BYTES (32u << 20)
int topk_bucketed_noalloc(const float *scores_dev, int64_t rows, int64_t n, int k, int b, int kb,
                          float *out_vals_dev, int32_t *out_idx_dev, void *stream);

/* ------------------------------------------------------------------------
 * The decoding step around the selections.  The pages leave these parts to
 * the model that calls the selector: the key-value cache that the decode
 * selector scores, the attention over the cache or over the selected
 * positions, and beam search over the vocabulary next to sampling.
 * ------------------------------------------------------------------------ */

#define TOPK_CACHE_BF16 0 /* rows of bf16 values */
#define TOPK_CACHE_E4M3 1 /* rows of 8-bit codes (4 exponent bits, 3 mantissa bits) and a float32 scale */

/* One paged cache tensor (the keys, or the values) in device memory:
 * element [page][head][offset][i], i < d contiguous, the other three with any
 * strides.  Token t of a sequence whose row of the block table is T lies on
 * page T[t / page_size] at offset t % page_size; pages are given out by the
 * caller.  With page_size = n and one page per sequence a contiguous
 * [batch][kv_heads][n][d] cache, as score_topk reads it, is such a tensor.
 * d is 64, 128 or 256 (else TOPK_EUNSUPPORTED); data is 16-byte aligned and
 * every stride a multiple of 16 bytes.  An E4M3 row (page, head, offset) with
 * scale s holds the values code_i * s; scales are read as any floats, and
 * cache_write writes powers of two. */
typedef struct {
    void *data;
    float *scale;            /* E4M3: [pages][kv_heads][page_size] with the strides below; else ignored */
    int64_t pages;           /* pages of the tensor, < 2^31 */
    int kv_heads;
    int page_size;           /* tokens per page, any number >= 1 */
    int d;
    int type;                /* TOPK_CACHE_BF16 or TOPK_CACHE_E4M3 */
    int64_t page_stride, head_stride, token_stride;                   /* elements of data */
    int64_t scale_page_stride, scale_head_stride, scale_token_stride; /* elements of scale */
} topk_cache;

/* Writes the keys and values of new tokens into their slots.
 *   k_dev, v_dev  bf16; row (token, head) starts at token * *_token_stride +
 *                 head * *_head_stride elements and holds d values; 16-byte
 *                 aligned, strides multiples of 8 elements.
 *   slots_dev     [tokens] int64: page * page_size + offset.  A negative slot
 *                 is skipped (padding); one behind the last page is skipped
 *                 and sets TOPK_DEV_BAD_INDEX.  The slots of one call must be
 *                 distinct (a repeated one ends up holding either row, or a
 *                 mix of both).
 *   k_cache, v_cache  of the same shape and type (host structures).
 * BF16 rows are copied.  An E4M3 row x becomes code_i = x_i / 2^e rounded to
 * nearest even and scale 2^e, with the smallest e >= -127 for which max|x_i|
 * <= 448 * 2^e (e = 0 for a row of zeros): the values read back are within
 * 2^-4 of x_i relatively, or within 2^(e-10) where that is more.  A row that
 * holds a NaN or an infinity reads back as NaN throughout.  Other slots are
 * left as they were.  Asynchronous on `stream`; no workspace. */
int cache_write(const uint16_t *k_dev, int64_t k_token_stride, int64_t k_head_stride,
                const uint16_t *v_dev, int64_t v_token_stride, int64_t v_head_stride,
                int64_t tokens, const topk_cache *k_cache, const topk_cache *v_cache,
                const int64_t *slots_dev, void *stream);

/* Reads the first n tokens of every sequence back as contiguous bf16 rows:
 * out[b][h][t] for t < min(n, seq_lens[b]), zeros behind.  With batch *
 * kv_heads rows of [n x d] keys this is what score_topk and score_rerank take,
 * for sequences of n tokens or more: they know no lengths, and a row of zeros
 * behind a sequence's end scores 0, above every key of negative score.  Read and
 * select from sequences of unlike lengths in calls of their own.
 * An E4M3 value is code * scale in float32, rounded to bf16 (exact for the scales
 * of cache_write; others round twice).
 *   block_table_dev  [batch] rows of table_width int32 page numbers, row b at
 *                    b * table_stride.  Entries behind a sequence's last page
 *                    are not read; a page that does not exist reads as zeros
 *                    and sets TOPK_DEV_BAD_INDEX.
 *   seq_lens_dev     [batch] int32; a negative length is 0, one above
 *                    table_width * page_size is held to that and sets
 *                    TOPK_DEV_BAD_INDEX.
 *   out_dev          [batch x kv_heads x n x d] bf16, 16-byte aligned. */
int cache_read(const topk_cache *cache, const int32_t *block_table_dev, int64_t table_stride,
               int table_width, const int32_t *seq_lens_dev, int64_t batch, int64_t n,
               uint16_t *out_dev, void *stream);

/* Attention of one new token per sequence: out[b][h] = sum_j p_j V_j with
 * p = softmax over j of scale * q[b][h] . K_j, and lse[b][h] = log sum_j
 * exp(scale * q[b][h] . K_j), over the tokens j < seq_lens[b], or over the
 * listed positions.  Query head h reads key-value head h / (heads / kv_heads).
 * Products, sums and softmax are float32.  A weight enters its product with V
 * with 16 significant bits beside BF16 values.  Beside E4M3 ones it is p_j times
 * the row's scale, with 11 significant bits down to 2^-24 of the largest such
 * product of the head, and within 2^-35 of that below.  out is rounded once to
 * bf16.  Equal calls give equal bits.
 *   q_dev         bf16, sequence b at b * q_stride elements, [heads x d]
 *                 contiguous there; 16-byte aligned, q_stride a multiple of 8.
 *   heads         a multiple of kv_heads.
 *   block_table_dev, table_stride, table_width, seq_lens_dev  as in
 *                 cache_read.  A token whose page does not exist is left out
 *                 and sets TOPK_DEV_BAD_INDEX.
 *   positions_dev NULL for the whole sequence (lists = c = 0), else int32
 *                 [batch x lists x c]: list l serves the query heads h with
 *                 h / (heads / lists) = l; lists is a multiple of kv_heads
 *                 that divides heads.  These are the indices score_topk or
 *                 score_rerank return.  A negative position is an empty slot,
 *                 one at or behind seq_lens[b] is left out (at or behind
 *                 table_width * page_size it also sets TOPK_DEV_BAD_INDEX);
 *                 a position listed twice counts twice.
 *   table_width   times page_size, or c, is taken for the length of the longest
 *                 sequence or list (the host cannot see seq_lens): many short
 *                 ones are spread otherwise than few long ones, and under a
 *                 table far wider than they need short ones take up to twice
 *                 the time (600 of up to 128 tokens, 82 us instead of 46).
 *   scale         scale * log2(e) finite in float32 (else TOPK_EINVAL).
 *   out_dev       [batch x heads x d] bf16; out_lse_dev NULL or [batch x
 *                 heads] float32.
 * A head with no token to attend to, or whose scores are all -inf, gives
 * zeros and an lse of -inf.  An infinite V_j makes its columns infinite (NaN
 * where infinities of both signs meet, or where p_j is below 2^-100 of the
 * largest p).  BF16 values above 2^119 / seq_lens[b] may overflow the sums, in
 * which weights are relative to a score up to 2^8 below the largest; E4M3 codes
 * take scales from 2^-127 on, and any whose product with 448 is finite.
 * The workspace holds paged_attention_workspace_bytes(...) bytes, 16-byte
 * aligned, on the device of the call.  Its first TOPK_DECODE_TICKET_BYTES must
 * be zero before its first use and are zero again after every call; the rest is
 * scratch.  It serves any later call of this operator or of topk_beam (not of
 * the selections above).  Calls that overlap on the GPU must not share one, nor
 * may a call be queued with the workspace of a topk_beam that another host
 * thread is queueing on the same stream: that is several launches. */
#define TOPK_DECODE_TICKET_BYTES 16384
int paged_attention(const uint16_t *q_dev, int64_t q_stride, int64_t batch, int heads,
                    const topk_cache *k_cache, const topk_cache *v_cache,
                    const int32_t *block_table_dev, int64_t table_stride, int table_width,
                    const int32_t *seq_lens_dev, const int32_t *positions_dev, int lists, int c,
                    float scale, uint16_t *out_dev, float *out_lse_dev, void *workspace_dev,
                    size_t workspace_bytes, void *stream);

/* Bytes of workspace of a paged_attention call on the current device (lists =
 * 0 without positions); 0 for invalid sizes. */
size_t paged_attention_workspace_bytes(int64_t batch, int heads, int lists, int d);

#define TOPK_BEAM_MAX 128 /* largest number of beams, and of continuations kept, per sentence */

/* One step of beam search: the k best continuations of every sentence's beams.
 * Continuation (i, t) is worth s_i + x_it - log sum_t' exp(x_it').
 *   logits_dev      [batch x beams x n] float32.
 *   beam_scores_dev [batch x beams] float32 s_i; -inf marks a beam that has
 *                   ended or does not exist yet: its logits are not looked at.
 *   k               1 <= k <= 128, beams <= 128 (else TOPK_EUNSUPPORTED); twice
 *                   the beams leaves enough when every beam may end.
 *   out_scores_dev  [batch x k] float32 values, best first; out_parent_dev
 *                   [batch x k] int32 beams; out_token_dev [batch x k] int32.
 * Continuations rank by value, compared in 64 bits (NaN first), then by lower
 * beam, larger logit, lower token.  A beam's log-sum-exp is within 2^-18 (n up
 * to 2^18), and in one call the same for equal logits wherever they lie: beams
 * of equal logits and scores tie exactly, and only continuations of unlike
 * beams whose values are within 2^-17 of each other may change places.  A logit
 * of -inf gives no continuation; a beam whose logits hold a NaN or +inf has the
 * value NaN for all of its own.
 * When there are fewer than k, the remaining slots hold -inf, -1, -1.
 * Where more than 512 continuations are within about 2^-7, relatively, of the
 * k-th best (many beams and a large k, or logits nearly all equal), they are
 * picked one by one: 16 beams with k = 32 and all logits equal take 0.6 ms, 128
 * beams with k = 128 take 14 ms.
 * Workspace: topk_beam_workspace_bytes(...), shared with paged_attention on
 * the terms given there. */
int topk_beam(const float *logits_dev, const float *beam_scores_dev, int64_t batch, int beams,
              int64_t n, int k, float *out_scores_dev, int32_t *out_parent_dev,
              int32_t *out_token_dev, void *workspace_dev, size_t workspace_bytes, void *stream);

/* topk_beam on bfloat16 logits (raw 16-bit patterns, widened exactly). */
int topk_beam_bf16(const uint16_t *logits_dev, const float *beam_scores_dev, int64_t batch,
                   int beams, int64_t n, int k, float *out_scores_dev, int32_t *out_parent_dev,
                   int32_t *out_token_dev, void *workspace_dev, size_t workspace_bytes,
                   void *stream);

/* Bytes of workspace of a topk_beam or topk_beam_bf16 call on the current
 * device; 0 for invalid sizes. */
size_t topk_beam_workspace_bytes(int64_t batch, int beams, int64_t n, int k);

/* Brings per-beam states into the order topk_beam chose: for every tensor s
 * and new beam (b, j), row dst[s][b][j] = row src[s][b][parents[b][j]].  A
 * parent of -1 (a slot topk_beam left empty) gives a row of zeros; any other
 * parent outside [0, beams) does too and sets TOPK_DEV_BAD_INDEX.  Page tables
 * are such states: beams of one parent then share pages, and of a page that is
 * not full each needs a copy before cache_write puts its next token there (a row
 * of zeros names page 0: the beam it stands for is to write nowhere).
 *   src, dst     HOST arrays of `count` device pointers, 1 <= count <= 256
 *                (else TOPK_EUNSUPPORTED); any alignment.
 *   row_bytes    HOST array [count]: bytes of one beam's row, contiguous; src[s]
 *                holds batch * beams rows, dst[s] batch * k.
 *   parents_dev  [batch x k] int32.
 * A destination that overlaps a source or another destination is refused
 * (TOPK_EINVAL).  Asynchronous on `stream`; no workspace. */
int beam_reorder(const void *const *src, void *const *dst, const int64_t *row_bytes, int count,
                 int64_t batch, int beams, int k, const int32_t *parents_dev, void *stream);

/* Self-test of the bounded waits (no counterpart in the paper): one thread
 * waits, for at most limit_ns nanoseconds (1e3 .. 2e9, else TOPK_EINVAL), on
 * a barrier that nothing completes, gives up and records TOPK_DEV_WAIT_TIMEOUT
 * in the device status, exactly as an expired wait of a selection kernel does.
 * The GPU neither faults nor hangs and the context stays usable; it lets a
 * caller check its error handling for expired waits.  Asynchronous on
 * `stream`. */
int topk_selftest_wait_timeout(unsigned long long limit_ns, void *stream);

/* Human-readable name of a topk_status value (static string). */
const char *topk_status_string(int status);

/* Reads and clears the device-side status word of the current device: 0 when
 * no bounded wait has expired since the last read, else a bit set of
 * TOPK_DEV_* codes.  Synchronises the device. */
int topk_device_status(int *status_out);

#define TOPK_DEV_WAIT_TIMEOUT 1 /* a bulk-copy wait in a streaming kernel expired */
#define TOPK_DEV_BAD_INDEX 2    /* an index out of range (of a candidate, position, slot, page, length or
                                beam) was skipped; see each call */
#define TOPK_DEV_DRAIN_TIMEOUT 4 /* after an expired wait, the kernel's wait for its own bulk copies
                                    still in flight expired too: the kernel returned while a copy
                                    may still have been writing to its shared memory, so the
                                    context must be treated as unusable (reset or exit) */

#ifdef __cplusplus
}
#endif

#endif /* TOPK_B200_H */
