/*
 * libfprefill: block-sparse causal prefill attention in the FlashPrefill
 * style (instantaneous block-pattern discovery, max-based dynamic threshold,
 * index compaction, sparse attention with block-mean correction) for one
 * NVIDIA GB300 GPU (sm_103a).
 *
 * Sources: the FlashPrefill V1 summary ("FlashPrefill: long-context
 * acceleration 28x", mhpn.cn; sections 3.1-3.3), the FlashPrefill V2 paper
 * reading (inkeast.github.io MessageDaily; sections 4, 4.1-4.3) and the
 * FlashPrefill V2 popular article (animattoys.com; sections on mean
 * correction, PackGQA, FP8, the CSR index and paged KV).
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 *  - The caller owns and allocates every buffer; the library allocates
 *    nothing.  Pointers named "device" must be device memory, 16-byte aligned.
 *    The varlen descriptors (cu_seqlens_q, seqlens_k, q_start_pos) are small
 *    HOST arrays read synchronously during the call.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream).  Argument errors are returned synchronously, before anything
 *    is enqueued.  Errors found by a kernel (a page-table entry out of range,
 *    a bounded wait that timed out) are recorded in a status word inside the
 *    workspace (the first error stays, but for a wait that ran out in
 *    fp_cache_attn) and read back with fp_device_status().
 *  - Every workspace is an opaque device buffer of at least the size its
 *    *_workspace_size() query returns.  Its first 256 bytes are a header
 *    holding the status word: zero them once (fp_reset_status) before first
 *    use.  One workspace may serve all stages in turn (take the largest
 *    size); calls that overlap on the GPU must not share one.
 *  - Query rows: token-major [total_q, h_q, d]; request r owns rows
 *    cu_seqlens_q[r] .. cu_seqlens_q[r+1]-1; its query i sits at absolute
 *    position q_start_pos[r] + i and attends causally to keys 0..position.
 *    seqlens_k[r] must equal q_start_pos[r] + (its query count): a prefill
 *    (q_start_pos = 0) or a chunk of a chunked prefill whose earlier tokens
 *    are already in the cache.  q_start_pos must be a multiple of the block.
 *  - Paged KV [V2 paper reading 4.3; V2 article, paged KV address rule]:
 *    k_cache / v_cache are [num_pages, page_size, h_kv, d] (contiguous); the
 *    key at position t of request r lives in physical page
 *    block_table[r * max_pages_per_seq + t / page_size], slot t % page_size.
 *    page_size must divide 128 or be a multiple of 128, and be >= 16.
 *  - Blocks: B = params.block = 128 tokens (query and key blocks alike).
 *    Request r has nqb_r = ceil(lq_r / B) query blocks starting at absolute
 *    block I0_r = q_start_pos[r] / B, and nkb_r = ceil(seqlens_k[r] / B) key
 *    blocks.
 *  - Rows: the index and the score map are organised in rows (r, i, h) -- a
 *    query block i of request r and a kv head h -- ordered request-major,
 *    then query block, then kv head:  row = rowbase_r + i * h_kv + h, with
 *    rowbase_r = sum_{r' < r} nqb_r' * h_kv.  R = total rows.  The absolute
 *    block of the row is I = I0_r + i; its causal key blocks are J = 0..I.
 *  - Pooled means: [sum_r nkb_r, h_kv, d] fp32; request r's blocks start at
 *    kbbase_r = sum_{r' < r} nkb_r'.
 *  - Score map: fp32, row (r, i, h) holds I + 1 values (J = 0..I) at offset
 *      scorebase_r + h_kv * (i * (I0_r + 1) + i * (i - 1) / 2)
 *                  + h * (I0_r + i + 1),
 *    scorebase_r = sum_{r' < r} h_kv * (nqb * (I0 + 1) + nqb * (nqb - 1) / 2).
 *    fp_score_size() returns the total.
 *  - CSR index [V2 paper reading 4 "CSR"; V1 3.3 "physical jump"]: row_ptr
 *    int32 [R + 1], col_idx int32 [nnz] listing the kept key blocks J of each
 *    row in ascending order.  col_capacity must be >= fp_score_size() (the
 *    causal upper bound), so selection never needs a host synchronisation.
 *  - Supported: d = 128, B = 128, h_q a multiple of 2*h_kv (query heads are
 *    processed in pairs of the same group), batch <= FP_MAX_BATCH.  Other
 *    shapes return FP_ERR_UNSUPPORTED.
 */
#ifndef FPREFILL_H
#define FPREFILL_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP_MAX_BATCH 128
#define FP_MAX_KEY_BLOCKS 16384

typedef enum {
    FP_OK = 0,
    FP_ERR_INVALID = 1,        /* bad argument (null pointer, inconsistent lengths, alignment) */
    FP_ERR_UNSUPPORTED = 2,    /* a shape or option this build does not implement */
    FP_ERR_WORKSPACE = 3,      /* workspace missing or smaller than required */
    FP_ERR_CUDA = 4,           /* a CUDA runtime call failed (launch, copy) */
    FP_ERR_DEVICE_BOUNDS = 5,  /* device status: a page-table entry outside [0, num_pages), or an
                                  index entry J outside [0, I] (its tile is read as zeros) */
    FP_ERR_TIMEOUT = 6         /* device status: a bounded wait inside a kernel gave up */
} fp_status;

typedef enum {
    FP_BF16 = 0,   /* q, k_cache, v_cache hold bf16 */
    FP_E4M3 = 1    /* q, k_cache, v_cache hold fp8 e4m3 codes; value = code * scale[head] */
} fp_dtype;

typedef struct {
    int block;            /* B, tokens per block: must be 128 */
    int sink_tokens;      /* blocks holding any of the first sink_tokens are always kept (256) */
    int local_tokens;     /* the ceil(local_tokens / B) blocks ending at I are always kept (512) */
    float alpha;          /* keep J when Score[I,J] >= alpha * max_J Score[I,J] (0.1) */
    float softmax_scale;  /* logit scale; <= 0 selects 1/sqrt(d) */
    int mean_correction;  /* 1: skipped blocks J < I add their block-mean term */
    int kv_splits;        /* attention only: split each row's key list into this many
                             parts merged by their LSE (split-KV); 0 chooses (more
                             parts when the problem has too few work units to fill
                             the GPU), 1 never splits; at most FP_MAX_KV_SPLITS */
    int select_rule;      /* fp_select rule (fp_select_rule); sink and local blocks are
                             kept under every rule */
    int top_k;            /* FP_SELECT_TOPK: blocks kept per row (>= 1) */
    float top_p;          /* FP_SELECT_TOPP: share of the row's score mass kept, (0, 1] */
    int score_mode;       /* fp_discover: FP_SCORE_PACKED or FP_SCORE_HEAD_UNION */
    int p_terms;          /* FP_E4M3 attention only: the softmax weights P enter the PV
                             product as 1 e4m3 term, e4m3(256 p) [V2 paper reading 4.2 (4)],
                             or 2: that term plus the residual e4m3(256 p - term) in a second
                             PV pass, which cuts the weights' rounding from 2^-4 to about
                             2^-8 relative; 0 means 1 */
} fp_params;

/* Score modes of fp_discover.  PACKED is the reading of the V1 summary 3.1
 * with PackGQA (the g heads x B queries of a group are one set of packed
 * rows); HEAD_UNION is the alternative: each query head's row is normalised
 * on its own and the row keeps the maximum over the group's heads, so the
 * threshold keeps the union of the heads' own selections. */
typedef enum { FP_SCORE_PACKED = 0, FP_SCORE_HEAD_UNION = 1 } fp_score_mode;

/* Selection rules of fp_select.  THRESHOLD is the method's rule [V1 summary
 * 3.2]; TOPK and TOPP are the alternatives it is compared with [V1 summary
 * 4.4], kept here as ablations. */
typedef enum {
    FP_SELECT_THRESHOLD = 0,  /* Score >= alpha * max_J Score */
    FP_SELECT_TOPK = 1,       /* the top_k highest scores; among equal scores the lower J */
    FP_SELECT_TOPP = 2        /* the highest scores, down to the largest t such that the
                                 scores >= t hold at least top_p of the row's total */
} fp_select_rule;

#define FP_MAX_KV_SPLITS 32

typedef struct {
    int batch;
    int h_q;
    int h_kv;
    int d;
    fp_dtype dtype;
    /* HOST arrays */
    const int *cu_seqlens_q;      /* [batch + 1], cu_seqlens_q[0] = 0, non-decreasing */
    const int *seqlens_k;         /* [batch] */
    const int *q_start_pos;       /* [batch] */
    /* DEVICE arrays */
    const void *q;                /* [total_q, h_q, d] at the strides below */
    long long q_stride_tok;       /* elements between consecutive tokens (>= h_q * d) */
    long long q_stride_head;      /* elements between consecutive heads (>= d) */
    const void *k_cache;          /* [num_pages, page_size, h_kv, d] */
    const void *v_cache;
    int page_size;
    int num_pages;
    const int *block_table;       /* [batch, max_pages_per_seq] physical page ids */
    int max_pages_per_seq;
    const float *q_scale;         /* [h_q]   FP_E4M3 only (may be NULL for FP_BF16) */
    const float *k_scale;         /* [h_kv]  FP_E4M3 only */
    const float *v_scale;         /* [h_kv]  FP_E4M3 only */
    int v_layout;                 /* fp_v_layout of v_cache (0: token-major, like k_cache) */
} fp_problem;

/* Layout of the value cache [V2 popular article, FP8 passage: a value cache
 * stored by rows or by columns].  TOKEN_MAJOR: [num_pages, page_size, h_kv, d],
 * the layout of k_cache.  DIM_MAJOR: [num_pages, h_kv, d, page_size], each
 * (page, head, d) holding the page's tokens contiguously; page_size must be a
 * multiple of 64 for FP_BF16 and of 128 for FP_E4M3 (FP_ERR_UNSUPPORTED
 * otherwise).  The result is the same either way (up to the summation order
 * of the PV product); the attention takes DIM_MAJOR tiles as K-major operands
 * and TOKEN_MAJOR ones as MN-major operands, so neither is transposed on chip. */
typedef enum { FP_V_TOKEN_MAJOR = 0, FP_V_DIM_MAJOR = 1 } fp_v_layout;

/* Defaults of the pages: B=128, sink 256, local 512, alpha 0.1, 1/sqrt(d),
 * mean correction on [V2 paper reading, section 4 configuration]; kv_splits 0
 * (chosen by the library); the threshold rule (top_k 0, top_p 0: unused);
 * p_terms 1 (the pages' e4m3 P). */
fp_params fp_default_params(void);

/* Sizes derived from the host descriptors (element counts, not bytes). */
long long fp_num_rows(const fp_problem *p, const fp_params *prm);        /* R */
long long fp_num_key_blocks(const fp_problem *p, const fp_params *prm);  /* sum_r nkb_r */
long long fp_score_size(const fp_problem *p, const fp_params *prm);      /* floats in the score map */
long long fp_total_q(const fp_problem *p);                               /* cu_seqlens_q[batch] */

/* Offsets of the score-map rows (the closed form above), for callers that
 * index the score map or the dense mask: offsets (HOST int64, n entries)
 * receives the offset of row k = 0 .. R-1 in row order, then
 * offsets[R] = fp_score_size().  Host-only: enqueues nothing.  Returns R + 1,
 * or -1 when an argument is invalid or n < R + 1. */
long long fp_score_offsets(const fp_problem *p, const fp_params *prm, long long *offsets, long long n);

/* ---------------------------------------------------------------------------
 * fp_discover -- instantaneous pattern discovery
 * [V1 3.1 key pooling + query-block scoring; V2 4.1 block means of K and V]
 *
 *   k_mean, v_mean (device, fp32 [sum_r nkb_r, h_kv, d]): block means over the
 *     n_J = min(B, lk - J*B) tokens of each key block (FP8: of the
 *     dequantised values).
 *   score (device, fp32, fp_score_size() floats, layout above): for row
 *     (r, i, h) with absolute query block I, each of the g*B packed query rows
 *     (g = h_q / h_kv heads of the group x the block's queries) contributes
 *     exp(s_J - max_J' s_J') to S'[J], s_J = scale * q . k_mean_J for J <= I;
 *     Score[I,J] = S'[J] / max_J' S'[J'] (so each row peaks at exactly 1).
 *     FP_SCORE_HEAD_UNION: the same per query head (its B queries alone),
 *     and Score[I,J] = max over the group's heads of those rows (still
 *     peaking at 1); rows over 12480 key blocks: FP_ERR_UNSUPPORTED.
 *   ws: fp_discover_workspace_size() bytes (status header only).
 * ------------------------------------------------------------------------- */
size_t fp_discover_workspace_size(const fp_problem *p, const fp_params *prm);
fp_status fp_discover(const fp_problem *p, const fp_params *prm, float *k_mean, float *v_mean,
                      float *score, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * fp_select -- max-based dynamic threshold + sink/local forcing + compaction
 * [V1 3.2 threshold alpha * max_{J<=I} Score[I,J], sink and local safety net;
 *  V1 3.3 compaction of kept indices; V2 4 CSR index]
 *
 *   keep[I,J] = sel(I,J)  or  J * B < sink_tokens  or  J >= I - ceil(local_tokens / B) + 1
 *   sel: FP_SELECT_THRESHOLD  Score[I,J] >= alpha * max_J Score[I,J];
 *        FP_SELECT_TOPK  J is among the top_k highest scores of the row
 *                        (equal scores: lower J first);
 *        FP_SELECT_TOPP  Score[I,J] >= t, t the largest value such that the
 *                        scores >= t sum to at least top_p * sum_J Score[I,J].
 *   row_ptr (device int32 [R + 1]), col_idx (device int32, col_capacity
 *   entries; the first nnz are written), nnz_dev (device int32 [1]).
 *   dense_mask_opt (device uint8, fp_score_size() bytes, may be NULL): the
 *   keep decision of every score entry, at the score map's offsets.
 *   ws: fp_select_workspace_size() bytes.
 * ------------------------------------------------------------------------- */
size_t fp_select_workspace_size(const fp_problem *p, const fp_params *prm);
fp_status fp_select(const fp_problem *p, const fp_params *prm, const float *score, int *row_ptr,
                    int *col_idx, long long col_capacity, int *nnz_dev,
                    unsigned char *dense_mask_opt, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * fp_discover_select -- fp_discover and fp_select in one call
 * [V1 summary 3.1-3.3 run back to back]
 *
 * Same results as fp_discover followed by fp_select with the same params (the
 * same k_mean / v_mean, score map and CSR index).  With the threshold rule on
 * rows the tensor-core score kernel takes, that kernel decides each row and
 * lists its kept blocks itself, so the score map is neither written (unless
 * score_opt is given) nor read back.
 *   score_opt (device fp32, fp_score_size() floats, may be NULL).
 *   row_ptr, col_idx, col_capacity, nnz_dev as fp_select.
 *   ws: fp_discover_select_workspace_size() bytes.
 * ------------------------------------------------------------------------- */
size_t fp_discover_select_workspace_size(const fp_problem *p, const fp_params *prm);
fp_status fp_discover_select(const fp_problem *p, const fp_params *prm, float *k_mean, float *v_mean,
                             float *score_opt, int *row_ptr, int *col_idx, long long col_capacity,
                             int *nnz_dev, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * fp_sparse_attn -- block-sparse attention with block-mean correction
 * [V2 paper reading 4.1 (mean correction), 4.2 (PackGQA, warp
 *  specialisation, FP8), 4.3 (paged KV through the page table)]
 *
 * For query position p in absolute block I of row (r, i, h):
 *   O = [ sum_{J in row} sum_{t in J, t <= p} e^{s_t - m} v_t
 *         + mc * sum_{J < I, J not in row} n_J e^{scale q.kmean_J - m} vmean_J ]
 *       / [ the same sums without v ],   s_t = scale q.k_t,
 *   mc = params.mean_correction, m a common shift; LSE = m + ln(denominator).
 *   row_ptr/col_idx: a CSR index as produced by fp_select (ascending J <= I).
 *   k_mean/v_mean: as produced by fp_discover (read only when mc = 1).
 *   out (device bf16 [total_q, h_q, d], contiguous).
 *   lse_opt (device fp32 [h_q, total_q], natural log; may be NULL).
 *   ws: fp_attn_workspace_size() bytes (work schedule, the tensor-core copies
 *   of the block means, and with split-KV the fp32 partial outputs and LSEs).
 * A row with no term at all (an empty index row, no correction) yields O = 0.
 * The mean tokens' logits run on the tensor cores: bf16 problems take the key
 * means as fp16 (a power-of-two scale per 128-block tile and kv head) against
 * the queries in fp16 (exact under a power-of-two scale per row), so a mean
 * logit errs by about 2^-12 relative; e4m3 problems take them as two e4m3
 * terms.
 *
 * Split-KV (the kept-count load balancing of the V2 popular article, "KV
 * split", for rows too long for the number of rows): with S = the split count
 * chosen from params.kv_splits, each row's terms (kept blocks, then mean
 * tiles) are cut into S consecutive parts of equal size.  Part s yields
 * O_s, LSE_s over its own terms, and O = sum_s e^{LSE_s - LSE} O_s with
 * LSE = ln sum_s e^{LSE_s}: the same O up to rounding.  The workspace size
 * depends on the split count, so query it with the same params.
 * ------------------------------------------------------------------------- */
size_t fp_attn_workspace_size(const fp_problem *p, const fp_params *prm);
/* The split count S the attention calls use for these params (>= 1), or -1
 * on an argument error. */
int fp_attn_kv_splits(const fp_problem *p, const fp_params *prm);
fp_status fp_sparse_attn(const fp_problem *p, const fp_params *prm, const int *row_ptr,
                         const int *col_idx, const float *k_mean, const float *v_mean,
                         void *out, float *lse_opt, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * fp_sparse_attn_noalloc -- fp_sparse_attn for callers that cannot allocate
 * (no counterpart in the pages: an interface addition of this library).
 *
 * For callers that have no way to provide a device workspace: a plugin whose
 * host framework owns all device memory and hands it none, or a serving loop
 * held to a fixed device-memory budget where allocating mid-request could fail
 * or stall the device.  The function allocates nothing: its scratch is one
 * file-scope device array of FP_NOALLOC_SCRATCH_BYTES, reserved on every GPU
 * that loads the library until the process exits.  The caller still provides
 * the inputs and the outputs.
 *
 *   Arguments and results as fp_sparse_attn, without ws / ws_bytes; rows are
 *   split only when params.kv_splits asks for it (0 means no split here).
 *   status_dev_opt (device int32 [1], may be NULL): receives this call's
 *     device status word (FP_OK or an fp_status code), in stream order after
 *     the kernels -- the scratch itself is not visible to the caller.
 *   Returns FP_ERR_WORKSPACE when the problem needs more scratch than
 *     FP_NOALLOC_SCRATCH_BYTES (compare fp_attn_workspace_size()), before
 *     touching the GPU; other argument errors as fp_sparse_attn.
 *   Every call looks up the array's device address in the caller's current
 *     context (nothing is cached, so non-primary contexts and a device reset
 *     between calls are fine).  The first call in a context may load the
 *     library's device code into it: make that first call before any stream
 *     capture.
 *   Every call on a device shares the one array, and the array keeps the last
 *   call's contents (the call clears what must start at zero).  Calls that
 *   overlap on the GPU -- on different streams, or from different threads --
 *   race on it: serialise them.
 * ------------------------------------------------------------------------- */
#define FP_NOALLOC_SCRATCH_BYTES (8u << 20)
fp_status fp_sparse_attn_noalloc(const fp_problem *p, const fp_params *prm, const int *row_ptr,
                                 const int *col_idx, const float *k_mean, const float *v_mean,
                                 void *out, float *lse_opt, int *status_dev_opt, void *stream);

/* ---------------------------------------------------------------------------
 * fp_dense_attn -- the same kernel keeping every causal block, no correction
 * (the in-house dense baseline [V2 paper reading 5.3, 5.6]).  Same arguments
 * as fp_sparse_attn without the index and the means.
 * ------------------------------------------------------------------------- */
fp_status fp_dense_attn(const fp_problem *p, const fp_params *prm, void *out, float *lse_opt,
                        void *ws, size_t ws_bytes, void *stream);

/* ===========================================================================
 * Serving operators: page tables built on the GPU, a K/V cache held in 4 bits,
 * and attention over it at any position (no counterpart in the pages: what a
 * server runs beside the prefill above).
 *
 * Lengths, tables and slot maps are DEVICE arrays here, read when the kernels
 * run, so a call captured into a CUDA graph replays on the lengths of the
 * moment.  Each call takes a `ws` of at least FP_WS_HEADER_BYTES whose first
 * word is the status (fp_reset_status, fp_device_status); what a kernel finds
 * wrong in device data is recorded there as FP_ERR_DEVICE_BOUNDS, the part
 * concerned is left out as described at each call, and nothing outside the
 * buffers is touched.
 *
 * Slots: the token at position t of request r is at slot
 *   block_table[r * max_pages_per_seq + t / page_size] * page_size + t % page_size
 * of a cache, whatever its type; a slot of -1 stands for a padding row.
 * page_size as above (it divides 128 or is a multiple of 128, >= 16) and
 * num_pages * page_size <= 2^31 - 1.
 * ========================================================================= */
#define FP_WS_HEADER_BYTES 256
#define FP_TABLES_MAX_BATCH 4096

/* ---------------------------------------------------------------------------
 * fp_page_tables -- block tables, lengths and slot maps of one step
 *
 * Request r has seqlens[r] tokens cached and brings new_lens[r] more.  With
 *   used_r = ceil(seqlens[r] / page_size)
 *   need_r = ceil((seqlens[r] + new_lens[r]) / page_size) - used_r
 *   off_r  = sum_{r' < r} need_r',   head = *free_head (0 when NULL):
 *   block_table[r][used_r + k] = free_pages[head + off_r + k],  k < need_r
 *   cu_seqlens_q[r] = sum_{r' < r} new_lens[r'],  seqlens_k[r] = seqlens[r] + new_lens[r]
 *   positions[cu_seqlens_q[r] + i] = seqlens[r] + i, slots[...] = that token's slot
 *   *free_next = head + sum_r need_r
 * positions and slots behind the last token, up to capacity, are 0 and -1.
 * The other entries of block_table stay as they are.
 * A request that cannot be served -- a negative length, more than 2^31 - 1
 * tokens or max_pages_per_seq pages, a free list or a capacity that does not reach --
 * is refused as a whole: it takes no page, seqlens_k[r] = seqlens[r], its
 * slots are -1 and its positions 0 (its rows stay counted in cu_seqlens_q
 * unless new_lens[r] < 0, and saturate at 2^31 - 1), and the status says so.  When free list or
 * capacity run out at some request, the later ones that need any are refused
 * too.  A page id outside [0, num_pages) in either list gives slots of -1 and
 * the status.
 * seqlens_k may be seqlens, and free_next free_head: the step then advances
 * them in place, whatever the capacity (and runs in one thread block, which is
 * for steps of few tokens: 524288 take 327 us, and 8 us with arrays apart).
 * ------------------------------------------------------------------------- */
typedef struct {
    int batch;                    /* 1 .. FP_TABLES_MAX_BATCH */
    int page_size, num_pages, max_pages_per_seq;
    int num_free;                 /* entries of free_pages */
    int capacity;                 /* entries of positions and slots (>= 1) */
    /* DEVICE int32 arrays, read */
    const int *seqlens;           /* [batch] */
    const int *new_lens;          /* [batch] */
    const int *free_pages;        /* [num_free] (may be NULL when num_free is 0) */
    const int *free_head;         /* [1], or NULL for 0 */
    /* DEVICE int32 arrays, written */
    int *block_table;             /* [batch, max_pages_per_seq], updated in place */
    int *cu_seqlens_q;            /* [batch + 1] */
    int *seqlens_k;               /* [batch] */
    int *positions;               /* [capacity], 16-byte aligned */
    int *slots;                   /* [capacity], 16-byte aligned */
    int *free_next;               /* [1] */
} fp_tables;
fp_status fp_page_tables(const fp_tables *t, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * The 4-bit cache
 *
 * For each token and kv head, K and V are cut into d / group groups of
 * consecutive dims; a group holds an f16 step s, an f16 minimum m and 4-bit
 * codes c, and stands for s * c + m.  data is [num_pages, h_kv, page_size / 16]
 * chunks; a chunk holds 16 tokens of one kv head, with n = 128 / group:
 *   bytes    0 .. 1023   K codes: token t's dim 32 q + 8 j + i (i < 8) is nibble
 *                        i of the 4 bytes at  64 t + 16 j + 4 q
 *   bytes 1024 .. 2047   V codes: token t's dim 32 y + 4 r + i (i < 4) is nibble
 *                        i of the 2 bytes at  512 (t / 8) + 64 r + 16 (t % 8 / 2) + 8 (t % 2) + 2 y
 *   then f16 [16][n]          K steps, and K minima
 *   then f16 [4][n][2][2]     V steps, and V minima: token t, group g at
 *                             [t % 8 / 2][g][t / 8][t % 2]
 * (nibble 0 is the low half of the first byte), which is the order in which
 * the attention's matrix instructions take them.
 * ------------------------------------------------------------------------- */
typedef struct {
    void *data;                   /* DEVICE, fp_qcache_bytes() bytes, 16-byte aligned */
    int num_pages, page_size;
    int h_kv;
    int d;                        /* must be 128 */
    int group;                    /* 32, 64 or 128 */
} fp_qcache;
/* Bytes of a chunk (2048 + 128 * n) and of the whole cache; 0 on an argument
 * error.  Host-only. */
size_t fp_qcache_chunk_bytes(const fp_qcache *c);
size_t fp_qcache_bytes(const fp_qcache *c);

/* fp_qcache_write -- quantise tokens into the cache
 *
 *   x' = x clamped to +-65504;  m = f16(min x');  s = f16(max(0, (max x' - m) / 15))
 *   c = min(15, max(0, rint((x' - m) * (1 / s))))   (0 where s = 0), in fp32.
 *   A NaN in a group makes its minimum NaN, so all of the group reads as NaN.
 *   k, v (device): row i, head h at  i * stride_tok + h * stride_head  elements
 *     (pointers and strides multiples of 16 bytes, stride_head >= d,
 *     stride_tok >= stride_head * (h_kv - 1) + d), dtype FP_BF16, or FP_E4M3
 *     codes times k_scale / v_scale [h_kv].
 *   slots (device int32 [rows]): where row i goes; -1 skips the row, another
 *     value outside the cache skips it and sets the status.  No slot may appear
 *     twice in one call (which row's parts it then holds is not defined).
 *   Slots that no row names stay as they are. */
typedef struct {
    int rows;                     /* >= 0 */
    fp_dtype dtype;
    void *k, *v;                  /* DEVICE; read by the write, written by the read */
    long long stride_tok, stride_head;      /* elements, of k and v alike */
    const int *slots;             /* [rows] slots in the 4-bit cache */
    const int *out_slots;         /* fp_qcache_read: [rows] target rows, or NULL (row i) */
    int out_rows;                 /* fp_qcache_read: rows of k and v */
    const float *k_scale, *v_scale;         /* [h_kv], FP_E4M3 only */
} fp_qcache_rows;
fp_status fp_qcache_write(const fp_qcache *c, const fp_qcache_rows *r, void *ws, size_t ws_bytes, void *stream);

/* fp_qcache_read -- bring tokens back into rows of bf16 or e4m3
 *
 *   k, v row out_slots[i] (row i when out_slots is NULL) = s * c + m of slot
 *   slots[i], rounded once to bf16, or to the e4m3 nearest to
 *   (s * c + m) / scale[head], saturated at 448.  With out_slots a slot map of
 *   a bf16 / e4m3 paged cache, its pages are what the prefill entry points read.
 *   Rows with a slot of -1 in either map are left as they were; another value
 *   out of range too, with the status set.  No row of k and v may be named twice. */
fp_status fp_qcache_read(const fp_qcache *c, const fp_qcache_rows *r, void *ws, size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * fp_qcache_attn -- attention over the 4-bit cache
 *
 * Request r owns query rows cu_seqlens_q[r] .. cu_seqlens_q[r+1]-1 (or, with
 * cu_seqlens_q NULL, max_q rows from r * max_q); its query i, of lq_r, sits at
 * position  p = seqlens_k[r] - lq_r + i  and attends keys 0 .. p: a decode
 * step (lq_r = 1), a run of drafted tokens, or a chunk, from any position.
 *   O = sum_t e^{s_t - m} v_t / sum_t e^{s_t - m},  s_t = scale q.k_t,  k_t and
 *   v_t the values the cache stands for;  LSE = m + ln(sum_t e^{s_t - m}).
 * A row with no key (an empty cache, or p < 0) yields O = 0 and LSE = -inf.
 *   out (device bf16 [total_q, h_q, d], contiguous), lse_opt (device fp32
 *   [h_q, total_q], natural log; may be NULL).
 *   Rows behind the last request, up to total_q, are left as they were.
 *   Queries are finite and below 2^115 in magnitude; a NaN or an infinity makes
 *   its row NaN.  So does a NaN that the cache keeps in a key that the row attends;
 *   in a value that it attends, it makes the dims of the NaN's group NaN.  Keys and
 *   values that a row does not attend -- later tokens of its request, what lies behind
 *   the last one -- may be anything.
 *   A page id outside [0, num_pages) reads as zeros; a length below 0, above
 *   max_pages_per_seq * page_size or above 2^31 - 64 reads as an empty cache; query rows outside
 *   [0, total_q) are left out: each sets the status.
 *   Logits, weights' sums and outputs are summed in fp32.  Weights enter the sum of
 *   values in fp16 (2^-11 of each; nothing below 2^-35 of the row's largest), and so do
 *   their products with a value's step (nothing below 2^-33 of the largest weight times
 *   the largest step of that group of dims, and a step to 2^-23 of that largest, among
 *   the tokens of the request up to its last row's).
 *   scratch: fp_qcache_attn_scratch_bytes() bytes (partial results of requests
 *   that several thread blocks share); it holds nothing between calls.  A call
 *   enqueues two kernels that hand these over: calls that may run at once, or
 *   that two threads enqueue on one stream with no lock around each call, need
 *   scratch of their own.
 *   max_q is the callers' bound of lq_r, which picks the kernel's tile: the
 *   result does not depend on it beyond rounding.  Long chunks (lq_r in the
 *   hundreds) are better served by fp_qcache_read and the prefill kernels.
 * ------------------------------------------------------------------------- */
typedef struct {
    int batch;                    /* 1 .. FP_TABLES_MAX_BATCH */
    int h_q;                      /* a multiple of the cache's h_kv */
    int total_q;                  /* rows of q and out (>= 0) */
    int max_q;                    /* >= 1 */
    fp_dtype dtype;               /* of q */
    const void *q;                /* DEVICE [total_q, h_q, d] at the strides below */
    long long q_stride_tok, q_stride_head;  /* elements, as in fp_qcache_rows */
    const float *q_scale;         /* [h_q], FP_E4M3 only */
    const int *cu_seqlens_q;      /* DEVICE [batch + 1], or NULL */
    const int *seqlens_k;         /* DEVICE [batch] */
    const int *block_table;       /* DEVICE [batch, max_pages_per_seq] */
    int max_pages_per_seq;
    float softmax_scale;          /* <= 0 selects 1/sqrt(d) */
} fp_qcache_query;
size_t fp_qcache_attn_scratch_bytes(const fp_qcache *c, const fp_qcache_query *q);
fp_status fp_qcache_attn(const fp_qcache *c, const fp_qcache_query *q, void *out, float *lse_opt, void *scratch,
                         size_t scratch_bytes, void *ws, size_t ws_bytes, void *stream);

/* ===========================================================================
 * The bf16 / e4m3 paged cache at any position: rotary positions, and keys and values
 * appended to the pages that the prefill entry points read, with values stored by tokens
 * (FP_V_TOKEN_MAJOR: a value cache stored by columns is the prefill's alone).  Lengths,
 * positions, slots and tables are DEVICE arrays, as for the 4-bit cache above.
 * ========================================================================= */

/* ---------------------------------------------------------------------------
 * Rotary positions
 *
 * The first `rot` dims of a head form pairs (a, b) of dims: (i, i + rot / 2) in the half
 * layout, (2 i, 2 i + 1) in the interleaved one, i < rot / 2.  With the angle
 * t = position * inv_freq[i],
 *   a' = scale * (a cos t - b sin t),   b' = scale * (b cos t + a sin t),
 * t negated for the inverse: with scale 1 the inverse undoes the rotation, and with any
 * scale it is the gradient.  Dims from `rot` on stay as they are (and are not scaled).
 * Angles are kept to 2^-32 of a turn at any int32 position (negative ones too), and rounded to
 * fp32, by 2^-26 of a turn at most, where their cosine and sine are taken; products and sums are
 * fp32, rounded once to the output's type.
 * ------------------------------------------------------------------------- */
typedef enum { FP_ROPE_HALF = 0, FP_ROPE_INTERLEAVED = 1 } fp_rope_layout;
typedef struct {
    int rot;                          /* even, 2 .. 128 */
    fp_rope_layout layout;
    float scale;                      /* multiplies cos and sin (1, or a long context's factor) */
    const unsigned long long *turns;  /* DEVICE [rot / 2], of fp_rope_turns */
} fp_rope_table;
/* turns[i] = the fraction of a turn that one position makes, inv_freq[i] / 2 pi modulo 1, in
 * units of 2^-64, for n frequencies in radians a position.  Host-only, host arrays.
 * FP_ERR_INVALID: a frequency that is not finite, or above 2^20 in magnitude. */
fp_status fp_rope_turns(const double *inv_freq, int n, unsigned long long *turns);

/* fp_rope -- rotate rows
 *
 *   x (device bf16): row i, head h at  i * stride_tok + h * stride_head  elements (pointer
 *     and strides multiples of 16 bytes, stride_head >= 128, stride_tok >= stride_head *
 *     (heads - 1) + 128); out the same with its own strides, bf16, or e4m3 codes of
 *     value / out_scale[head] (times the positive scale's rounded reciprocal; saturated at 448).
 *   out may be x itself, with like strides and type; otherwise they do not overlap. */
typedef struct {
    int rows;                         /* >= 0 */
    int heads;                        /* >= 1 */
    const void *x;                    /* DEVICE */
    long long x_stride_tok, x_stride_head;
    void *out;                        /* DEVICE */
    long long out_stride_tok, out_stride_head;
    fp_dtype out_dtype;
    const float *out_scale;           /* DEVICE [heads], FP_E4M3 only */
    const int *positions;             /* DEVICE [rows] */
    int inverse;                      /* 0 or 1 */
} fp_rope_rows;
fp_status fp_rope(const fp_rope_table *t, const fp_rope_rows *r, void *stream);

/* ---------------------------------------------------------------------------
 * fp_cache_append -- new tokens into the paged cache, rotated on the way
 *
 *   k and v rows i go to slot slots[i] of their caches; -1 skips the row, another value
 *   outside the cache skips it and sets the status.  No slot may appear twice in one call.
 *   Slots that no row names stay as they are.  With `rope`, k (and q) are rotated by
 *   positions[i].  q (may be NULL): every row i, whatever its slot, to row i of q_out, which
 *   may be q itself when both are bf16 with like strides.  bf16 in; out in the cache's type
 *   (q: q_dtype), rounded and scaled as fp_rope's.  Rows do not overlap the caches. */
typedef struct {
    void *k, *v;                      /* DEVICE [num_pages, page_size, h_kv, d], 16-byte aligned */
    int num_pages, page_size;         /* page_size as above; num_pages * page_size <= 2^31 - 1 */
    int h_kv;
    int d;                            /* must be 128 */
    fp_dtype dtype;
    const float *k_scale, *v_scale;   /* DEVICE [h_kv], FP_E4M3 only */
} fp_cache;
typedef struct {
    int rows;                         /* >= 0 */
    int h_q;                          /* heads of q (any number; 0 with q NULL) */
    const void *k, *v, *q;            /* DEVICE bf16, strides as fp_rope's */
    long long k_stride_tok, k_stride_head, v_stride_tok, v_stride_head, q_stride_tok, q_stride_head;
    void *q_out;                      /* DEVICE */
    long long q_out_stride_tok, q_out_stride_head;
    fp_dtype q_dtype;                 /* of q_out */
    const float *q_scale;             /* DEVICE [h_q], q_dtype FP_E4M3 only */
    const int *slots;                 /* DEVICE [rows] */
    const int *positions;             /* DEVICE [rows], with rope only */
} fp_cache_rows;
fp_status fp_cache_append(const fp_cache *c, const fp_rope_table *rope_opt, const fp_cache_rows *r, void *ws,
                          size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * fp_cache_attn -- attention over the paged cache at any position
 *
 *   As fp_qcache_attn, over the bf16 values, or the e4m3 codes times their head's scales, of
 *   `c`: the same query structure, results, refusals, status and scratch rules (with
 *   fp_cache_attn_scratch_bytes(); a call enqueues up to five kernels).  Queries are bf16 or
 *   e4m3, whatever the cache's type; scales are positive.
 *   A NaN in a query makes its row NaN, and so does one in a key that the row attends; what an
 *   infinity in either makes of the row is not defined.  In a value that a row attends, a NaN
 *   or an infinity makes that dim of the row one that is not finite.  Other rows and dims are
 *   what they would be without, and keys and values that a row does not attend may be
 *   anything.  Finite values, and logits, are below 2^100 in magnitude.
 *   Logits and sums are fp32.  Weights enter the sum of values rounded: to bf16 for a bf16 cache
 *   (2^-8 of each at most), to fp16 for an e4m3 one (2^-11 of each, or 2^-34 of the row's
 *   largest where that is more).  Weights below 2^-136 of the row's largest may count as none.
 *   bf16 queries of an e4m3 cache enter as two e4m3 terms under a power of two of the row: exact
 *   down to 2^-9 of the row's largest element, the rest to 2^-17 of it.
 *   Requests of many rows have bounded waits in their kernel, as the prefill's: one that runs
 *   out records FP_ERR_TIMEOUT, and until fp_reset_status such requests are left unwritten. */
size_t fp_cache_attn_scratch_bytes(const fp_cache *c, const fp_qcache_query *q);
fp_status fp_cache_attn(const fp_cache *c, const fp_qcache_query *q, void *out, float *lse_opt, void *scratch,
                        size_t scratch_bytes, void *ws, size_t ws_bytes, void *stream);

/* Zero the status header of a workspace (enqueued on stream). */
fp_status fp_reset_status(void *ws, void *stream);

/* Wait for `stream`, then read the status word of `ws` into *device_status
 * (an fp_status value; FP_OK when no kernel recorded an error): the first error
 * since the last reset, or FP_ERR_TIMEOUT over it where fp_cache_attn recorded
 * one -- its results are not defined then. */
fp_status fp_device_status(const void *ws, void *stream, int *device_status);

/* Time limit of every bounded wait inside the attention kernel, in
 * nanoseconds (default 200 ms; 0 restores the default).  A wait that runs out
 * records FP_ERR_TIMEOUT and the kernel returns instead of hanging.
 * fp_cache_attn gives waits that may span a request's keys 64 us more for
 * every 128 tokens that its table holds and every 128 rows, some 40 times what
 * they take: no length of a cache is too long for the limit. */
void fp_set_wait_limit_ns(unsigned long long ns);

/* Failure-path check of the bounded waits, with no GPU fault: launches one
 * thread that waits, through the prefill's bounded wait, on an mbarrier that
 * nothing arrives on, for limit_ns nanoseconds (1 .. 1e10), then one that does
 * so through fp_cache_attn's (and stops at once where the first has recorded
 * its wait).  FP_ERR_TIMEOUT lands in the status word of ws (over any other
 * error there), and the context stays usable: reset the status and carry on.
 * Returns FP_ERR_INVALID for a null ws or a limit out of range. */
fp_status fp_check_wait_timeout(void *ws, unsigned long long limit_ns, void *stream);

/* Static description of an fp_status value. */
const char *fp_status_string(fp_status s);

#ifdef __cplusplus
}
#endif
#endif /* FPREFILL_H */
