/*
 * mmvq_serve.h - C ABI of the operators of a step over many requests, in the
 * same library as mmvq.h and mmvq_decode.h (MI355X, gfx950).
 *
 * A program that serves many requests with one model calls, around the
 * products of mmvq.h and the operators of mmvq_decode.h:
 *   mmvq_kv_release   pages of finished requests and of dropped tokens back
 *                     to the free ones;
 *   mmvq_kv_plan      from the requests' lengths and new tokens: pages for
 *                     them, the descriptor arrays of mmvq_kv_batch, and each
 *                     row's request, position and cache slot;
 *   mmvq_embed        the tokens' rows of an embedding table in any weight
 *                     format;
 *   mmvq_lora         each request's low-rank adapter beside a projection
 *                     that all of them share;
 *   mmvq_sample       after the LM head: the next tokens, by temperature,
 *                     top-k, top-p and min-p, or the distributions that
 *                     these leave, which mmvq_verify_draft takes.
 * A request has a place s in 0..n_seqs-1 in all arrays of a step; row_seq[t]
 * is the place of the request that row t is of, -1 for rows of none.
 *
 * Conventions are those of mmvq_decode.h: data pointers are DEVICE pointers
 * owned by the caller, struct arguments are read on the host during the
 * call; everything is enqueued on `stream` and nothing synchronizes; the
 * library keeps no allocation and no state; return values are MMVQ_OK or
 * MMVQ_ERR_*, arguments are validated on the host before anything is
 * enqueued, and an invalid call enqueues nothing. Buffers that hold nothing
 * may be NULL. The kernels run on the stream's device (NULL: the current
 * device). Calls can be captured into HIP graphs. A workspace (16-byte
 * aligned, at least the bytes that its query names, fewer: MMVQ_ERR_SHAPE)
 * belongs to one call until the stream has passed it; calls that may run at
 * the same time need one each. Results do not depend on what a workspace
 * held before. Runs of the same call on the same device give the same bits.
 * Values in device memory that the host cannot check (lengths, ids, pages)
 * never lead outside the buffers.
 */
#ifndef MMVQ_SERVE_H
#define MMVQ_SERVE_H

#include <stdint.h>

#include "mmvq.h"
#include "mmvq_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of tables and adapters that are not quantized (ggml numbering);
 * MMVQ_F16 is in mmvq_decode.h. */
enum { MMVQ_F32 = 0, MMVQ_BF16 = 30 };

/* out[t*ldo + i] = scale * W[ids[t]][i], i < K, for n tokens, rounded to fp32
 * (formats with an offset, d q + m, from 64 bits, 2^-52 off). table: vocab rows back to back, of a weight format of mmvq.h (so a
 * tied LM head serves as it is; K a multiple of the type's block) or F32, F16
 * or BF16 (any K). A token outside 0..vocab-1 gives a row of zeros.
 * Requires 1 <= K <= 2^24, 1 <= vocab < 2^31, n >= 0, n*K <= 2^40, ldo >= K;
 * table 16-byte aligned, ids and out 4-byte. */
int mmvq_embed(const void *table, int type, int64_t vocab, int64_t K,
               const int32_t *ids, int64_t n, float scale, float *out,
               int64_t ldo, void *stream);

/* Page tables of the requests of one cache, and the pages that none of them
 * holds. Device arrays, all in/out:
 *   page_table   page of positions p*page_size .. of request s:
 *                page_table[s*table_stride + p], as in mmvq_kv_batch;
 *   pages_held   of each request: its entries p < pages_held[s] are its own
 *                (or holes: entries outside 0..n_pages-1);
 *   free_pages   n_pages entries, of which the first *n_free are free pages.
 * pages_per_seq entries of a table row are used; page_size a power of two,
 * 16..MMVQ_KV_MAX_PAGE. Requires 1 <= pages_per_seq <= 2^26, table_stride >=
 * pages_per_seq, n_pages >= 1; all 4-byte aligned. */
typedef struct mmvq_kv_pool {
    int32_t *page_table;
    int64_t table_stride;
    int32_t *pages_held;
    int32_t *free_pages;
    int32_t *n_free;
    int pages_per_seq;
    int n_pages;
    int page_size;
} mmvq_kv_pool;

/* Each request keeps its first keep[s] pages (keep[s] < 0: all of them). The
 * entries behind them become -1, and the pages that they named are put
 * behind the free ones, in the order of requests and positions, but for
 * entries p < shared[s] (pages that other tables name, too; shared NULL: 0)
 * and holes. Free pages beyond n_pages would be pages given back twice: they
 * are dropped. Requires 0 <= n_seqs <= 2^20; 4-byte aligned. */
int mmvq_kv_release(const mmvq_kv_pool *pool, int n_seqs, const int32_t *keep,
                    const int32_t *shared, void *stream);

/* Workspace of mmvq_kv_plan in bytes. Host-only. */
int mmvq_kv_plan_workspace(int n_seqs, int64_t *bytes);

/* A step of n_new[s] new tokens for each request s behind the cached[s] that
 * it has in the cache (values below 0 count as 0, cached ones above 2^30 as
 * 2^30), in n_rows rows:
 *   token_start  n_seqs + 1 entries: request s has the rows token_start[s] ..
 *                token_start[s+1]-1, the requests one after the other from
 *                row 0 (new tokens that n_rows leaves no room for are cut);
 *   seq_len      cached[s] and its new tokens (may be cached itself);
 * A request with new tokens gets the pages that its length needs beyond
 * those it holds, up to pages_per_seq. In the order of requests and
 * positions, page i of all that are needed is entry *n_free - g + i of the
 * free pages, with g of them given: all that are needed, or as many as are
 * free; the entries of those that are not there become -1 (holes, which
 * mmvq_kv_write and mmvq_attn skip) and stay outside pages_held. So pages
 * given and released again are in their order. n_missing (one number, NULL if
 * not wanted): how many were not there.
 * For each of n_rows rows (each NULL if not wanted):
 *   row_seq      its request, -1 behind the last request's rows;
 *   row_pos      its position, -1 there;
 *   row_slot     page*page_size + position % page_size, -1 there and in holes.
 * Requires 0 <= n_seqs <= 2^20, 0 <= n_rows <= 2^20; row_slot 8-byte aligned,
 * the others 4-byte. Without requests token_start[0] = 0, the rows' -1 and
 * n_missing = 0 are still written. cached, n_new, token_start and seq_len do
 * not overlap otherwise. */
int mmvq_kv_plan(const mmvq_kv_pool *pool, const int32_t *cached,
                 const int32_t *n_new, int n_seqs, int n_rows,
                 int32_t *token_start, int32_t *seq_len, int32_t *row_seq,
                 int32_t *row_pos, int64_t *row_slot, int32_t *n_missing,
                 void *workspace, int64_t workspace_bytes, void *stream);

/* Low-rank adapters of one projection of K inputs and M outputs. type
 * MMVQ_F16, MMVQ_BF16 or MMVQ_F32:
 *   A     adapter a's max_rank x K matrix at A + a*stride_a elements, rows of
 *         K back to back;
 *   B     its M x max_rank matrix at B + a*stride_b, rows of max_rank;
 *   rank  n_adapters ranks, of which A's first rows and B's first columns are
 *         used (above max_rank: max_rank; below 1: no effect); NULL: max_rank;
 *   scale n_adapters factors (alpha / rank, usually); NULL: 1.
 * Requires K and max_rank multiples of 8, 8 <= K <= 2^20, 8 <= max_rank <=
 * 256, 1 <= M <= 2^24, 1 <= n_adapters <= 2^20, strides multiples of 8 of at
 * least max_rank*K and M*max_rank; A and B 16-byte aligned, rank and scale
 * 4-byte. */
typedef struct mmvq_lora_set {
    const void *A;
    const void *B;
    const int32_t *rank;
    const float *scale;
    int64_t stride_a;
    int64_t stride_b;
    int64_t K;
    int64_t M;
    int type;
    int n_adapters;
    int max_rank;
} mmvq_lora_set;

/* Workspace of mmvq_lora for n rows in bytes. Host-only; the pointers of the
 * set are not looked at. */
int mmvq_lora_workspace(const mmvq_lora_set *set, int64_t n, int64_t *bytes);

/* out[t] = base[t] + scale[a] * B_a (A_a x[t]) for n rows, with a the adapter
 * of the row's request: adapter[row_seq[t]], or adapter[t] where row_seq is
 * NULL (n_seqs >= n then). Rows of no request (row_seq outside 0..n_seqs-1)
 * and of none of the adapters (outside 0..n_adapters-1) get base[t]. base may
 * be out itself (same pointer and stride): the projection's own output, to
 * which the adapters' is added. Rows of x, base and out at + t*ld floats.
 * Products are those of fp32 values (x in three bf16 parts, which hold all
 * its bits but those below 2^-133, the last that bf16 has; weights in one to
 * three), sums fp32. x and the weights must be finite; a row's own values that
 * are not reach no other row.
 * Consecutive rows of one adapter share its weights: rows are best ordered
 * by request. Requires 0 <= n <= 2^20, ldx >= K, ldb and ldo >= M, buffers
 * without overlap but for base; 4-byte aligned. */
int mmvq_lora(const mmvq_lora_set *set, const float *x, int64_t ldx, int64_t n,
              const int32_t *row_seq, const int32_t *adapter, int n_seqs,
              const float *base, int64_t ldb, float *out, int64_t ldo,
              void *workspace, int64_t workspace_bytes, void *stream);

/* Settings of n_seqs requests; each array NULL: off for all. */
typedef struct mmvq_sampling {
    const float *temperature;  /* not above 0: greedy; NULL: 1            */
    const int32_t *top_k;      /* below 1: off                            */
    const float *top_p;        /* 1 and above: off                        */
    const float *min_p;        /* not above 0: off; above 1 counts as 1   */
} mmvq_sampling;

/* Workspace of mmvq_sample in bytes. Host-only. */
int mmvq_sample_workspace(int n_rows, int vocab, int64_t *bytes);

/* The next token of each of n_rows rows of logits (fp32, row r at + r*ldl),
 * by the settings of the row's request s: row_seq[r], or r where row_seq is
 * NULL (n_seqs >= n_rows then). With the weights w_i = exp((l_i - top) / T),
 * top the largest logit (a greedy row: 1 at its lowest index, 0 elsewhere),
 * and the tokens in the order of falling logits, equal ones by rising index:
 *   top-k   keeps the first k;
 *   top-p   of these, those before which less than p times their sum has
 *           passed;
 *   min-p   of these, those with w_i >= m (that is m * w_top);
 * and the first token is kept in any case. The token is the lowest index j
 * with w_0 + .. + w_j > u[r] * sum(w), the sums over the kept ones.
 *   tokens   n_rows tokens;
 *   chosen   the probability that each was drawn with, w_j / sum(w);
 *   probs    the kept tokens' probabilities w_i / sum(w), 0 for the others,
 *            row r at + r*ldp: target weights (MMVQ_TARGET_WEIGHTS) or
 *            draft_probs of mmvq_verify_draft. May be logits itself (same
 *            pointer and stride).
 * Each NULL if not wanted, not all of them; u is read for tokens and chosen.
 * -inf and NaN logits have the weight 0; where a row has +inf logits these
 * have 1 and all others 0. A row without any weight, or of no request
 * (row_seq outside 0..n_seqs-1): token -1, chosen 0, probs 0. An infinite
 * temperature gives equal weights. Exponentials, sums and comparisons are in
 * 64 bits, but for two kinds of sums. In those that p is measured against each
 * weight is rounded by at most 2^-38 of itself, or 2^-64 of w_top; and so it is
 * in those that u is measured against and that chosen and probs are divided by,
 * where many tokens of a filtered row (more than 5120, or than 256 of 4096
 * neighbours) come up to the last kept one and those that weigh like it. Where
 * the sum before a token is that near to p or to u times all of them, it may
 * count either way.
 * u in [0, 1).
 * Requires 0 <= n_rows <= 2^20, 1 <= vocab <= 2^24, n_seqs >= 0, ldl and ldp
 * >= vocab; 4-byte aligned. params NULL: all off. */
int mmvq_sample(const float *logits, int64_t ldl, int vocab, int n_rows,
                const mmvq_sampling *params, const int32_t *row_seq,
                int n_seqs, const float *u, int32_t *tokens, float *chosen,
                float *probs, int64_t ldp, void *workspace,
                int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MMVQ_SERVE_H */
