/*
 * mmvq_decode.h - C ABI of the operators between the mat-vecs of a decode
 * step, in the same library as mmvq.h (MI355X, gfx950).
 *
 * A decode step of a transformer layer calls, around the products of mmvq.h:
 *   mmvq_add_rms_norm   residual addition and RMS norm, handing q8_1 columns
 *                       (or fp32 ones) to the next product;
 *   mmvq_kv_write       new tokens' keys and values into a paged cache,
 *                       quantized as they are written;
 *   mmvq_attn           attention of the new tokens over that cache;
 *   mmvq_verify_draft   after the LM head: which drafted tokens stand, and
 *                       the token that follows them.
 * mmvq_kv_read and mmvq_dequantize_q8_1 read the stored forms back. What else
 * a model puts between these (a rotary embedding of queries and keys, biases,
 * norms of its heads) is the caller's: q, k and v are fp32 rows in memory.
 *
 * Conventions are those of mmvq.h: data pointers are DEVICE pointers owned by
 * the caller; the struct arguments themselves are read on the host during the
 * call; everything is enqueued on `stream` and nothing synchronizes; the
 * library keeps no allocation and no state; return values are MMVQ_OK or
 * MMVQ_ERR_*, arguments are validated on the host before anything is
 * enqueued, and an invalid call enqueues nothing. Buffers that hold nothing
 * (no column, row, token or sequence) may be NULL. The kernels run on the
 * stream's device (NULL: the current device). Calls can be captured into HIP
 * graphs. A workspace belongs to one call until the stream has passed it;
 * calls that may run at the same time (two streams, two graphs) need one
 * each. Results do not depend on what a workspace held before. Runs of the
 * same call on the same device give the same bits.
 */
#ifndef MMVQ_DECODE_H
#define MMVQ_DECODE_H

#include <stdint.h>

#include "mmvq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Cache element types: MMVQ_F16 (ggml numbering), MMVQ_Q8_0, MMVQ_Q4_0. */
enum { MMVQ_F16 = 1 };

/* Limits of the operators below. */
#define MMVQ_KV_MAX_HEAD_DIM 256
#define MMVQ_KV_MAX_PAGE 1024

/* y = (x + residual) / sqrt(mean((x + residual)^2) + eps) * weight, per
 * column of K values; n columns, column j of a buffer at + j*ld floats.
 *   h = x + residual, rounded to fp32 (h = x where residual is NULL);
 *   y[i] = fp32(h[i] * (1/sqrt(sum(h^2)/K + eps)) * weight[i]), the sum,
 *   the root and both products in 64 bits, rounded once (weight NULL: 1).
 * Outputs, each NULL if not wanted: sum_out (h), y (fp32), y_q (q8_1 columns
 * of y, n * K/32 blocks of 36 bytes, what mmvq and its variants take: q =
 * roundf(y/d) and s = d*sum(q) as mmvq_quantize_q8_1 has them, with d =
 * max|y| * fp32(1/127) in fp32, the product with the rounded reciprocal,
 * which is what torch computes for amax / 127.0 on this GPU). That function's
 * d is a quotient: stored scales differ by at most one fp16 step and codes by
 * at most 1, where y/d lies within 2^-14 of a border (some 10^-7 of them).
 * Where its bits matter, take y and call it. sum_out may be x or residual
 * itself (same pointer and stride), and y may be x where sum_out is not;
 * otherwise the buffers do not overlap.
 * Requires 1 <= K <= 2^24, n >= 0 and n*K <= 2^40, every ld >= K, K % 32 == 0
 * with y_q, and at least one of y and y_q (MMVQ_ERR_NULL). fp32 buffers
 * 4-byte aligned, y_q 16-byte. With y_q the values must be finite, as for
 * mmvq_quantize_q8_1. */
int mmvq_add_rms_norm(const float *x, int64_t K, int64_t n, int64_t ldx,
                      const float *residual, int64_t ldr, const float *weight,
                      float eps, float *sum_out, int64_t lds, float *y,
                      int64_t ldy, void *y_q, void *stream);

/* x[j*ldx + i] = d * q of value i of q8_1 column j (d as stored, fp16).
 * Requires K % 32 == 0, 1 <= K <= 2^24, n >= 0, n*K <= 2^40, ldx >= K; y_q
 * 16-byte aligned, x 4-byte. */
int mmvq_dequantize_q8_1(const void *y_q, int64_t K, int64_t n, float *x,
                         int64_t ldx, void *stream);

/* A paged key/value cache of one layer. k and v hold n_pages pages of
 * mmvq_kv_page_bytes each (16-byte aligned); a page holds page_size
 * consecutive tokens of one sequence for every key/value head.
 *   type       MMVQ_F16 (nearest even; beyond 65504 infinite), MMVQ_Q8_0
 *              (per 32 values of a head: d = max|x| * fp32(1/127) in fp32,
 *              q = roundf(x/d), 0 where d is 0; value fp16(d)*q) or MMVQ_Q4_0
 *              (d = m/-8 with m the value of largest magnitude, the first of
 *              equals; q = min(15, floor(x/d + 8.5)), 8 where d is 0; value
 *              fp16(d)*(q - 8)); a d beyond 65504 is stored as 65504; the
 *              values to quantize must be finite;
 *   page_size  a power of two, 16..MMVQ_KV_MAX_PAGE;
 *   head_dim   64, 96, 128 or 256; n_kv_heads 1..1024.
 * Layout of a page: per head, page_size/16 units of 16 tokens, each in the
 * order in which the attention kernel's matrix instructions take it: the
 * library's own, read back by mmvq_kv_read. */
typedef struct mmvq_kv_cache {
    void *k;
    void *v;
    int type;
    int n_pages;
    int page_size;
    int n_kv_heads;
    int head_dim;
} mmvq_kv_cache;

/* A ragged batch of new tokens of n_seqs sequences. Device arrays:
 *   token_start  n_seqs + 1 rising row numbers; sequence s has the rows
 *                token_start[s] .. token_start[s+1]-1 of the activation
 *                buffers, possibly none;
 *   seq_len      tokens of each sequence, the new ones included: new token i
 *                of c is at position seq_len - c + i;
 *   page_table   page of positions p*page_size ..: page_table[s*table_stride
 *                + p], p < pages_per_seq. An entry outside 0..n_pages-1, or
 *                a position past the table, is a hole: nothing is written
 *                there, it reads back as zero and attention does not see it.
 * Host values: n_tokens rows in the buffers (rows before token_start[0] and
 * behind token_start[n_seqs] are left as they are); max_new and max_len,
 * the largest token count and length of any sequence, from which the launch
 * is shaped (larger device values cost time, not correctness).
 * Requires n_seqs >= 0, n_tokens >= 0 (0 of either: nothing is done), max_new
 * and max_len >= 1, pages_per_seq >= 1, table_stride >= pages_per_seq;
 * n_seqs, n_tokens and max_new <= 2^20, max_len <= 2^30, pages_per_seq <=
 * 2^26. A cache slot is given to at most one token of a call (which of two
 * would stay is open; reading shared pages is fine). */
typedef struct mmvq_kv_batch {
    const int32_t *token_start;
    const int32_t *seq_len;
    const int32_t *page_table;
    int64_t table_stride;
    int n_seqs;
    int n_tokens;
    int pages_per_seq;
    int max_new;
    int max_len;
} mmvq_kv_batch;

/* Bytes of one page of k (or of v). Host-only. MMVQ_ERR_TYPE, _SHAPE, _NULL. */
int mmvq_kv_page_bytes(int type, int page_size, int n_kv_heads, int head_dim,
                       int64_t *bytes);

/* Rows of k and v (fp32, row t at + t*ld floats, head h's values at
 * h*head_dim) into the cache at their tokens' positions. ld >= n_kv_heads *
 * head_dim; 4-byte aligned, so they can be slices of one product's output.
 * Nothing but the tokens' own slots is changed. */
int mmvq_kv_write(const mmvq_kv_cache *cache, const mmvq_kv_batch *batch,
                  const float *k, int64_t ldk, const float *v, int64_t ldv,
                  void *stream);

/* The reverse: the values that the cache holds at the batch's positions, as
 * fp32 rows; zero for holes and for positions below 0 (token_start of whole
 * lengths reads whole sequences). k or v NULL: not read. */
int mmvq_kv_read(const mmvq_kv_cache *cache, const mmvq_kv_batch *batch,
                 float *k, int64_t ldk, float *v, int64_t ldv, void *stream);

/* Workspace of mmvq_attn for these arguments, in bytes (0: none). Host-only;
 * the pointers in the structs are not looked at. */
int mmvq_attn_workspace(const mmvq_kv_cache *cache, const mmvq_kv_batch *batch,
                        int n_heads, int64_t *bytes);

/* out[t][h] = sum over visible keys of softmax(scale * q[t][h] . k) v, for
 * the batch's new tokens (written to the cache before) and n_heads query
 * heads, n_heads a multiple of n_kv_heads (head h reads key/value head
 * h / (n_heads / n_kv_heads)). A token at position p sees the keys at
 * positions 0..p, the last `window` of them where window > 0. sinks: NULL or
 * n_heads logits that join each head's softmax as a key without a value. A
 * token that sees no key gets zeros; an infinite cached value makes the
 * results of the tokens that see it infinite or NaN, and no others. q and
 * out: fp32, row t at + t*ld, head h at h*head_dim; ld >= n_heads*head_dim,
 * 4-byte aligned, without overlap; q must be finite.
 * Keys and values enter at their stored precision; scores, softmax and sums
 * are fp32, with q carried as two fp16 parts (21 bits of the row's largest
 * value) and each probability as two fp16 parts (20 bits; a key's share of the
 * result is good to 2^-32 of the largest value that the row sees, where that
 * is more).
 * The launch is shaped by max_new and max_len, for all sequences alike: one
 * chunk of a prompt among single tokens, or one long sequence among many short
 * ones, makes the others wait. A descriptor holds any consecutive sequences
 * (token_start + a, seq_len + a, page_table + a * table_stride, with their own
 * maxima), so such batches are better given in two calls over the same rows.
 * workspace: 16-byte aligned, at least mmvq_attn_workspace bytes (fewer:
 * MMVQ_ERR_SHAPE). n_heads <= 65535 and n_tokens * n_heads <= 2^30; a launch
 * beyond 2^23 workgroups (sequences * key/value heads * tiles of 16 to 128
 * rows) is refused, too. */
int mmvq_attn(const mmvq_kv_cache *cache, const mmvq_kv_batch *batch,
              const float *q, int64_t ldq, int n_heads, float scale,
              int window, const float *sinks, float *out, int64_t ldo,
              void *workspace, int64_t workspace_bytes, void *stream);

/* What mmvq_verify_draft's target rows hold. */
enum {
    MMVQ_TARGET_LOGITS = 0,   /* p = softmax(row / temperature)              */
    MMVQ_TARGET_WEIGHTS = 1   /* p = row / sum(row): probabilities, filtered
                                 or not                                      */
};

/* Workspace of mmvq_verify_draft in bytes. Host-only. */
int mmvq_verify_workspace(int n_seqs, int n_rows, int vocab, int64_t *bytes);

/* Verification of drafted tokens (speculative sampling). Sequence s has rows
 * row_start[s] .. row_start[s+1]-1 of target (fp32, row r at + r*ldt): c rows
 * for c - 1 drafted tokens, row i being the target's distribution p_i of the
 * token after i drafted ones; draft_tokens[r] is the token drafted at row r
 * (not read for a sequence's last row) and draft_probs row r (+ r*ldd) the
 * distribution q it was drawn from, or draft_probs NULL where the draft was
 * certain of it. In order, drafted token x of row i is accepted iff
 *   u_accept[r] * q(x) < p_i(x)
 * (a token outside 0..vocab-1 never). At the first that is not, a token is
 * drawn from max(p_i - q, 0) (from p_i where that is zero throughout); if
 * all are, from p of the last row. Drawn from weights w with a given number:
 * the lowest index j with w_0 + .. + w_j > u_sample[s] * sum(w).
 *   n_accepted[s]                drafted tokens accepted;
 *   tokens[s*max_out + i]        those tokens, then the drawn one, then -1,
 *                                for i < max_out.
 * temperature: n_seqs floats for MMVQ_TARGET_LOGITS, NULL = 1; where it is
 * not above 0 the sequence is greedy: p is 1 at the row's largest logit, the
 * lowest index of equals. -inf logits have probability 0, NaN likewise;
 * where a row has +inf logits they share all of it. Weights that are not
 * positive and finite count as 0. A row without any probability ends its
 * sequence: -1 in place of the drawn token. A sequence without rows gets 0
 * and -1. All sums, exponentials and comparisons are in 64 bits. u_accept:
 * n_rows floats, u_sample: n_seqs, in [0, 1).
 * Requires n_seqs and n_rows >= 0 (0 sequences: nothing is done), both <=
 * 2^20, 1 <= vocab <= 2^24, ldt and ldd >= vocab, max_out >= 1, row_start
 * rising within 0..n_rows (other rows have no effect); MMVQ_ERR_TYPE for an
 * unknown target kind. All 4-byte aligned, workspace 16-byte and at least
 * mmvq_verify_workspace bytes (fewer: MMVQ_ERR_SHAPE). */
int mmvq_verify_draft(const float *target, int64_t ldt, int vocab, int kind,
                      const float *temperature, const int32_t *draft_tokens,
                      const float *draft_probs, int64_t ldd,
                      const int32_t *row_start, int n_seqs, int n_rows,
                      const float *u_accept, const float *u_sample,
                      int32_t *n_accepted, int32_t *tokens, int max_out,
                      void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MMVQ_DECODE_H */
