/*
 * ninfer_decode.h -- the operators that surround the ternary projections in one
 * decode step of a batch of requests (same library, libninfer_ternary.so):
 *
 *   ninfer_kv_tables       block tables and slot maps from request lengths
 *   ninfer_kv_append       new keys and values into a paged cache
 *   ninfer_kv_attention    attention of one new token per request over that cache
 *   ninfer_logits_process  penalties, biases and grammar masks on the logits
 *
 * The conventions are those of ninfer_ternary.h: every function returns an
 * ninfer_status; sizes are uint64_t element counts unless called bytes; device
 * work is asynchronous on the caller's stream; the library allocates no device
 * memory and keeps no pointer after the call; on any status but NINFER_OK
 * nothing was launched or written. Every launch is a programmatic dependent one
 * that touches no buffer before the preceding work on the stream has completed.
 * Problems that only the device can see (a page list that ran out, a slot
 * outside the cache) set bits of an optional caller-owned int32 status word,
 * which the library never clears.
 */
#ifndef NINFER_DECODE_H
#define NINFER_DECODE_H

#include "ninfer_ternary.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One more element type, for caches only: 8-bit floats with four exponent and
 * three mantissa bits, largest value 448, no infinities. */
typedef enum { NINFER_E4M3 = 3 } ninfer_cache_dtype;

/*
 * A paged key/value cache. Element e of head h of token t of page p lies at
 * element p * page_stride + t * token_stride + h * head_stride + e of k and of
 * v, so that both [page][token][head][e] and [page][head][token][e] pools (and
 * slices of larger ones) are described by their strides. The value it stands
 * for is the stored one times k_scale (v_scale).
 *   dtype: NINFER_BF16, NINFER_F16 or NINFER_E4M3.
 *   pages, page_size, kv_heads > 0, pages < 2^31, page_size < 2^31;
 *   head_dim: 1..256, a multiple of 8 (NINFER_E4M3: of 16).
 *   strides: multiples of 16 bytes, token_stride below 2^25 bytes, the others below 2^40
 *     (token_stride unread for page_size 1, head_stride for kv_heads 1, page_stride for pages 1).
 *   k, v: device, 16-byte aligned. k_scale, v_scale: finite, > 0.
 */
typedef struct {
    void *k, *v;
    uint64_t pages, page_size, kv_heads, head_dim;
    uint64_t page_stride, token_stride, head_stride;
    float k_scale, v_scale;
    int dtype;
    int reserved;   /* 0 */
} ninfer_kv_cache;

/* Bits of *status. */
enum {
    NINFER_KV_OUT_OF_PAGES = 1,   /* tables: the free list is shorter than the pages needed */
    NINFER_KV_ROW_TOO_SHORT = 2,  /* tables: a request with new tokens needs more than table_pages pages */
    NINFER_KV_OUT_OF_SLOTS = 4,   /* tables: more new tokens than `capacity` (whether or not slots is given) */
    NINFER_KV_BAD_LENGTH = 8,     /* tables: a negative length, or one past 2^31 - 1 */
    NINFER_KV_BAD_SLOT = 16,      /* append: a slot at or past pages * page_size */
    NINFER_LOGITS_BAD_TOKEN = 32  /* logits: a history or bias token outside [0, vocab), or a mask row past the last */
};

/*
 * ninfer_kv_tables -- what a step needs to know about where its tokens live,
 * built on the device from the requests' lengths (P = page_size):
 *   held_i = ceil(lengths[i] / P), last_i = ceil((lengths[i] + new_i) / P);
 *   request i takes last_i - held_i pages of free_pages, in request order:
 *   block_table[i][held_i + q] = free_pages[q + sum over j < i of (last_j - held_j)];
 *   its new tokens are offsets[i] .. offsets[i + 1] - 1, offsets[i] = sum over j < i of new_j;
 *   token t of request i has positions[t] = lengths[i] + t - offsets[i], token_rows[t] = i and
 *   slots[t] = block_table[i][positions[t] / P] * P + positions[t] % P.
 * A decode step has one new token per request; admitting a prompt is lengths 0.
 *   lengths: device int32[requests], tokens that request i holds already.
 *   new_tokens: device int32[requests], 0 and more, or NULL for one each.
 *   free_pages: device int32[free_count], ids of pages that no request holds (NULL when
 *     free_count is 0); the caller drops counts[1] of them from the front afterwards.
 *   block_table: device int32, row i at i * table_stride, table_pages entries. Entries
 *     below held_i are read, those from held_i to last_i - 1 written, others untouched:
 *     a second call with the same inputs writes the same values.
 *   slots int64[capacity], positions and token_rows int32[capacity]: device, entries past the
 *     last new token are set to -1 (append skips them), so that a captured step can have
 *     a fixed size; offsets int32[requests + 1], lengths_out int32[requests] (lengths +
 *     new), counts int32[2] (new tokens, pages taken). Any of the six may be NULL.
 *     Outputs may not overlap inputs or block_table (a loop cannot write its lengths in place).
 *   A token that got no page (list or row too short) has slot -1, and its table entry
 *   (if there is one) is -1; offsets, lengths_out and counts are unaffected. Negative
 *   lengths count as 0; results past 2^31 - 1 are clamped to it.
 * Errors: INVALID_ARGUMENT (NULL lengths or block_table; free_pages NULL with a
 *   count; an output that overlaps an input or block_table), SHAPE (requests, page_size
 *   or table_pages 0; any of them, or capacity or free_count, over 2^31 - 1;
 *   table_stride < table_pages), ALIGNMENT, CUDA.
 */
int ninfer_kv_tables(const int32_t *lengths, const int32_t *new_tokens, uint64_t requests,
                     uint64_t page_size, const int32_t *free_pages, uint64_t free_count,
                     int32_t *block_table, uint64_t table_pages, uint64_t table_stride,
                     int64_t *slots, int32_t *positions, int32_t *token_rows, uint64_t capacity,
                     int32_t *offsets, int32_t *lengths_out, int32_t *counts, int32_t *status,
                     ninfer_stream stream);

/*
 * ninfer_kv_append -- new keys and values into the cache:
 *   cache.k[slots[t]][h][e] = round(k_new[t][h][e] / k_scale), the same for v,
 *   the exact quotient rounded once to nearest-even; NINFER_E4M3 saturates at +-448 and keeps NaN.
 *   k_new, v_new: device, src_dtype f32, bf16 or f16; element e of head h of token t at
 *     t * token_stride + h * head_stride + e (its own strides for each of the two; multiples
 *     of 16 bytes, so that slices of a fused projection's rows can be given as they are).
 *   slots: device int64[tokens], each page * page_size + token; a negative slot is skipped,
 *     one past the cache is skipped and sets NINFER_KV_BAD_SLOT. Slots given twice: one of
 *     the tokens is kept for each element.
 * Errors: INVALID_ARGUMENT, SHAPE (tokens 0; the cache's rules above), ALIGNMENT, CUDA.
 */
int ninfer_kv_append(const void *k_new, const void *v_new, int src_dtype, uint64_t tokens,
                     uint64_t k_token_stride, uint64_t k_head_stride, uint64_t v_token_stride,
                     uint64_t v_head_stride, const int64_t *slots, const ninfer_kv_cache *cache,
                     int32_t *status, ninfer_stream stream);

/*
 * ninfer_kv_attention -- attention of one new token per request:
 *   s_j = scale * (q[r][h] . key_j of head h / (q_heads / kv_heads)),
 *   out[r][h] = sum_j e^{s_j - m} value_j / sum_j e^{s_j - m},  lse[r][h] = ln sum_j e^{s_j},
 *   over the keys j of request r with max(0, n - window) <= j < n (window 0: all of them),
 *   n = lengths[r], the new token included (append it first), key j in page
 *   block_table[r][j / page_size]. A request without keys (n <= 0), or whose scores are
 *   all -infinity, gives zeros and lse -infinity. An infinite value among the keys' values
 *   makes its element of the result infinite or NaN. Cache entries outside the range are
 *   never part of the result, whatever they hold. Lengths past table_pages * page_size are
 *   cut to it; table entries outside [0, pages) stand for a page of zeros.
 *   q: device, q_dtype f32, bf16 or f16, element e of head h of request r at
 *     r * q_request_stride + h * q_head_stride + e (strides multiples of 16 bytes).
 *   q_heads: a multiple of kv_heads.
 *   block_table: device int32, row r at r * table_stride; lengths: device int32[requests].
 *   scale: finite. out: device [requests][q_heads][head_dim] of out_dtype (f32, bf16, f16).
 *   lse: device float[requests][q_heads] or NULL.
 *   workspace: device, at least ninfer_kv_attention_workspace() bytes, 256-byte aligned;
 *     its contents are not preserved.
 * Arithmetic: products of 16-bit operands with fp32 sums on the tensor cores. fp32 queries,
 * and the weights e^{s - m} of fp32 results, enter as sums of 16-bit terms that hold 22 bits
 * (NINFER_F16 and NINFER_E4M3 caches; of a query's elements no bit under 2^-39 of its head's
 * largest one) or 24; other weights have 16 bits (NINFER_BF16) or 11 and more. Running maxima and sums are fp32.
 * How the work is divided follows from the lengths of the call's requests and, for few rows, from
 * table_pages * page_size and the window, which bound them: where these stay the same, results repeat
 * bit for bit. Few and short rows are fastest under a table no wider than they need (a view of a wider
 * one's first entries will do).
 * ninfer_kv_attention_workspace: bytes for these arguments and any lengths; host only.
 * Errors: INVALID_ARGUMENT, SHAPE, SIZE_MISMATCH (workspace), ALIGNMENT, OVERFLOW, CUDA.
 */
int ninfer_kv_attention_workspace(const ninfer_kv_cache *cache, uint64_t requests,
                                  uint64_t q_heads, uint64_t *bytes);
int ninfer_kv_attention(const void *q, int q_dtype, uint64_t requests, uint64_t q_heads,
                        uint64_t q_request_stride, uint64_t q_head_stride,
                        const ninfer_kv_cache *cache, const int32_t *block_table,
                        uint64_t table_pages, uint64_t table_stride, const int32_t *lengths,
                        float scale, uint64_t window, void *out, int out_dtype, float *lse,
                        void *workspace, uint64_t workspace_bytes, ninfer_stream stream);

/*
 * ninfer_logits_process -- for every row b and token v of the logits, in this order:
 *   x = logits[b][v];
 *   x = x > 0 ? x / repetition[b] : x * repetition[b]    if v is in history[b][0 .. n),
 *   x -= frequency[b] * c + presence[b] * (c > 0)         c: how often v is in history[b][p .. n),
 *   x += bias                                             if v is listed with one,
 *   x = -infinity                                         if row mask_rows[b] of the mask forbids v,
 *   n = history_lengths[b], p = prompt_lengths[b] (the prompt is known, not answered with).
 * Computed in fp32 (the quotient as the product with the reciprocal, where that is a normal number), rounded
 * once to dtype.
 *   logits, out: device, dtype f32, bf16 or f16, row b at b * stride elements; out may be
 *     logits itself (same stride).
 *   history: device int32, row b at b * history_stride, below 2^30 (tokens outside [0, vocab) are ignored and
 *     set NINFER_LOGITS_BAD_TOKEN); NULL: no history. history_lengths: device
 *     int32[rows] (needed with a history; cut to [0, history_stride]).
 *     prompt_lengths: device int32[rows] or NULL (0).
 *   repetition, presence, frequency: device float[rows], each may be NULL (1, 0, 0).
 *   bias_offsets: device int32[rows + 1]: entries bias_offsets[b] .. bias_offsets[b + 1] - 1 of
 *     bias_ids (int32) and bias_values (float) belong to row b; all three or none. bias_count:
 *     entries in all (offsets are cut to it). Ids of one row differ from each other.
 *   mask: device uint32, row i at i * mask_stride words, bit v % 32 of word v / 32 set where v is
 *     allowed; mask_row_count rows. mask_rows: device int32[rows], the mask row of each
 *     logits row, negative for none; NULL: row b uses mask row b. mask NULL: no masks.
 * Errors: INVALID_ARGUMENT, SHAPE (rows or vocab 0, vocab over 2^31 - 1, strides too
 *   small, mask_row_count < rows without mask_rows), ALIGNMENT, CUDA.
 */
typedef struct {
    const int32_t *history, *history_lengths, *prompt_lengths;
    uint64_t history_stride;
    const float *repetition, *presence, *frequency;
    const int32_t *bias_offsets, *bias_ids;
    const float *bias_values;
    uint64_t bias_count;
    const uint32_t *mask;
    const int32_t *mask_rows;
    uint64_t mask_row_count, mask_stride;
} ninfer_logits_controls;

int ninfer_logits_process(const void *logits, uint64_t logits_stride, void *out, uint64_t out_stride,
                          int dtype, uint64_t rows, uint64_t vocab,
                          const ninfer_logits_controls *controls, int32_t *status,
                          ninfer_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* NINFER_DECODE_H */
