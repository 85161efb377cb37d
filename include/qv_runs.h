/*
 * qv_runs.h -- C ABI of libqv for runs of tokens: prompts, frames, chunks of them and guessed tokens, of many sequences of
 * different lengths at once, over the paged cache of qv_decode.h.
 *
 *   qv_page_tables     which pages, places and slots the new tokens of each sequence take, worked out on the GPU
 *   qv_run_attention   attention of each sequence's new tokens over its cache, with a sliding window and first tokens that
 *                      stay visible; the single token of a sequence is a run of one
 *
 * Between them stands qv_kv_append, which takes qv_page_tables' outputs as they are.  The conventions are those of
 * qv_decode.h.
 */
#ifndef QV_RUNS_H
#define QV_RUNS_H

#include "qv_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What qv_page_tables says of a sequence. */
typedef enum {
  QV_RUN_OK = 0,
  QV_RUN_NO_ROOM = 1,  /* the run passes the table's max_pages pages */
  QV_RUN_NO_PAGES = 2, /* there are too few free pages */
  QV_RUN_NO_ROWS = 3   /* the run's rows pass T */
} qv_run_status;

/*
 * qv_page_tables -- n_b new tokens of each of B sequences take their places: pages from a list of free ones, rows of the call.
 *   runs        [B] int32 n_b;  lens [B] int32 tokens that the sequence has.  Negative numbers count as 0.
 *   page_size   positive;  max_pages * page_size is below 2^31.
 *   free_pages  [num_free] int32 pages that no sequence holds, of which the first free_count [1] int32 count (cut to
 *               [0, num_free]).  They are taken from the end: the j-th new page of sequence b is
 *               free_pages[free_count - 1 - (pages that the sequences before asked for) - j].
 *   page_table  [B][ld_table] int32: the entries of new pages are written, pages ceil(len / page_size) onwards; all others
 *               stay.  ld_table >= max_pages, any.
 *   starts      [B + 1] int32 out: rows starts[b] .. starts[b + 1] - 1 are those of sequence b, sums of n_b (cut to 2^31 - 1).
 *   lens_out    [B] int32 out: lens + n_b, or lens of a sequence that is refused.  May be lens itself.
 *   free_left   [1] int32 out: free_count less the pages taken.  May be free_count itself.
 *   token_seq, token_index, slots   [T] int32, int32, int64 out: of each row its sequence, its place in it, and its place
 *               among all slots of the cache, page * page_size + place % page_size.  Rows of a sequence that is refused, and
 *               rows from starts[B] on, are -1 (which qv_kv_append does not store).
 *   status      [B] int32 out: qv_run_status.  A sequence is refused as a whole: it takes no pages and keeps its length, but
 *               its rows stay its own (what attention makes of them means nothing).  One without room or rows asks for no
 *               pages, whatever is free.  Sequences are served in order: one that lacks pages has asked for them all the same,
 *               so that no later one that needs a page gets any.  A sequence without new tokens is never refused for pages or
 *               rows.
 * Outputs other than those two, and the table, do not overlap the inputs or each other.
 * The page of a place before lens[b] is read from the table.  T = 0 is accepted with null outputs of [T].  T <= 2^31 - 1.
 */
qv_status qv_page_tables(const int32_t* runs, const int32_t* lens, int64_t B, int64_t page_size, const int32_t* free_pages,
                         int64_t num_free, const int32_t* free_count, int32_t* page_table, int64_t max_pages,
                         int64_t ld_table, int32_t* starts, int32_t* lens_out, int32_t* free_left, int32_t* token_seq,
                         int32_t* token_index, int64_t* slots, int64_t T, int32_t* status, void* hip_stream);

/* Bytes of workspace qv_run_attention needs for T rows of B sequences with runs of up to max_run tokens and page tables of up to
 * `capacity` tokens each (max_pages * page_size), rounded up to 256 and at least 256 (0 for invalid sizes). */
size_t qv_run_attention_workspace_size(int64_t T, int64_t B, int64_t max_run, int64_t q_heads, int64_t heads,
                                       int64_t head_dim, int64_t capacity);

/*
 * qv_run_attention -- attention of each sequence's new tokens over the paged cache, which holds them already:
 *   O[s][i] = sum_t softmax_t(scale Q[s][i] . k[t][i / (q_heads / heads)]) v[t][i / (q_heads / heads)]
 * Row s of sequence b, which has n_b of them, is its token at place p = lens[b] - n_b + s - starts[b], and sees the tokens t of b with
 *   t <= p (causal) or t < lens[b] (causal = 0),  and  t < sinks or t > p - window (window = 0: all of them).
 *   Q           [T][q_heads][head_dim] fp32 or bf16;  q_heads a multiple of the cache's heads.
 *   starts      [B + 1] int32, not falling: rows starts[b] .. starts[b + 1] - 1 are sequence b's n_b, its last ones (cut to
 *               [0, T] and to max_run rows); or NULL: row b is sequence b's one token (then T = B and max_run = 1).
 *   page_table, lens   as for qv_paged_attention, max_pages * page_size below 2^31 - 64.  Tokens on a page outside [0, num_pages)
 *               do not take part.
 *   max_run     the longest run, up to T (of a captured call, the longest that its replays will have).  A longer run is its
 *               first max_run rows: n_b is max_run, so that these are taken for the last max_run tokens of the sequence.  Rows
 *               behind them are not written, nor are rows that no sequence has.
 *   scale       finite;  window >= 0, sinks >= 0 (else QV_ERR_SHAPE).
 *   O           [T][q_heads][head_dim] of Q's type.  A row that sees no token gives zeros; a query of NaN, or a NaN among the
 *               tokens that a row sees, gives NaN; what a row does not see does not count, whatever it holds.
 *               Scores, softmax and sums are fp32.  For the product with the values, bf16 queries in runs with more than
 *               QV_RUN_FEW_ROWS rows to a cache head (QV_RUN_FEW_ROWS_8BIT over 8-bit caches), max_run * q_heads / heads, have
 *               each probability as two bf16 pieces that leave 2^-17 of it at most; else it is not rounded.  An fp32 query is
 *               taken as three bf16 pieces that sum to it.
 *   workspace   at least qv_run_attention_workspace_size bytes, 256-byte aligned, reused freely.
 */
#define QV_RUN_FEW_ROWS 32
#define QV_RUN_FEW_ROWS_8BIT 64
qv_status qv_run_attention(const qv_heads* Q, qv_dtype q_dtype, int64_t T, int64_t q_heads, const int32_t* starts, int64_t B,
                           int64_t max_run, const qv_kv_cache* cache, const int32_t* page_table, int64_t max_pages,
                           int64_t ld_table, const int32_t* lens, float scale, int64_t window, int64_t sinks, int32_t causal,
                           const qv_heads* O, void* workspace, size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* QV_RUNS_H */
