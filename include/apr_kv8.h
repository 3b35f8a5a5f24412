/*
 * apr_kv8.h — C ABI of the 8-bit paged key/value cache (GB300, sm_103a): what
 * decoding needs after a prefill. Part of libapr_qgemm; errors, streams,
 * scratch and apr_stream_status are those of apr_qgemm.h.
 *
 *   apr_kv8_append     quantises new k and v rows into the cache
 *   apr_kv8_read       gives rows of the cache back as numbers
 *   apr_kv8_attention  causal attention of each sequence's last rows over its
 *                      cache, and the weight that each position received
 *   apr_kv8_evict      keeps the positions of the largest weights and the most
 *                      recent ones, in fresh pages
 *
 * The cache. K and V are held in pages of page_tokens tokens: signed 8-bit
 * codes [num_pages][num_kv_heads][page_tokens][head_dim] and one float32 scale
 * for each page and head, [num_pages][num_kv_heads]; the value of a code c
 * under the scale s is c * s. A sequence's pages are listed in its row of
 * page_table; pages may be in any order, and sequences may share pages that
 * no call writes. Any positive scales and any codes are read; the append writes
 * codes -127..127.
 *
 * The rows of a call. Every call is about num_seqs sequences. lens[b] counts
 * the tokens that sequence b holds, this call's rows included: a sequence's n
 * rows are its positions lens[b] - n .. lens[b] - 1. Rows are packed: sequence
 * b has the rows row_start[b] .. row_start[b + 1] - 1 of the call's num_rows;
 * row_start == NULL is one row for each sequence (num_rows == num_seqs, a
 * decode step). A row whose position would be negative (a slot with lens 0 in
 * a step of fixed width) is skipped by the append, and reads, and attends to,
 * zeros. lens, row_start and page_table are device arrays, read when the
 * kernels run, so a captured step can be replayed as they change.
 *
 * What the device arrays say is checked where it is used: a page id outside
 * 0 .. num_pages - 1, a length below 0 or past table_ld * page_tokens or max_len, a
 * row_start that is not within 0 .. num_rows and non-decreasing, or more rows
 * of one sequence than max_rows make no access outside the call's arrays; they
 * set a bit of the device status word, and the next apr_stream_status returns
 * APR_E_INVAL (the call's outputs are then unspecified). Where a page id is out
 * of range, the append writes none of that page's rows, the read none of its
 * values, the eviction takes them for zeros or writes no such page, and the
 * attention reads page 0 in its place. A sequence whose length is out of range
 * counts as one of no tokens, one whose rows are as one without rows: nothing of
 * it is appended or moved, what it holds in the cache stays as it is, and weights
 * that are added up over calls do not change.
 *
 * All pointers are device pointers, caller owned; codes, rows and outputs on
 * 16-byte boundaries, the other arrays on their element's. Calls are
 * asynchronous on the stream, may be captured, and follow its order: a call
 * touches none of its arguments before the work ahead of it is done. The same
 * inputs give the same bits: no result depends on timing.
 */
#ifndef APR_KV8_H
#define APR_KV8_H

#include "apr_qgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of rows (GGUF type ids). */
enum { APR_T_F32 = 0, APR_T_F16 = 1, APR_T_BF16 = 30 };

typedef struct apr_kv8_cache {
  signed char* K;
  signed char* V;
  float* k_scale;
  float* v_scale;
  int num_pages;     /* 1 .. 2^27 */
  int num_kv_heads;  /* 1 .. 1024 */
  int page_tokens;   /* 32, 64, 128 or 256 */
  int head_dim;      /* 64, 128 or 256 */
} apr_kv8_cache;

typedef struct apr_kv8_rows {
  const int* page_table;  /* [num_seqs][table_ld] */
  int table_ld;           /* entries from one sequence's row to the next; table_ld * page_tokens <= 2^30 */
  const int* lens;        /* [num_seqs] */
  const int* row_start;   /* [num_seqs + 1] or NULL */
  int num_seqs;           /* 0 .. 16384 */
  int num_rows;           /* 0 .. 2^24 */
  int max_rows;           /* most rows of one sequence; 0: num_rows (1 without row_start) */
  int max_len;            /* most tokens of one sequence; 0: table_ld * page_tokens */
} apr_kv8_rows;

/*
 * Appends k and v: [num_rows][ld] rows of num_kv_heads * head_dim elements of
 * `type`, head g at g * head_dim (a slice of a wider buffer of projections:
 * ld >= num_kv_heads * head_dim, in elements; rows on 16-byte boundaries).
 * For each page and head that gets rows, with amax their largest finite
 * magnitude, s_old the page's scale (0 for a page whose first slot is one of
 * the rows):
 *   s = max(s_old, amax / 127)                   rounded to float32
 *   c = rint(x / s) clamped to +-127             for the new rows
 *   c = rint((c_old * s_old) / s)                for what the page held, if s > s_old
 * rint to the nearest whole number, ties to the even one, of the exact
 * quotient (c_old * s_old rounded to float32 first); codes under s = 0 are 0.
 * A value is off by at most s / 2, and each raise of its page's scale re-rounds
 * it once more. NaN is stored as 0, infinities as the largest code. Two
 * sequences of one call must not append into the same page. No scratch.
 */
int apr_kv8_append(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, const void* k, const void* v,
                   long long ld, apr_stream_t stream);

/*
 * Reads the rows back: k and v [num_rows][ld] of `type`, laid out as for the
 * append; each value the float32 product code * scale rounded to `type`. With
 * row_start over whole lengths it gives the float32 rows that
 * apr_prefill_attention takes. No scratch.
 */
int apr_kv8_read(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, void* k, void* v, long long ld,
                 apr_stream_t stream);

/*
 * Attention of the rows over their sequences' caches (which hold the rows' own
 * k and v already). For row i of sequence b's n rows, query head h, and
 * g = h / (num_heads / num_kv_heads):
 *   p_j = softmax_j(scale * q . K[j][g])   over j <= lens[b] - n + i
 *   out = sum_j p_j V[j][g]
 *   q, out   [num_rows][ldq], [num_rows][ldo] rows of num_heads * head_dim
 *            elements of `type`
 *   scale    0: 1 / sqrt(head_dim); else finite and positive
 *   rows     a few for each sequence is what this is for (a decode step, a draft
 *            of several tokens, the last rows of a prompt that rate its
 *            positions): each further 8 (row, head) pairs of a KV head cost about
 *            as much again. Chunks of hundreds of rows: apr_kv8_read, then
 *            apr_prefill_attention.
 *   weights  NULL, or [num_seqs][num_kv_heads][weights_ld] float32: the weight
 *            that each position received, w_j = sum over the sequence's rows
 *            and the query heads of group g of p_j. accumulate == 0: positions
 *            past the length, and all of sequences without rows, are set to 0;
 *            accumulate != 0: w_j is added to what the positions before this
 *            call's rows hold (the rows' own positions start at w_j; positions
 *            past the length keep what they hold). weights_ld >= max_len, or >= table_ld * page_tokens where
 *            max_len is 0.
 * A row that sees no position gives zeros. q is split into two fp16 pieces
 * (22 bits of the row's largest magnitude), the softmax weights likewise, the
 * codes enter the products exactly, and every sum is float32: of rows of about
 * unit variance float32 results are within a few 1e-6 of the exact attention of
 * the cache's values. What limits them is a score's error, some 2^-22 of the sum of
 * |scale q K|, and that weights below 2^-34 of the row's largest are left out of
 * its outputs (but not of its total): at most 2^-34 of V's largest value for each
 * such position, 2^-14 for a million of them beside one that takes all. A NaN or an
 * infinity in a query row makes that row and head NaN, and the weights of the
 * positions that the row sees.
 * out must not overlap q, the cache or weights. Scratch per stream: partial
 * results of 8 or 16 (row, head) pairs for each resident CTA (at most 8 MB), and,
 * with weights, the scores (4 * num_rows * num_heads * max_len bytes, max_len
 * rounded up to 32: give max_len where the table is much wider than the
 * sequences).
 * num_heads a multiple of num_kv_heads, at most 65536 in all.
 */
int apr_kv8_attention(const apr_kv8_cache* cache, const apr_kv8_rows* rows, int type, const void* q, long long ldq,
                      void* out, long long ldo, int num_heads, float scale, float* weights, long long weights_ld,
                      int accumulate, apr_stream_t stream);

/*
 * Eviction. A sequence of more than `budget` positions is cut to budget, for
 * each KV head on its own: its last `recent` positions stay, and of the others
 * those of the budget - recent largest weights (equal weights: the lowest
 * position first; NaN ranks above all numbers), in their order. Their K and V are written to the pages
 * fresh_pages[b][0 .. ceil(budget / page_tokens)), quantised anew (the append's
 * formula over the float32 values code * scale). Other sequences are left
 * alone. rows gives page_table, lens and their sizes (row_start, num_rows and
 * max_rows are not looked at).
 *   weights      [num_seqs][num_kv_heads][weights_ld], as the attention gives
 *                them; weights_ld >= max_len (table_ld * page_tokens where 0)
 *   budget >= 1, 0 <= recent <= budget
 *   fresh_pages  [num_seqs][ceil(budget / page_tokens)] pages of the same
 *                cache that nothing else uses; those of sequences that are not
 *                cut are not written
 * Outputs (none may overlap an input):
 *   table_out    [num_seqs][table_ld]: the pages that hold each sequence now
 *                (the fresh ones, or its own), -1 past its length
 *   lens_out     [num_seqs] = min(lens, budget)
 *   weights_out  [num_seqs][num_kv_heads][weights_out_ld], weights_out_ld >=
 *                budget: the kept positions' weights, 0 past the length
 *   kept         [num_seqs][num_kv_heads][budget]: the positions kept, -1
 *                past the length
 * No scratch. The old pages are the caller's to free or reuse.
 */
int apr_kv8_evict(const apr_kv8_cache* cache, const apr_kv8_rows* rows, const float* weights, long long weights_ld,
                  int budget, int recent, const int* fresh_pages, int* table_out, int* lens_out, float* weights_out,
                  long long weights_out_ld, int* kept, apr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* APR_KV8_H */
