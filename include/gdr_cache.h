/*
 * gdr_cache.h -- the paged key-value cache of libgdr's attention layers: the
 * write of new tokens, attention of new tokens over the cache, and eviction
 * by accumulated attention weight (MI355X, gfx950).
 *
 * A placement gives every decoder layer one of four mixers.  gdr.h holds the
 * calls of the recurrent ones (GDR_GDN, GDR_KDA), whose state is a matrix
 * per head; the calls here serve the other two, full attention (GDR_FA,
 * window = 0) and sliding-window attention (GDR_SWA, window > 0), whose
 * state is a cache of keys and values that grows with the sequence.
 *
 * The cache.  k_cache and v_cache are [num_pages, Hkv, page_size, D], one
 * page being page_size consecutive tokens of one sequence, head by head.
 * page_table [B, max_pages] (device int32) names the pages of each sequence:
 * token j of sequence b lies in page page_table[b, j / page_size] at slot
 * j % page_size.  An entry outside 0..num_pages-1 marks an absent page
 * (serving loops fill unused entries with -1): its tokens are never read,
 * attended to or written.  scores [num_pages, Hkv, page_size] fp32, where a
 * call takes them, hold one accumulated attention weight per token and
 * key-value head, in pages of their own that share the table.
 *
 * The conventions of gdr.h hold here as well (device pointers, dense
 * row-major tensors, 16-byte alignment -- page tables, lengths and offsets
 * 4-byte --, host checks before any HIP call, no allocation or
 * synchronisation, gdr_status codes, gdr_last_error, GDR_DEBUG).  Results
 * are the same bits on every run: no floating-point sum goes through atomics.
 *
 * Supported shapes: D in {64, 128}; page_size in {16, 32, 64, 128, 256};
 * max_pages * page_size < 2^30; num_pages * Hkv < 2^31; per call fewer than
 * 2^26 rows (T_total * Hkv) written, 2^23 query rows (B * n_tok * Hq) and
 * 2^21 trimmed (sequence, head) pairs (GDR_EUNSUPPORTED otherwise).  k, v, q,
 * o and the caches share one dtype, GDR_F32 or GDR_BF16.  Outputs overlap no
 * input except where a call says so.
 */
#ifndef GDR_CACHE_H
#define GDR_CACHE_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Write new tokens into the cache: token t of sequence b goes to position
 * start[b] + t.  A position that is negative, past the table's end or on an
 * absent page is left out.
 *
 *   B            sequences (>= 0)
 *   n_tok        tokens per sequence (cu_seqlens == NULL; T_total is then
 *                B * n_tok)
 *   T_total      rows of k and v
 *   k, v         [T_total, Hkv, D] dt: [B, n_tok, Hkv, D], or packed
 *   cu_seqlens   NULL, or device int32 [B+1]: sequence b's tokens are rows
 *                [cu_seqlens[b], cu_seqlens[b+1]); rows at or past
 *                cu_seqlens[B] belong to no sequence and are left out (a
 *                padded batch)
 *   cu_seqlens_host  host copy, optional: validated first (starts at 0, does
 *                not decrease, ends at or below T_total)
 *   start        device int32 [B]
 *   scores       NULL, or the accumulated weights: set to 0 at every
 *                position written (a page may come from an earlier request)
 *
 * The places of one call's tokens must differ: sequences may share pages that
 * the call does not write, but a place that two tokens name (a page under two
 * sequences, or twice in a table) is left with unspecified contents, K and V
 * of different tokens or pieces of both among them.
 */
gdr_status gdr_cache_append(enum gdr_dtype dt, int B, int n_tok, int T_total, int Hkv, int D,
                            const void *k, const void *v, const int32_t *cu_seqlens,
                            const int32_t *cu_seqlens_host, const int32_t *start,
                            const int32_t *page_table, int max_pages, int page_size,
                            int num_pages, void *k_cache, void *v_cache, float *scores,
                            void *stream);

/*
 * Attention of the newest n_tok tokens of each sequence over its cache
 * (their own keys and values included: append them first).  Sequence b holds
 * seq_lens[b] tokens (values outside 0..max_pages*page_size are taken as the
 * nearest bound); its query token t stands at position
 * p = seq_lens[b] - n_tok + t and attends to the tokens
 *     A = { j : 0 <= j <= p,  j > p - window if window > 0,  page present },
 * with query head h reading key-value head h / (Hq / Hkv):
 *     s_j = scale * q . k_j,   w_j = e^{s_j} / sum_A e^{s_i},
 *     o = sum_A w_j v_j.
 * A row whose weights e^{s_j} are all zero, or that attends to nothing
 * (seq_lens[b] == 0, p < 0, absent pages), gives o = 0.  What lies in
 * tokens a row does not attend to has no part in its result, NaN and
 * infinities included.
 *
 *   n_tok        query tokens per sequence (>= 0): one for a decode step,
 *                several to verify a draft
 *   Hq, Hkv      query and key-value heads, Hq a multiple of Hkv
 *   scale        multiplies the dot products (finite)
 *   window       0: every token up to the row's own; W > 0: the last W
 *   q, o         [B, n_tok, Hq, D] dt
 *   seq_lens     device int32 [B]
 *   scores       NULL, or the accumulated weights, to which the call adds
 *                for every token and key-value head the sum of w_j over the
 *                n_tok * Hq / Hkv rows that read it.  A page must then
 *                be in the table once (without scores, pages may be shared).
 *   page_table_host  host copy of page_table, optional: validated first
 *                (values in -1..num_pages-1; with scores, no page twice)
 *   workspace    device buffer of gdr_attention_workspace_bytes bytes (0 for a
 *                table without pages: NULL is accepted then), 16-byte
 *                aligned; needs no clearing; not to be shared with a
 *                concurrent call.  With scores it holds the products q.k of
 *                every row and place of the table, 4 * B * n_tok * Hq *
 *                max_pages * page_size bytes whatever the lengths and the
 *                window are (64 sequences, one token, 32 heads, a table of
 *                131,072 tokens: 1 GiB)
 *
 * The lengths are on the device: sizes, launches and the choice of a kernel
 * follow the table's width.  A table no wider than the longest sequence of
 * the call needs less memory and, for short sequences, less time than one as
 * wide as the longest context served.
 *
 * Numerics: fp32 accumulation, logits, softmax statistics and weights; with
 * bf16 inputs a weight enters the product with V as the sum of two bf16
 * numbers, off by at most 2^-15 of it (scores take it unrounded).
 */
size_t gdr_attention_workspace_bytes(int B, int n_tok, int Hq, int Hkv, int D, int max_pages,
                                     int page_size, int with_scores);

gdr_status gdr_attention_decode(enum gdr_dtype dt, int B, int n_tok, int Hq, int Hkv, int D,
                                float scale, int window, const void *q, const void *k_cache,
                                const void *v_cache, const int32_t *page_table,
                                const int32_t *page_table_host, int max_pages, int page_size,
                                int num_pages, const int32_t *seq_lens, float *scores, void *o,
                                void *workspace, size_t ws_bytes, void *stream);

/*
 * Trim every sequence to at most `budget` tokens by accumulated weight.  Of
 * a sequence of len > budget tokens each key-value head keeps, on its own,
 * the first `sink`, the last `recent` and, of the others, the
 * budget - sink - recent with the largest score: equal scores prefer the
 * lower index, NaN counts as -infinity, and a token on an absent page ranks
 * below every other.  The kept tokens close up in their order: token i of
 * the new sequence is token kept[b, h, i] of the old one, with its key, its
 * value and its score.  Positions belong to the keys (they were applied
 * before the cache was written), so attention over the trimmed cache is
 * attention over the kept tokens; a window, counted in cached tokens, is
 * not meant for trimmed sequences.  A sequence of len <= budget keeps all
 * of its tokens.
 *
 *   budget       >= 1;  sink, recent >= 0, sink + recent <= budget
 *   page_table   [B, max_pages]: where the tokens are
 *   new_page_table  NULL: in place, the kept tokens take the first places of
 *                page_table's pages, and places past them keep their bytes.
 *                Otherwise device int32 [B, new_max_pages]: the kept tokens
 *                are copied into these pages and the old ones keep their
 *                bytes (pages shared by several sequences are trimmed that
 *                way); no page may be in both tables.  new_max_pages *
 *                page_size must hold min(budget, max_pages * page_size).
 *   page_table_host, new_page_table_host
 *                host copies, optional: validated first (values in
 *                -1..num_pages-1; a page that the call writes is in the
 *                tables once)
 *   seq_lens     device int32 [B], clamped as in gdr_attention_decode
 *   new_lens     device int32 [B]: min(len, budget) (written); may be
 *                seq_lens itself
 *   kept         device int32 [B, Hkv, budget] (written), -1 past the new
 *                length
 *   workspace    device buffer of gdr_cache_evict_workspace_bytes bytes (0 for
 *                most sizes: NULL is accepted then), 16-byte aligned; needs no
 *                clearing; not to be shared with a concurrent call
 *
 * A kept token whose old or new page is absent is not moved.
 */
size_t gdr_cache_evict_workspace_bytes(int B, int Hkv, int max_pages, int page_size);

gdr_status gdr_cache_evict(enum gdr_dtype dt, int B, int Hkv, int D, int budget, int recent,
                           int sink, void *k_cache, void *v_cache, float *scores,
                           const int32_t *page_table, const int32_t *page_table_host,
                           int max_pages, const int32_t *new_page_table,
                           const int32_t *new_page_table_host, int new_max_pages,
                           int page_size, int num_pages, const int32_t *seq_lens,
                           int32_t *new_lens, int32_t *kept, void *workspace, size_t ws_bytes,
                           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_CACHE_H */
