/*
 * gdr_attention.h -- the attention layers of a placement beside the decode
 * over their cache (gdr_cache.h): the attention of whole prompts and its
 * gradients, the attention of a tree of drafted tokens over the cache, what is
 * kept of such a tree, and the page tables that follow the requests' lengths
 * (MI355X, gfx950).
 *
 * The conventions of gdr.h and gdr_cache.h hold here as well (device pointers,
 * dense row-major tensors, 16-byte alignment -- page tables, lengths, offsets
 * and other int32 arrays 4-byte --, host checks before any HIP call, no
 * allocation or synchronisation, gdr_status codes, gdr_last_error, GDR_DEBUG).
 * Results are the same bits on every run: no floating-point sum goes through
 * atomics.  Outputs overlap no input except where a call says so.
 *
 * Supported shapes: D in {64, 128}; Hq a multiple of Hkv; dtypes GDR_F32 and
 * GDR_BF16; the paged cache as in gdr_cache.h.
 */
#ifndef GDR_ATTENTION_H
#define GDR_ATTENTION_H

#include "gdr_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Attention over whole prompts: every token of a sequence attends to the
 * tokens up to its own, or to the last `window` of them.  With i and j
 * counted within a sequence and query head h reading key-value head
 * h / (Hq / Hkv):
 *     A_i = { j : j <= i,  j > i - window if window > 0 },
 *     s_ij = scale * q_i . k_j,   lse_i = ln sum_A e^{s_ij},
 *     w_ij = e^{s_ij - lse_i},    o_i = sum_A w_ij v_j.
 * A row whose e^{s_ij} are all zero gives o = 0 and lse = -inf.  What lies in
 * tokens a row does not attend to, and in other sequences, has no part in its
 * result, NaN and infinities included.
 *
 *   B            sequences (>= 0)
 *   T            tokens per sequence (cu_seqlens == NULL; T_total is then
 *                B * T)
 *   T_total      rows of q, k, v and o
 *   scale        multiplies the dot products (finite)
 *   window       0: every token up to the row's own; W > 0: the last W
 *   q, o         [T_total, Hq, D] dt: [B, T, Hq, D], or packed
 *   k, v         [T_total, Hkv, D] dt
 *   cu_seqlens   NULL, or device int32 [B+1]: sequence b is rows
 *                [cu_seqlens[b], cu_seqlens[b+1]); rows at or past
 *                cu_seqlens[B] belong to no sequence (a padded batch): they
 *                are not read, and o and lse keep their bytes there
 *   cu_seqlens_host  host copy, optional: validated first (starts at 0, does
 *                not decrease, ends at or below T_total)
 *   lse          [T_total, Hq] fp32 or NULL (the backward pass needs it)
 *
 * Limits (GDR_EUNSUPPORTED): T_total < 2^29, (T_total / 64 + B) * Hq < 2^24
 * (T_total * Hq < 2^30 for a few sequences), Hq * D <= 2^20.
 *
 * Numerics: fp32 accumulation, logits, softmax statistics and weights; with
 * bf16 inputs a weight enters the product with V as one bf16 number, off by
 * at most 2^-8 of it, and o is rounded once.  Values of V up to 2^127 in
 * magnitude give finite results (those past 2^120 / tokens at up to three
 * times the cost).
 */
gdr_status gdr_attention_prefill(enum gdr_dtype dt, int B, int T, int T_total, int Hq, int Hkv,
                                 int D, float scale, int window, const void *q, const void *k,
                                 const void *v, const int32_t *cu_seqlens,
                                 const int32_t *cu_seqlens_host, void *o, float *lse,
                                 void *stream);

/*
 * The gradients of gdr_attention_prefill for an upstream gradient d_o of o
 * (none of lse):
 *     delta_i = d_o_i . o_i,   ds_ij = w_ij (d_o_i . v_j - delta_i),
 *     dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,
 *     dv_j = sum_i w_ij d_o_i,
 * the sums of dk and dv over every row that attends to token j, in all query
 * heads of its key-value head.
 *
 *   dt .. v, cu_seqlens, cu_seqlens_host
 *                as in gdr_attention_prefill
 *   o, lse       what that call gave for these inputs
 *   d_o          [T_total, Hq, D] dt
 *   dq           [T_total, Hq, D] dt (written)
 *   dk, dv       [T_total, Hkv, D] dt (written); rows behind the last
 *                sequence keep their bytes in all three
 *   workspace    device buffer of gdr_attention_backward_workspace_bytes
 *                bytes, 16-byte aligned; needs no clearing; not to be shared
 *                with a concurrent call
 *
 * The gradients of a token that a row with a NaN or an infinity attends to,
 * and of a row that attends to one, are not finite numbers or unspecified
 * ones; no other gradient is touched by it.
 *
 * Numerics: fp32 accumulation, weights and their gradients; with bf16 inputs
 * w_ij and ds_ij enter the products as one bf16 number each, and every
 * gradient is rounded once (off by 2.5e-3 of its norm in the mean, 1.9e-3 with
 * unrounded w_ij and ds_ij; o of gdr_attention_prefill by 2.2e-3, 1.65e-3;
 * gdr_attention_decode and gdr_attention_tree take two numbers a weight).
 */
size_t gdr_attention_backward_workspace_bytes(enum gdr_dtype dt, int B, int T_total, int Hq,
                                              int Hkv, int D);

gdr_status gdr_attention_backward(enum gdr_dtype dt, int B, int T, int T_total, int Hq, int Hkv,
                                  int D, float scale, int window, const void *q, const void *k,
                                  const void *v, const int32_t *cu_seqlens,
                                  const int32_t *cu_seqlens_host, const void *o,
                                  const float *lse, const void *d_o, void *dq, void *dk,
                                  void *dv, void *workspace, size_t ws_bytes, void *stream);

/*
 * Attention of a tree of drafted tokens over the cache.  The n_tok newest
 * tokens of sequence b (places seq_lens[b] - n_tok .. seq_lens[b] - 1, keys
 * and values appended first) are a forest: draft t follows draft
 * parents[b, t] < t, or the context where parents[b, t] is anything else (-1).
 * With c = seq_lens[b] - n_tok the context's tokens, d(t) the number of
 * drafts before t on its way to the context, and the position p = c + d(t),
 * row t attends to
 *     the context's tokens j < c, j > p - window if window > 0, and
 *     the places c + u of the drafts u on its way, itself included, whose
 *     positions are above p - window if window > 0,
 * as far as they are at 0 or above and on a present page.  (A chain, parents
 * t - 1, is gdr_attention_decode.)  Everything else is as there: the softmax,
 * rows without tokens, absent pages, the numerics (sums of weights times
 * values are divided last: values below 2^128 / tokens in magnitude give
 * finite results), the workspace (gdr_attention_workspace_bytes, without
 * scores).
 *
 *   n_tok        drafts per sequence, 0..64 (a smaller tree is padded with
 *                drafts that follow the context)
 *   parents      device int32 [B, n_tok]
 */
gdr_status gdr_attention_tree(enum gdr_dtype dt, int B, int n_tok, int Hq, int Hkv, int D,
                              float scale, int window, const void *q, const void *k_cache,
                              const void *v_cache, const int32_t *page_table,
                              const int32_t *page_table_host, int max_pages, int page_size,
                              int num_pages, const int32_t *seq_lens, const int32_t *parents,
                              void *o, void *workspace, size_t ws_bytes, void *stream);

/*
 * Keep one way through each sequence's tree of drafts: the tokens from the
 * context to draft leaf[b] take the places behind the context, in their
 * order, and the sequence ends there.
 *
 *   n_tok, seq_lens, parents
 *                as in gdr_attention_tree (seq_lens with the drafts)
 *   leaf         device int32 [B]: the last draft kept; a value outside
 *                0..n_tok-1 (-1) keeps none
 *   scores       NULL, or the accumulated weights, moved along
 *   new_lens     device int32 [B]: max(seq_lens[b] - n_tok, 0) + the kept
 *                drafts that have a place (written); may be seq_lens itself
 *   path         device int32 [B, n_tok]: the kept drafts from the context
 *                on, -1 past them (written)
 *
 * Lengths are clamped as in gdr_attention_decode; drafts at places below 0
 * (a sequence shorter than n_tok) are not kept.  The pages of the drafts
 * belong to one sequence each.  A token whose old or new page is absent is
 * not moved.  Places past the new length keep their bytes.
 */
gdr_status gdr_cache_accept(enum gdr_dtype dt, int B, int n_tok, int Hkv, int D,
                            const int32_t *page_table, int max_pages, int page_size,
                            int num_pages, const int32_t *seq_lens, const int32_t *parents,
                            const int32_t *leaf, void *k_cache, void *v_cache, float *scores,
                            int32_t *new_lens, int32_t *path, void *stream);

/*
 * Page tables that follow the sequences' lengths.  Sequence b holds
 * seq_lens[b] tokens, on the pages of the first ceil(seq_lens[b] / page_size)
 * columns of its row; the call makes them the pages of want[b] tokens.  The
 * tables are all there is: a page is free if no row keeps it, so that every
 * sequence that holds pages has to have a row (one that is not to change asks
 * for what it has), and pages that several sequences share stay while one of
 * them keeps them.
 *   * A row that shrinks drops its entries past the new length (-1), and
 *     their pages are free if no other row keeps them.
 *   * Rows that grow are served in their order, their new columns in theirs,
 *     with the free pages from the lowest number up.  A row that asks for
 *     pages is served in full or not at all: it is if the pages asked for by
 *     the rows up to it (itself included, served or not) are at most the free
 *     ones.  A row that grows within its last page asks for none.
 *   * new_lens[b] = want[b], or seq_lens[b] for a row that is not served.
 *   * Columns past a row's old and new pages are neither read nor written.  They
 *     are to hold -1 (a call that shortens lengths in another way, as
 *     gdr_cache_evict, is followed by one with the old lengths and the new ones):
 *     then tokens appended to a row that was not served fall on absent pages.
 *     Such a row has no drafts: gdr_attention_tree and gdr_cache_accept would
 *     take its newest tokens for them (leaf -1 moves nothing).
 * A table of one column whose rows hold 0 or 1 tokens is a slot map of a
 * state pool (gdr_decode_tokens, gdr_prefill_varlen_pool).
 *
 *   max_pages    columns of page_table
 *   page_size    tokens of a page (>= 1)
 *   num_pages    pages there are, 0..2^20 (GDR_EUNSUPPORTED above, and for
 *                (num_pages + B) * page_size >= 2^31 tokens)
 *   page_table   device int32 [B, max_pages] (read and written)
 *   seq_lens, want  device int32 [B], clamped to 0..max_pages * page_size
 *   new_lens     device int32 [B] (written); may be seq_lens or want
 *   cu_seqlens   NULL, or device int32 [B+1] (written): where the tokens that
 *                the rows grow by lie in a packed batch (sums of max(0,
 *                new_lens[b] - seq_lens[b])), for gdr_cache_append with start
 *                = seq_lens
 *   free_pages   NULL, or device int32 [1] (written): free pages after the
 *                call
 */
gdr_status gdr_cache_resize(int B, int max_pages, int page_size, int num_pages,
                            int32_t *page_table, const int32_t *seq_lens, const int32_t *want,
                            int32_t *new_lens, int32_t *cu_seqlens, int32_t *free_pages,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_ATTENTION_H */
