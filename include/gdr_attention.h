/*
 * gdr_attention.h -- the attention layers of a placement beside the decode
 * over their cache (gdr_cache.h): the attention of whole prompts and its
 * gradients (MI355X, gfx950).
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
 * Limits (GDR_EUNSUPPORTED): T_total < 2^30, T_total * Hq < 2^31, Hq * D <=
 * 2^20.
 *
 * Numerics: fp32 accumulation, logits, softmax statistics and weights; with
 * bf16 inputs a weight enters the product with V as one bf16 number, off by
 * at most 2^-8 of it, and o is rounded once.
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
 * gradient is rounded once.
 */
size_t gdr_attention_backward_workspace_bytes(enum gdr_dtype dt, int B, int T_total, int Hq,
                                              int Hkv, int D);

gdr_status gdr_attention_backward(enum gdr_dtype dt, int B, int T, int T_total, int Hq, int Hkv,
                                  int D, float scale, int window, const void *q, const void *k,
                                  const void *v, const int32_t *cu_seqlens,
                                  const int32_t *cu_seqlens_host, const void *o,
                                  const float *lse, const void *d_o, void *dq, void *dk,
                                  void *dv, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_ATTENTION_H */
