/*
 * oda_serve.h - what a served request needs around the decode step of oda.h: attention over a whole
 * prompt, attention for a tree of drafted tokens over the paged cache, the write of many positions
 * into the pages, and the choice of a token from the logits.
 *
 * The method notes ("On-Demand Attention：让语言模型按需读取完整历史") start from a fully retained
 * cache C_{t-1} and decode one token a step [notes §2.1, §2.3]; how the cache was filled, drafted
 * tokens and sampling are outside them.  These calls keep their index sets: a prompt row at position t
 * reads S^F_t = {1..t} (oda_attend_full_prompt) or S^L_t = {1..min(s,t)} U {max(1,t-w+1)..t}
 * (oda_attend_local_prompt), as the decode calls do.
 *
 * Same conventions as oda.h: device pointers unless stated otherwise, asynchronous on `stream`, no
 * allocation, graph capturable, calls on one context ordered on one stream, argument errors returned
 * before anything is launched (a context of another device than the current one among them), data-
 * dependent violations reported in the context's error word.  Heads, sinks, window, page table width and
 * batch come from the context's configuration.
 *
 * Packed rows: the rows of sequence i are cu_rows[i] .. cu_rows[i+1] - 1 of every packed tensor
 * (device int32 [n_seqs + 1], 0 <= cu_rows[i] <= cu_rows[i+1] <= n_rows; a sequence may be empty).
 * Output rows outside all sequences are left as they were.  A sequence whose bounds break this rule
 * counts as empty and sets ODA_DEVERR_ROW_RANGE; where bounds overlap, what the rows in common and
 * behind them give is undefined.
 */
#ifndef ODA_SERVE_H
#define ODA_SERVE_H

#include "oda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bit of the sticky device error word. */
#define ODA_DEVERR_ROW_RANGE 0x8  /* cu_rows, a picked row or a parent out of range              */

#define ODA_MAX_TREE 64           /* nodes of one drafted tree                                   */
#define ODA_MAX_VOCAB 262144      /* logits of one row                                           */

/* Causal attention over whole prompts, n_seqs (1..ODA_MAX_BATCH) packed sequences of any lengths.
 * The row at place p (0-based) of its sequence is position t = p + 1; query head h reads KV head
 * h / (Hq/Hkv):
 *   out = sum_{j in S_t} softmax_j(q . k_j / sqrt(128)) v_j,  S_t = S^F_t (full) or S^L_t (local).
 * q: bf16, head h of row r at q + r*q_stride + h*128; k, v: bf16, KV head c of row r at
 * + r*kv_stride + c*128 (strides in elements, multiples of 8, >= Hq*128 and Hkv*128; so q, k and v
 * may be columns of one projection output); out: bf16 [n_rows][Hq][128], apart from them.  q, k, v and
 * out 16-byte aligned.  Products of bf16 operands with fp32 sums; softmax statistics fp32; the weights are
 * rounded to bf16 before the product with V, and the output once at the end.  A NaN or infinity in
 * one sequence's rows never reaches another sequence.  Within its own, one of k reaches the rows that see
 * it, as the formula says (NaN, but for a score of -inf beside finite ones, whose weight is 0); one of v
 * makes every row that sees it NaN and may make others NaN.  A finite v in a place that a row does not see has
 * weight 0.  The sums of weights (up to 2^8 each) times v are held unnormalised: over n positions, v beyond
 * 2^119 / n may overflow in a row that sees it. */
oda_status oda_attend_full_prompt(oda_ctx* ctx, int32_t n_seqs, int64_t n_rows,
                                  const int32_t* cu_rows, const void* q, const void* k,
                                  const void* v, int64_t q_stride, int64_t kv_stride, void* out,
                                  cudaStream_t stream);
oda_status oda_attend_local_prompt(oda_ctx* ctx, int32_t n_seqs, int64_t n_rows,
                                   const int32_t* cu_rows, const void* q, const void* k,
                                   const void* v, int64_t q_stride, int64_t kv_stride, void* out,
                                   cudaStream_t stream);

/* Attention for a tree of drafted tokens over the cache (bf16 pages), full set, all sequences of
 * the context's batch with flag[b] != 0 (flag NULL: all).  Sequence b has cached positions
 * 1..pos[b]-1 and the nodes cu_rows[b] .. cu_rows[b+1] - 1 (cu_rows [batch + 1]; 0..ODA_MAX_TREE
 * nodes, more sets ODA_DEVERR_ROW_RANGE and the sequence counts as empty).  parent[r] is node r's
 * parent counted inside its sequence (0-based) and smaller than the node's own index, or -1 for a
 * child of the last cached position; a parent out of range sets ODA_DEVERR_ROW_RANGE and counts as
 * -1.  Node i reads every cached position, its ancestors and itself.  q: bf16 [n_rows][Hq][128];
 * k_new, v_new: bf16 [n_rows][Hkv][128] (the nodes' own keys and values, never in the cache);
 * out: bf16 [n_rows][Hq][128], apart from them; all 16-byte aligned; 1 <= n_rows <= batch*ODA_MAX_TREE (0 nodes:
 * cu_rows all equal).  Rows of skipped sequences are left as they were.  A page-table entry outside
 * the pool sets ODA_DEVERR_PAGE_RANGE, a position outside the table's capacity ODA_DEVERR_POS_RANGE
 * (the sequence is skipped); the outputs of a sequence with a bad page are undefined.  Arithmetic and
 * what NaN and infinities reach as in the prompt calls; the cached range is split over the SMs and joined in a fixed order, so equal
 * calls give equal bits. */
oda_status oda_attend_full_tree(oda_ctx* ctx, const oda_kv_layer* layer, const int32_t* page_table,
                                const int32_t* pos, const int32_t* flag, int64_t n_rows,
                                const int32_t* cu_rows, const int32_t* parent, const void* q,
                                const void* k_new, const void* v_new, void* out,
                                cudaStream_t stream);

/* Writes many positions of every sequence of the batch into the cache: the i-th row of sequence b
 * (i = 0 .. cu_rows[b+1] - cu_rows[b] - 1, cu_rows [batch + 1]) goes to position pos[b] + i of all
 * n_layers pools (host array).  Its source is staging row rows[cu_rows[b] + i], or cu_rows[b] + i where
 * rows is NULL (then n_rows <= n_stage): k_stage, v_stage bf16 [n_layers][n_stage][Hkv][128], 16-byte
 * aligned.  rows: device int32 [n_rows]; an entry outside 0..n_stage-1 sets ODA_DEVERR_ROW_RANGE and
 * writes nothing; the same row may be picked twice.  A position outside the table's capacity sets
 * ODA_DEVERR_POS_RANGE, a page-table entry outside a pool ODA_DEVERR_PAGE_RANGE; neither writes.
 * Where h_stage (fp32 [n_stage][head_in_dim]) and h_prev (fp32 [batch][head_in_dim]) are given (both or
 * none, 16-byte aligned), h_prev[b] <- the hidden row of the sequence's last appended position; sequences
 * with no rows keep theirs.  Where pos_next (int32 [batch]) is given, pos_next[b] <- pos[b] + the
 * sequence's row count (unchanged where pos[b] < 1 or the bounds are bad); it may be pos itself.  With
 * rows of a prompt this fills the cache, layer by layer (pos_next NULL until the last layer) or all
 * layers at once; with rows picking an accepted path it commits drafted tokens. */
oda_status oda_append(oda_ctx* ctx, const oda_kv_layer* layers, int32_t n_layers,
                      const int32_t* page_table, const int32_t* pos, int64_t n_rows, int64_t n_stage,
                      const int32_t* cu_rows, const int32_t* rows, const void* k_stage,
                      const void* v_stage, const float* h_stage, float* h_prev, int32_t* pos_next,
                      cudaStream_t stream);
/* The same into fp8 pages: every row is quantised as oda_commit_fp8 does.  A page that is filled in part is
 * read and written back with its other bytes, so sequences must not share a page that they write to, and
 * calls that run at once must not write to the same one. */
oda_status oda_append_fp8(oda_ctx* ctx, const oda_kv8_layer* layers, int32_t n_layers,
                          const int32_t* page_table, const int32_t* pos, int64_t n_rows,
                          int64_t n_stage, const int32_t* cu_rows, const int32_t* rows,
                          const void* k_stage, const void* v_stage, const float* h_stage,
                          float* h_prev, int32_t* pos_next, cudaStream_t stream);

/* One token for each of n_rows (1..65535) rows of fp32 logits (row r at logits + r*row_stride, vocab
 * values, 4-byte aligned; vocab 1..ODA_MAX_VOCAB), from a given uniform number u[r] in [0, 1).  The
 * settings are device arrays of n_rows, each may be NULL: temperature T (NULL: 1), top_k (NULL: off),
 * top_p (NULL: off), min_p (NULL: off).  With z_i = (l_i - max l) / T and w_i = e^z_i:
 *   S1 = the top_k largest l_i, ties to the lowest index (top_k < 1 or >= vocab: all);
 *   S2 = the shortest prefix of S1, largest first, ties to the lowest index, whose mass is >= top_p
 *        times S1's (top_p >= 1 or NaN: all; top_p <= 0: the first);
 *   S3 = {i in S2 : w_i >= min_p}  (min_p <= 0 or NaN: all; > 1 keeps the largest only);
 *   token = the first i of S3, in index order, whose running mass exceeds u * mass(S3);
 *   prob  = w_token / mass(S3) (fp32, may be NULL).
 * T <= 0 or NaN: the lowest index of the largest logit, prob 1.  NaN and -inf logits are masked (never
 * chosen); where +inf logits are present only they count, with equal weights; a row with nothing
 * left gives token -1 and prob 0.  u is clamped to [0, 1), NaN counts as 0.  Weights are computed in
 * 64 bits and summed as whole multiples of 2^-43 of the largest weight (smaller weights count as 0), so the
 * draw does not depend on the order of any sum.  Top-p without top-k over
 * more than 1024 values places its end with fp32 sums of the weights below e^-3 of the largest, in an order
 * that depends only on the row's length and its place modulo 16 bytes: equal calls give equal bits, and
 * the end may lie some values off, by less than 2^-16 of the mass (1.5e-7 is the most that was measured). */
oda_status oda_sample(oda_ctx* ctx, int32_t n_rows, int32_t vocab, int64_t row_stride,
                      const float* logits, const float* temperature, const int32_t* top_k,
                      const float* top_p, const float* min_p, const float* u, int32_t* token,
                      float* prob, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* ODA_SERVE_H */
