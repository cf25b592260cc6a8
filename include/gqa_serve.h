/*
 * gqa_serve — serving operators beside the attention forward of gqa_attn.h, for NVIDIA B200
 * (sm_100a): attention over packed prompts, attention of a tree of drafted tokens over a
 * cache, and the pages of a paged KV cache (taking, sharing, compacting and freeing them).
 *
 * C ABI of libgqa_serve.so.  Plain pointers and sizes only; status codes, output types and
 * the general rules (device memory owned by the caller, 16-byte aligned tensors, calls
 * asynchronous on `stream`, argument errors returned before anything is launched or
 * written, the current device's kernels) are those of gqa_attn.h.
 *
 * Scratch comes from the library's own stream-ordered memory pool on `stream` and is freed
 * on it (as gqa_attn_fwd does), so calls on different streams and captured graphs share
 * none of it.
 */
#ifndef GQA_SERVE_H
#define GQA_SERVE_H

#include "gqa_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gqa_attn_fwd_varlen — the forward of gqa_attn_fwd over sequences of different lengths that
 * lie one behind the other, without padding.
 *
 *   q    bf16 [total_q, Hq, d]; row t starts q_row_stride elements after row t - 1.
 *   k, v bf16 [total_k, Hk, d], with k_row_stride and v_row_stride.  A row's heads are
 *        contiguous.  A stride is 0 (contiguous rows) or a multiple of 8 of at least one
 *        row's elements: Q, K and V may be columns of one packed projection.
 *   cu_seqlens_q, cu_seqlens_k   device int32 [B + 1]: sequence b has query rows
 *        [cu_seqlens_q[b], cu_seqlens_q[b+1]) and key rows [cu_seqlens_k[b],
 *        cu_seqlens_k[b+1]).  They start at any value >= 0 and do not decrease; bounds
 *        outside [0, total] are clamped to it.  Where they decrease, a sequence that starts
 *        before the end of an earlier one gives unspecified values in the rows of out and lse
 *        that it covers, and nothing else.
 *   causal   bottom-right aligned in each sequence: with Lq queries and Lk keys, query i
 *        sees key j iff j <= i + Lk - Lq.  A row that sees no key gets out = 0, lse = -inf.
 *   out  fp32 or bf16 [total_q, Hq, d] (out_dtype as in gqa_attn_fwd_kvcache).
 *   lse  fp32 [Hq, total_q].  Rows that belong to no sequence are left as they were, in both.
 *
 * What other sequences hold does not reach a sequence's result, not even infinities or NaN.
 * Within a sequence, a row that sees a key whose score is NaN or +inf gets NaN in out and lse; a
 * score of -inf weighs nothing, and a row all of whose scores are -inf is one that sees no key.
 * (With scale = 0, a product q.k of -inf leaves its row's values unspecified.)
 * A value of V that is not finite reaches every row of its 128-key block, as in gqa_attn_fwd.
 *
 * total_q = 0 returns GQA_OK and does nothing; total_k = 0 is a batch without keys (k and v
 * may be NULL).  Errors as gqa_attn_fwd; GQA_ERR_SHAPE also for a stride that is not
 * allowed, GQA_ERR_ALIGN for a cu_seqlens pointer that is not 4-byte aligned.
 */
GQA_API gqa_status gqa_attn_fwd_varlen(const void* q, long long q_row_stride, const void* k,
                                       long long k_row_stride, const void* v,
                                       long long v_row_stride, const int* cu_seqlens_q,
                                       const int* cu_seqlens_k, void* out, int out_dtype,
                                       float* lse, int B, int total_q, int total_k, int Hq,
                                       int Hk, int d, float scale, int causal, void* stream);

/*
 * gqa_attn_fwd_tree — attention of T drafted tokens per sequence, arranged as a tree, over a
 * KV cache that already holds their keys and values (speculative decoding's verification).
 *
 *   q               bf16 [B, T, Hq, d]: the nodes' queries.
 *   k_cache, v_cache  without a block_table: bf16 [B, Sk, Hk, d], as gqa_attn_fwd_kvcache;
 *                   with one: bf16 page pools [num_pages, page_size, Hk, d], as
 *                   gqa_attn_fwd_paged (then Sk is ignored; without one, max_pages_per_seq,
 *                   num_pages and page_size are).
 *   cache_seqlens   device int32 [B], required: L_b keys, the drafted ones included.
 *   tree_lens       device int32 [B] or NULL: sequence b has n_b = tree_lens[b] nodes,
 *                   clamped to [0, min(T, L_b)]; NULL: n_b = min(T, L_b).  Node j of sequence
 *                   b is key L_b - n_b + j.
 *   tree_mask       device int32 [B, T, ceil(T/32)], or with mask_shared != 0 one
 *                   [T, ceil(T/32)] for every sequence: bit j % 32 of word j / 32 of row i
 *                   is set iff node i sees node j.  Every node sees all L_b - n_b keys before
 *                   the tree.  Any bits are allowed (a node need not see itself); those of
 *                   nodes >= n_b are ignored.
 *   out, lse        [B, T, Hq, d] and [B, Hq, T].  A row that sees no key, and rows i >= n_b,
 *                   get out = 0 and lse = -inf.
 *
 * Keys at or past L_b do not reach the result, whatever they hold.  Scores and values of V
 * before L_b that are not finite count as in gqa_attn_fwd_varlen.  A table entry outside
 * [0, num_pages) reads as a page of zeros.  Errors as gqa_attn_fwd_paged; GQA_ERR_NULL for a
 * NULL tree_mask or cache_seqlens, GQA_ERR_ALIGN for an int32 pointer that is not 4-byte
 * aligned.
 */
GQA_API gqa_status gqa_attn_fwd_tree(const void* q, const void* k_cache, const void* v_cache,
                                     const int* block_table, int max_pages_per_seq, int num_pages,
                                     int page_size, const int* cache_seqlens, const int* tree_mask,
                                     int mask_shared, const int* tree_lens, void* out,
                                     int out_dtype, float* lse, int B, int T, int Sk, int Hq,
                                     int Hk, int d, float scale, void* stream);

/*
 * The pages of a cache.  Their state is three device int32 arrays of the caller's:
 *
 *   block_table    [S, max_pages_per_seq], as gqa_attn_fwd_paged reads it.  Sequence slot s of
 *                  length L uses its first ceil(L / page_size) entries; these calls set an
 *                  entry that is given up to -1 and neither read nor write the others.
 *   cache_seqlens  [S], each slot's length; 0 = the slot is free.
 *   page_refs      [num_pages]: how many table entries name each page; 0 = the page is free.
 *                  Pages that the caller handles itself keep any other value (e.g. 1).
 *
 * Calls that read or change the same state are ordered by the caller, on one stream or with
 * events.  page_size is a power of two >= 16.  Pages are taken lowest number first, for the requests
 * in their order: the outcome does not depend on scheduling.  Each request's outcome is
 * written to status[i] (device int32):
 */
typedef enum {
    GQA_CACHE_DONE = 0,
    GQA_CACHE_NO_PAGES = 1, /* not enough free pages for this request and those before it   */
    GQA_CACHE_INVALID = 2,  /* a slot or length out of range, a slot named by an earlier    */
                            /* request, or a list that breaks the call's rules              */
    GQA_CACHE_SHARED = 3    /* the request would leave or write rows in part of a page that */
                            /* another sequence uses too                                    */
} gqa_cache_status;

/* The most requests that one gqa_cache_resize or gqa_cache_fork takes. */
#define GQA_CACHE_MAX_REQUESTS 4096

/*
 * gqa_cache_resize — gives each listed slot the pages for its new length: more pages for a
 * longer one, fewer for a shorter one, none for 0 (the sequence is freed).
 *
 *   slots     [n], or NULL: slots 0 .. n-1.   new_lens  [n], 0 <= new_lens[i] <=
 *             max_pages_per_seq * page_size.
 *
 * The pages given up in the call are free for its growing sequences.  A request whose status
 * is not GQA_CACHE_DONE leaves its sequence as it was.  GQA_CACHE_SHARED: the page that
 * holds row min(old, new) would stay partly filled while another sequence names it too.
 * Once a request finds too few pages, later requests that need some find too few as well.
 * The rows of new pages are not written.  GQA_ERR_SHAPE for n < 0, n > GQA_CACHE_MAX_REQUESTS
 * or sizes < 1, GQA_ERR_NULL for a missing array, GQA_ERR_ALIGN for one that is not 4-byte
 * aligned.  n = 0 does nothing.
 */
GQA_API gqa_status gqa_cache_resize(int* block_table, int* cache_seqlens, int* page_refs, int S,
                                    int max_pages_per_seq, int num_pages, int page_size,
                                    const int* slots, const int* new_lens, int n, int* status,
                                    void* stream);

/*
 * gqa_cache_fork — makes each child slot a copy of its parent: the parent's whole pages are
 * shared (their counts rise), the rows of its last, partly filled page are copied to a new
 * page.  What a child held before is given up first, and those pages are free for the call.
 *
 *   k_pages, v_pages  [layers, num_pages, page_size, row_bytes]: the pools of all layers, of
 *             any element type; row_bytes (one token's heads) is a multiple of 16.
 *   parents, children  [n] slots.  A child is named once, and is no request's parent, except
 *             that a request with child = parent changes nothing (GQA_CACHE_DONE).
 *
 * All requests see the state before the call.  GQA_CACHE_NO_PAGES leaves the child empty.
 * Rows of the new page past the parent's length are left as they were.  Errors as
 * gqa_cache_resize; GQA_ERR_SHAPE also for layers < 1 or a row_bytes that is not allowed.
 */
GQA_API gqa_status gqa_cache_fork(void* k_pages, void* v_pages, int layers, long long row_bytes,
                                  int* block_table, int* cache_seqlens, int* page_refs, int S,
                                  int max_pages_per_seq, int num_pages, int page_size,
                                  const int* parents, const int* children, int n, int* status,
                                  void* stream);

/*
 * gqa_cache_compact — after a verification: of the n_s drafted nodes at the end of each slot
 * s (n_s as gqa_attn_fwd_tree's), the rows of the accepted ones are moved together behind the
 * context, in all layers, and the sequence ends behind them; pages that hold no row any more
 * are given up.
 *
 *   keep       device int32 [S, T]: the accepted nodes of slot s, increasing, the first
 *              keep_lens[s] of row s.  keep_lens  [S], 0 <= keep_lens[s] <= n_s.
 *   tree_lens  [S] or NULL, as gqa_attn_fwd_tree.   status  [S].
 *
 * The new length is L_s - n_s + keep_lens[s].  A list that does not increase or leaves
 * [0, n_s) is GQA_CACHE_INVALID; GQA_CACHE_SHARED: a page that would keep rows at or past
 * L_s - n_s, or that ends there partly filled, is named by another sequence too.  Both leave
 * the slot as it was.  Errors as gqa_cache_fork.
 */
GQA_API gqa_status gqa_cache_compact(void* k_pages, void* v_pages, int layers, long long row_bytes,
                                     int* block_table, int* cache_seqlens, int* page_refs, int S,
                                     int max_pages_per_seq, int num_pages, int page_size,
                                     const int* keep, const int* keep_lens, const int* tree_lens,
                                     int T, int* status, void* stream);

/* gqa_attn_device_status of this library's kernels. */
GQA_API gqa_status gqa_serve_device_status(int reset);

#ifdef __cplusplus
}
#endif

#endif /* GQA_SERVE_H */
