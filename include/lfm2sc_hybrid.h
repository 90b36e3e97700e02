/*
 * lfm2sc_hybrid.h -- C ABI of the operators that sit next to the ShortConv in
 * the LFM2 hybrid decoder, in the same library (liblfm2sc.so):
 *
 *   lfm2sc_attn_prefill / lfm2sc_attn_backward   causal attention with grouped
 *        heads over packed prompts, and its gradients (training);
 *   lfm2sc_attn_cached    attention of new tokens -- one per sequence (decode) or
 *        the block of lfm2sc_verify_window -- over a paged key/value cache whose
 *        first keys are a prefix shared by the whole batch;
 *   lfm2sc_accept_drafts  verification of drafted tokens; its keep_len is the
 *        accept_len that lfm2sc_commit_window takes.
 *
 * The conventions of lfm2sc.h hold: device pointers owned by the caller, no
 * device memory allocated, asynchronous on `stream`, row-major layouts with
 * strides in elements, the same status codes, lfm2sc_last_error and
 * lfm2sc_status_string, LFM2SC_CHECK=1 for checks of device-side data.  Calls
 * launch kernels only (no memset, no copy), so they can be captured into a graph.
 * Results are deterministic: no atomics, every sum in a fixed order.  Sizes that
 * need 2^32 or more work-items in one launch (about 2^24 blocks of 32 to 128 rows
 * times heads) are refused with LFM2SC_ERR_BAD_SHAPE.
 *
 * Attention, shared by its entry points
 * -------------------------------------
 *  - dtype LFM2SC_BF16 only (else LFM2SC_ERR_UNSUPPORTED).  Scores, softmax
 *    statistics and all sums are fp32; the probabilities (and, backward, the
 *    score gradients) are rounded to bf16 as operands of the second product;
 *    outputs are rounded once.
 *  - D, the head dimension, is 64 or 128 (else LFM2SC_ERR_UNSUPPORTED);
 *    num_heads is a positive multiple of num_kv_heads; query head h uses
 *    key/value head h / (num_heads / num_kv_heads).
 *  - A row holds its heads one after the other (head h in columns
 *    [h*D, (h+1)*D)); strides are multiples of 8 elements, at least heads * D,
 *    below 2^22; pointers are 16-byte aligned (lse and int32 arrays: 4-byte), so
 *    q, k and v may be column ranges of one projection's rows.
 *  - scale multiplies q.k; finite and > 0.  total_T, prefix_len and max_pages *
 *    page_size are below 2^30.
 *  - An infinity or NaN in k or v of a token reaches the rows that see the token,
 *    and may reach earlier rows of the same sequence within 127 tokens of it
 *    (their probability of it is 0, but 0 * infinity is not; over a cache, any
 *    earlier row of the sequence's L).  One in q, out or d_out of a row reaches
 *    dk and dv of the keys that the row sees, and may reach those of later keys
 *    within 127 tokens.  It reaches no other sequence.
 */
#ifndef LFM2SC_HYBRID_H
#define LFM2SC_HYBRID_H

#include "lfm2sc.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Causal attention over packed prompts.
 *
 * q, k, v    [total_T][*_stride]; cu_seqlens [num_seqs+1] int32 as for
 *            lfm2sc_prefill_ragged: sequence i owns rows [cu[i], cu[i+1]), and its
 *            row t attends its rows 0..t.  Offsets are clamped to [0, total_T].
 * out        [total_T][out_stride]  softmax(scale q k^T) v.
 * lse        [num_heads][total_T] fp32 or NULL: ln sum_j exp(scale q.k_j), which
 *            the backward takes.
 * Rows that belong to no sequence are not written.
 */
int lfm2sc_attn_prefill(int dtype, int D, int num_heads, int num_kv_heads,
                        const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                        const void* v, int64_t v_stride, int64_t total_T,
                        const int32_t* cu_seqlens, int num_seqs, float scale,
                        void* out, int64_t out_stride, float* lse, void* stream);

/* Bytes of workspace lfm2sc_attn_backward needs; 0 for invalid sizes. */
size_t lfm2sc_attn_backward_workspace_bytes(int dtype, int D, int num_heads, int num_kv_heads, int64_t total_T,
                                            int num_seqs);

/*
 * Backward of lfm2sc_attn_prefill: with p = exp(scale q.k - lse),
 * delta = d_out.out and ds = p (d_out.v - delta),
 *   dv[j] = sum p d_out,  dk[j] = scale sum ds q  (over the rows and the heads of
 *   the group that see key j),  dq[t] = scale sum_j ds k[j].
 *
 * out, lse   as the forward wrote them; d_out [total_T][d_out_stride].
 * dq, dk, dv [total_T][*_stride], overwritten; rows of no sequence are not
 *            written.  They may be column ranges of one buffer.
 * workspace  lfm2sc_attn_backward_workspace_bytes(...) bytes, 16-byte aligned.
 */
int lfm2sc_attn_backward(int dtype, int D, int num_heads, int num_kv_heads,
                         const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                         const void* v, int64_t v_stride, int64_t total_T,
                         const int32_t* cu_seqlens, int num_seqs, float scale,
                         const void* out, int64_t out_stride, const float* lse,
                         const void* d_out, int64_t d_out_stride,
                         void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                         void* dv, int64_t dv_stride,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace lfm2sc_attn_cached needs; 0 for invalid sizes, when num_seqs
 * or L is 0, and for few keys, which need none (workspace may then be NULL).
 */
size_t lfm2sc_attn_cached_workspace_bytes(int dtype, int D, int num_heads, int num_kv_heads, int num_seqs, int L,
                                          int prefix_len, int max_pages, int page_size);

/*
 * Attention of L new tokens per sequence over the cache.
 *
 * q            [num_seqs*L][q_stride]; row i*L+s is token s of sequence i (the row
 *              order of lfm2sc_verify_window; L = 1: decode).
 * k_pages, v_pages  pools of num_pages pages of page_size tokens; token t of page
 *              p is row p*page_size + t, kv_stride elements apart (>= num_kv_heads
 *              * D, multiple of 8).  page_size is a power of two, num_pages *
 *              page_size < 2^31.  The new tokens' keys and values are in the cache
 *              before the call.
 * prefix_pages [ceil(prefix_len / page_size)] int32, prefix_len >= 0: the shared
 *              keys, seen by every row.  May be NULL when prefix_len is 0.
 * page_table   [num_seqs][max_pages] int32: each sequence's own pages.  Entries past
 *              ceil(suffix_len[i] / page_size) are not used and may hold anything.
 * suffix_len   [num_seqs] int32: its own keys, the L new ones included; clamped to
 *              [0, max_pages * page_size].  Row i*L+s sees the prefix and own keys
 *              0 .. suffix_len[i]-L+s.  A row that sees no key gets zeros.
 * A page number outside [0, num_pages) reads as the nearest page.  Cache rows past
 * a sequence's length are never read.
 * out          [num_seqs*L][out_stride].
 * workspace    16-byte aligned.
 */
int lfm2sc_attn_cached(int dtype, int D, int num_heads, int num_kv_heads,
                       const void* q, int64_t q_stride, int num_seqs, int L,
                       const void* k_pages, const void* v_pages, int64_t kv_stride, int num_pages, int page_size,
                       const int32_t* prefix_pages, int prefix_len,
                       const int32_t* page_table, int max_pages, const int32_t* suffix_len, float scale,
                       void* out, int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace lfm2sc_accept_drafts needs; 0 for invalid sizes (and when
 * num_seqs is 0).
 */
size_t lfm2sc_accept_drafts_workspace_bytes(int num_seqs, int L, int V);

/*
 * Verification of drafted tokens (speculative sampling).
 *
 * Passage: SGLang PR 31041 summary, implementation item 2 and its related-work
 * note on the post-verify commit: the accept boundary that selects the tape's
 * window.  The rule is the published one for speculative sampling.
 *
 * dtype        of both probability arrays: LFM2SC_BF16 or LFM2SC_F32.
 * target_probs [num_seqs*(L+1)][target_stride], V columns: row i*(L+1)+s is the
 *              target's distribution of the token after s drafts.
 * draft_probs  [num_seqs*L][draft_stride] or NULL (deterministic drafts: the
 *              draft's own probability counts as 1).
 * draft_tokens [num_seqs][L] int32; one outside [0, V) is never accepted.
 * num_drafts   [num_seqs] int32 or NULL (= L for all), clamped to [0, L].  Draft
 *              tokens and numbers past it are not used and may hold anything.
 * u_accept     [num_seqs][L] fp32 and u_sample [num_seqs] fp32: uniform numbers in
 *              [0, 1) from the caller.
 * accept_len   [num_seqs] int32: a, the number of leading drafts s with
 *              u_accept[s] * q_s(x_s) < p_s(x_s).
 * keep_len     [num_seqs] int32 or NULL: a + 1, the rows to keep of a verify block
 *              that starts with the last sampled token: what lfm2sc_commit_window
 *              takes for a tape of L+1 steps.
 * next_token   [num_seqs] int32: drawn from r = p_a when every draft was
 *              accepted, else max(p_a - q_a, 0) (p_a without the draft's token
 *              when draft_probs is NULL), else p_a where that is all zero: the
 *              lowest j with r_0 + .. + r_j > u_sample * sum r.  Sums are fp64; rows
 *              need not add up to 1.  In r, NaN and negative entries of p_a and q_a
 *              count as 0 (accept_len's comparison takes them as they are: a NaN
 *              is never accepted).  For
 *              u_sample outside [0, 1) the last j with r_j > 0 (or, below 0, the
 *              first); -1 when the row has no positive entry.
 * 0 <= L <= 64, 1 <= V < 2^30; strides >= V, rows need only be aligned to an element.
 * draft_probs, draft_tokens and u_accept may be NULL when L is 0.
 * workspace    8-byte aligned.
 */
int lfm2sc_accept_drafts(int dtype, int V, int num_seqs, int L,
                         const void* target_probs, int64_t target_stride,
                         const void* draft_probs, int64_t draft_stride,
                         const int32_t* draft_tokens, const int32_t* num_drafts,
                         const float* u_accept, const float* u_sample,
                         int32_t* accept_len, int32_t* keep_len, int32_t* next_token,
                         void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LFM2SC_HYBRID_H */
