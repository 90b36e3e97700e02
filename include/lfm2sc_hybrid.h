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
 *        accept_len that lfm2sc_commit_window takes;
 *   lfm2sc_rotary         rotary positions of q and k rows, and the gradient, with
 *        lfm2sc_rotary_freqs for the frequencies;
 *   lfm2sc_cache8_write / lfm2sc_cache8_read   k and v rows quantised into a paged
 *        cache of 8-bit codes, and read back;
 *   lfm2sc_attn_cached8   lfm2sc_attn_cached over that cache.
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
 * It goes by the call's own splits, so fewer sequences or pages may need more: ask for
 * each of the sizes that a program uses.
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

/* ------------------------------------------------------------------------
 * Rotary positions: the rotation of the published method, for the attention layers
 * and for draft models, which pair channels either way.
 */

/* Frequencies for longer contexts than the model was trained on. */
enum {
    LFM2SC_ROPE_PLAIN = 0,    /* f_i = base^(-2i / R) */
    LFM2SC_ROPE_LINEAR = 1,   /* f_i / factor */
    LFM2SC_ROPE_BASE = 2,     /* base grows by factor^(R / (R - 2)); R >= 4 */
    LFM2SC_ROPE_PARTS = 3     /* by the turns r_i = original_len f_i / 2 pi that a pair makes over the trained length:
                                 w = clamp((r_i - low) / (high - low), 0, 1), f_i (w + (1 - w) / factor) */
};

/*
 * Fills freqs, HOST memory [R / 2], with the frequencies of R = rotary_dim rotated
 * columns, worked out in fp64 and rounded once.  base > 1; factor >= 1 (not for
 * PLAIN); original_len > 0 and 0 <= low < high for PARTS (usual: 1 and 4, or 1 and
 * 32 with a `magnitude` of 0.1 ln factor + 1).  What a scaling does not use may be 0.
 */
int lfm2sc_rotary_freqs(int rotary_dim, double base, int scaling, double factor, double original_len, double low,
                        double high, float* freqs);

/*
 * Rotates the first rotary_dim = R columns of every head of q and k; the others
 * stay.  With angle a = position * freqs[i], a pair (x, y) of a head's columns
 * becomes
 *   magnitude * (x cos a - y sin a, y cos a + x sin a);   inverse != 0: sin a -> -sin a,
 * the gradient of the call with respect to its rows.  Pairs are columns i and
 * i + R / 2 (interleaved 0), or 2 i and 2 i + 1 (interleaved 1).
 *
 * dtype        LFM2SC_BF16 or LFM2SC_F32, of the rows.  Angles are reduced in fp64
 *              (below 2^24 positions exact to 1e-8 of a turn, up to 2^31 to 1e-6),
 *              the rotation is fp32, a result is rounded once.
 * D            a multiple of 8 up to 512; R even, 2 <= R <= D.
 * q            [total_T][q_stride], num_heads heads of D columns; q_out the same.
 *              q_out may be q (with the same stride); otherwise the two do not
 *              overlap.  Strides as for attention: multiples of 8, below 2^22;
 *              pointers 16-byte aligned.
 * k, k_out     the same with num_kv_heads heads; with num_kv_heads 0 they are not
 *              used.
 * positions    int32.  cu_seqlens NULL: [total_T], the rows' positions.  Otherwise
 *              rows are packed sequences (offsets as for lfm2sc_prefill_ragged,
 *              clamped to [0, total_T]), row t of sequence i has position
 *              positions[i] + t - cu[i]; positions is [num_seqs], or NULL for 0.
 *              Rows of no sequence are not written.
 * freqs        [R / 2] fp32, device memory.
 */
int lfm2sc_rotary(int dtype, int D, int rotary_dim, int interleaved, int inverse,
                  const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int num_heads,
                  const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int num_kv_heads,
                  int64_t total_T, const int32_t* positions, const int32_t* cu_seqlens, int num_seqs,
                  const float* freqs, float magnitude, void* stream);

/* ------------------------------------------------------------------------
 * The cache of 8-bit codes.
 *
 * Page p of the pools (uint8 codes, page_stride bytes apart, 16-byte aligned, a
 * multiple of 16, at least num_kv_heads * page_size * D) holds page_size tokens,
 * page_size a power of two of at least 16:
 *   k_pages   [num_kv_heads][page_size][D]
 *   v_pages   [num_kv_heads][page_size / 16][D][16]: 16 tokens of a channel are neighbours
 * and its scales (fp32, scale_stride elements apart, at least num_kv_heads *
 * page_size / scale_tokens)
 *   k_scales, v_scales [num_kv_heads][page_size / scale_tokens]
 * with scale_tokens 1, or a power of two of 16 to 128 up to page_size.  A value is
 * its code times the scale of its head's block of scale_tokens tokens.
 *
 * Codes: LFM2SC_CACHE_E4M3 (1.4.3 floats, largest 448) or LFM2SC_CACHE_INT8 (-127 to
 * 127).  D is 64 or 128.  num_pages * page_size < 2^31.
 */
enum { LFM2SC_CACHE_E4M3 = 0, LFM2SC_CACHE_INT8 = 1 };

/*
 * Writes k and v rows (dtype LFM2SC_BF16 or LFM2SC_F32) as the newest tokens of their
 * sequences.
 *
 * k, v         [total_T][*_stride], num_kv_heads heads of D columns; strides as for
 *              attention.  Packed sequences by cu_seqlens; or, with cu_seqlens NULL,
 *              total_T / num_seqs rows of every sequence (the rows of a decode step or
 *              a verify block; total_T is a multiple of num_seqs).
 * seq_len      [num_seqs] int32: tokens of the sequence after the call, clamped to
 *              [0, max_pages * page_size]: its n rows are tokens seq_len - n to
 *              seq_len - 1 (a row that would come before token 0 is left out).
 * page_table   [num_seqs][max_pages] int32.  Nothing is written to a page whose number
 *              is outside [0, num_pages).  No two sequences of a call may write to one
 *              page.
 * A block's scale, from the magnitudes of the rows alone that join it (infinities and
 * NaN apart): where the block holds no earlier token, for INT8 the largest magnitude /
 * 127 and for E4M3 the lowest power of two s with magnitudes <= 448 s (both at least
 * 2^-100; 0 if all are 0); where it does (tokens before seq_len - n), the old scale
 * times the lowest power of two >= 1 that holds the rows (codes up to 127.5 before
 * rounding, or 448), and the earlier codes are rounded again in steps of the new one,
 * so that a value stays within one step, however many rows follow.  (An old scale of
 * 0, below 2^-100 or not finite, or 2^40 times too small, makes a new one and zeros of
 * the earlier codes; an E4M3 NaN among them stays NaN.)
 * A code is x * (1 / s) rounded to nearest even, 0 where s is 0; beyond the largest it
 * is the largest (infinities too), a NaN, or an infinity where s is 0, is NaN (E4M3) or
 * 0 (INT8).
 * Taking rows back (a smaller seq_len in the next call, as after rejected drafts) does
 * not undo what they did to a block that keeps earlier tokens: its scale stays as they
 * made it, and the earlier codes as rounded to it.  Later values of the block then
 * depend on the rows taken back; the bound of one step holds, a step being that scale's.
 * In the blocks that the call touches, codes of tokens from seq_len on are not values
 * of anything; they keep their bits, and tell nothing under a new scale.
 */
int lfm2sc_cache8_write(int dtype, int format, int D, int num_kv_heads,
                        const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t total_T,
                        const int32_t* cu_seqlens, int num_seqs,
                        void* k_pages, void* v_pages, int64_t page_stride,
                        float* k_scales, float* v_scales, int64_t scale_stride,
                        int num_pages, int page_size, int scale_tokens,
                        const int32_t* page_table, int max_pages, const int32_t* seq_len, void* stream);

/*
 * The other way round: row t of sequence i receives the value of token seq_len[i] - n
 * + t, rounded to dtype; a row before token 0 is not written.  Page numbers outside the
 * pool read as the nearest page.  k_out and v_out [total_T][*_stride].
 */
int lfm2sc_cache8_read(int dtype, int format, int D, int num_kv_heads,
                       const void* k_pages, const void* v_pages, int64_t page_stride,
                       const float* k_scales, const float* v_scales, int64_t scale_stride,
                       int num_pages, int page_size, int scale_tokens,
                       const int32_t* page_table, int max_pages, const int32_t* seq_len,
                       void* k_out, int64_t k_stride, void* v_out, int64_t v_stride, int64_t total_T,
                       const int32_t* cu_seqlens, int num_seqs, void* stream);

/*
 * Bytes of workspace lfm2sc_attn_cached8 needs; 0 for invalid sizes, when num_seqs or L
 * is 0, and where no call up to these sizes needs any (few keys).  Never less for a
 * larger num_seqs, L, prefix_len or max_suffix_len: a workspace taken for the largest
 * of a program's calls serves all of them (same D and heads).  A call that joins
 * nothing takes a NULL workspace too.
 */
size_t lfm2sc_attn_cached8_workspace_bytes(int dtype, int D, int num_heads, int num_kv_heads, int num_seqs, int L,
                                           int prefix_len, int max_suffix_len);

/*
 * lfm2sc_attn_cached over the cache of 8-bit codes: same queries (LFM2SC_BF16), prefix,
 * page table, lengths, output and workspace rules.  Scores are scale * k_scale * (q .
 * code); the probability times the value's scale is rounded to bf16 as an operand of
 * the second product; everything else is fp32.
 *
 * max_suffix_len  a bound of the caller's on suffix_len, at most max_pages * page_size
 *              (suffix_len is clamped to it): the work is split by it, so one near the
 *              longest sequence serves a wide page table best.
 * Codes and scales of tokens from a sequence's length on may hold anything.  A NaN code
 * or an infinite or NaN scale of a token reaches the rows that see it and may reach the
 * other rows of its sequence's L.
 */
int lfm2sc_attn_cached8(int dtype, int format, int D, int num_heads, int num_kv_heads,
                        const void* q, int64_t q_stride, int num_seqs, int L,
                        const void* k_pages, const void* v_pages, int64_t page_stride,
                        const float* k_scales, const float* v_scales, int64_t scale_stride,
                        int num_pages, int page_size, int scale_tokens,
                        const int32_t* prefix_pages, int prefix_len,
                        const int32_t* page_table, int max_pages, const int32_t* suffix_len, int max_suffix_len,
                        float scale, void* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                        void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LFM2SC_HYBRID_H */
