// api_hybrid.cpp -- the C entry points of include/lfm2sc_hybrid.h: argument
// checks on the host (all before the first HIP call) and dispatch.
#include <cmath>

#include "api_common.hpp"
#include "hybrid.hpp"
#include "kernels.hpp"
#include "lfm2sc_hybrid.h"

namespace {

using namespace lfm2sc;

constexpr int64_t kMaxRowStride = (int64_t)1 << 22;   // 64 rows of a tile stay within 32-bit byte offsets
constexpr int kMaxHeads = 1 << 14;
constexpr int kMaxV = 1 << 30;                        // a row's byte offsets are 32-bit
constexpr int64_t kMaxCachedRows = (int64_t)1 << 28;
constexpr int64_t kMaxKeys = (int64_t)1 << 30;        // a tile past a sequence's end still counts in an int

int check_heads(const char* fn, int dtype, int D, int Hq, int Hkv) {
    if (dtype != LFM2SC_BF16) return fail(LFM2SC_ERR_UNSUPPORTED, "%s: only LFM2SC_BF16 is supported", fn);
    if (D != 64 && D != 128) return fail(LFM2SC_ERR_UNSUPPORTED, "%s: D=%d is neither 64 nor 128", fn, D);
    if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq > kMaxHeads)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: num_heads=%d must be a positive multiple of num_kv_heads=%d, at most %d", fn,
                    Hq, Hkv, kMaxHeads);
    return LFM2SC_OK;
}

int check_scale(const char* fn, float scale) {
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: scale=%g is not finite and positive", fn, (double)scale);
    return LFM2SC_OK;
}

int check_rows(const char* fn, const char* name, int64_t stride, int64_t min) {
    TRY(check_stride(fn, name, stride, min));
    if (stride >= kMaxRowStride)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: %s=%lld is not below %lld", fn, name, (long long)stride,
                    (long long)kMaxRowStride);
    return LFM2SC_OK;
}

int check_tokens(const char* fn, int64_t total_T, int num_seqs) {
    if (num_seqs < 0) return fail(LFM2SC_ERR_BAD_SHAPE, "%s: num_seqs=%d is negative", fn, num_seqs);
    if (total_T < 0 || total_T >= kMaxKeys)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: total_T=%lld outside [0, 2^30)", fn, (long long)total_T);
    return LFM2SC_OK;
}

// row blocks of at least 32 rows, times the heads, in one launch
int check_grid(const char* fn, int64_t total_T, int num_seqs, int Hq) {
    if ((total_T / 32 + num_seqs) * 2 * Hq >= kMaxRows)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: too many tokens, sequences and heads for one launch", fn);
    return LFM2SC_OK;
}

int check_workspace(const char* fn, const void* ws, size_t bytes, size_t need, uintptr_t align) {
    if (need == 0) return LFM2SC_OK;
    if (ws == nullptr || bytes < need)
        return fail(LFM2SC_ERR_WORKSPACE, "%s: workspace %p of %zu bytes, %zu needed", fn, ws, bytes, need);
    if (!aligned(ws, align))
        return fail(LFM2SC_ERR_ALIGNMENT, "%s: workspace is not %u-byte aligned", fn, (unsigned)align);
    return LFM2SC_OK;
}

int check_cu(const char* fn, hipStream_t s, const int32_t* cu, int N, int64_t total_T) {
    if (!check_mode()) return LFM2SC_OK;
    hipError_t e;
    const int bad = check_device_preconditions(s, nullptr, N, 0, cu, total_T, nullptr, 0, &e);
    if (e != hipSuccess) return launched(fn, e);
    if (bad)
        return fail(LFM2SC_ERR_PRECONDITION, "%s: device data breaks a precondition: cu_seqlens not non-decreasing within "
                    "[0, total_T]", fn);
    return LFM2SC_OK;
}

int check_ranges(const char* fn, hipStream_t s, const RangeCheck* checks, const char* const* names, int count) {
    if (!check_mode()) return LFM2SC_OK;
    hipError_t e;
    const int bad = check_device_ranges(s, checks, count, &e);
    if (e != hipSuccess) return launched(fn, e);
    for (int k = 0; k < count; ++k)
        if (bad & (1 << k))
            return fail(LFM2SC_ERR_PRECONDITION, "%s: device data breaks a precondition: %s outside [%lld, %lld]", fn,
                        names[k], (long long)checks[k].lo, (long long)checks[k].hi);
    return LFM2SC_OK;
}

int submitted(const char* fn, hipError_t e) {
    if (e == hipErrorInvalidConfiguration)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: the sizes need 2^32 or more work-items in one launch", fn);
    return launched(fn, e);
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

size_t cached_bytes(int D, int Hq, int Hkv, int N, int L, int prefix_len, int max_keys) {
    const CachedPlan p = cached_plan(D, Hq, Hkv, N, L, prefix_len, max_keys);
    const size_t rows = (size_t)N * (size_t)L * (size_t)Hq * (size_t)(p.prefix_splits + p.suffix_splits);
    return round_up(rows * (size_t)D * 4) + round_up(rows * 8);
}

// rows and heads of the new tokens within the kernels' int counters (each factor is at most 2^31, so no product here
// passes 64 bits)
bool cached_rows_fit(int N, int L, int Hq) {
    const int64_t rows = (int64_t)N * L;
    return rows < kMaxCachedRows && rows * Hq < kMaxCachedRows;
}

int check_cached_sizes(const char* fn, int N, int L, int Hq, int prefix_len, int max_pages, int page_size) {
    if (N < 0 || L < 0) return fail(LFM2SC_ERR_BAD_SHAPE, "%s: num_seqs=%d or L=%d is negative", fn, N, L);
    if (!cached_rows_fit(N, L, Hq))
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: num_seqs * L * num_heads is 2^28 or more", fn);
    if (prefix_len < 0 || prefix_len >= kMaxKeys)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: prefix_len=%d outside [0, 2^30)", fn, prefix_len);
    if (page_size < 1 || (page_size & (page_size - 1)) != 0)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: page_size=%d is not a power of two", fn, page_size);
    if (max_pages < 0 || (int64_t)max_pages * page_size >= kMaxKeys)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: max_pages=%d of %d tokens outside [0, 2^30)", fn, max_pages, page_size);
    return LFM2SC_OK;
}

}  // namespace

extern "C" {

int lfm2sc_attn_prefill(int dtype, int D, int num_heads, int num_kv_heads, const void* q, int64_t q_stride, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, int64_t total_T, const int32_t* cu_seqlens,
                        int num_seqs, float scale, void* out, int64_t out_stride, float* lse, void* stream) {
    const char* fn = "lfm2sc_attn_prefill";
    TRY(check_heads(fn, dtype, D, num_heads, num_kv_heads));
    TRY(check_scale(fn, scale));
    TRY(check_tokens(fn, total_T, num_seqs));
    TRY(check_rows(fn, "q_stride", q_stride, (int64_t)num_heads * D));
    TRY(check_rows(fn, "k_stride", k_stride, (int64_t)num_kv_heads * D));
    TRY(check_rows(fn, "v_stride", v_stride, (int64_t)num_kv_heads * D));
    TRY(check_rows(fn, "out_stride", out_stride, (int64_t)num_heads * D));
    TRY(check_grid(fn, total_T, num_seqs, num_heads));
    if (num_seqs == 0 || total_T == 0) return ok();
    TRY(check_ptr(fn, "q", q, 16));
    TRY(check_ptr(fn, "k", k, 16));
    TRY(check_ptr(fn, "v", v, 16));
    TRY(check_ptr(fn, "cu_seqlens", cu_seqlens, 4));
    TRY(check_ptr(fn, "out", out, 16));
    if (lse != nullptr) TRY(check_ptr(fn, "lse", lse, 4));
    hipStream_t s = static_cast<hipStream_t>(stream);
    TRY(check_cu(fn, s, cu_seqlens, num_seqs, total_T));
    AttnArgs a;
    a.q = static_cast<const uint16_t*>(q); a.q_stride = q_stride;
    a.k = static_cast<const uint16_t*>(k); a.k_stride = k_stride;
    a.v = static_cast<const uint16_t*>(v); a.v_stride = v_stride;
    a.total_T = total_T; a.cu = cu_seqlens; a.N = num_seqs;
    a.Hq = num_heads; a.Hkv = num_kv_heads; a.scale = scale;
    a.out = static_cast<uint16_t*>(out); a.out_stride = out_stride; a.lse = lse;
    return submitted(fn, launch_attn_prefill(a, D, s));
}

size_t lfm2sc_attn_backward_workspace_bytes(int dtype, int D, int num_heads, int num_kv_heads, int64_t total_T,
                                            int num_seqs) {
    if (dtype != LFM2SC_BF16 || (D != 64 && D != 128) || num_kv_heads < 1 || num_heads < num_kv_heads ||
        num_heads % num_kv_heads != 0 || num_heads > kMaxHeads || total_T <= 0 || total_T >= kMaxKeys || num_seqs <= 0)
        return 0;
    const size_t rows = 2 * round_up((size_t)num_heads * (size_t)total_T * 4);
    const int splits = attn_backward_splits(num_heads, num_kv_heads, total_T, num_seqs);
    return rows + (splits > 1 ? (size_t)splits * 2 * (size_t)total_T * (size_t)num_kv_heads * (size_t)D * 4 : 0);
}

int lfm2sc_attn_backward(int dtype, int D, int num_heads, int num_kv_heads, const void* q, int64_t q_stride, const void* k,
                         int64_t k_stride, const void* v, int64_t v_stride, int64_t total_T, const int32_t* cu_seqlens,
                         int num_seqs, float scale, const void* out, int64_t out_stride, const float* lse,
                         const void* d_out, int64_t d_out_stride, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride,
                         void* dv, int64_t dv_stride, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "lfm2sc_attn_backward";
    TRY(check_heads(fn, dtype, D, num_heads, num_kv_heads));
    TRY(check_scale(fn, scale));
    TRY(check_tokens(fn, total_T, num_seqs));
    const int64_t wq = (int64_t)num_heads * D, wk = (int64_t)num_kv_heads * D;
    TRY(check_rows(fn, "q_stride", q_stride, wq));
    TRY(check_rows(fn, "k_stride", k_stride, wk));
    TRY(check_rows(fn, "v_stride", v_stride, wk));
    TRY(check_rows(fn, "out_stride", out_stride, wq));
    TRY(check_rows(fn, "d_out_stride", d_out_stride, wq));
    TRY(check_rows(fn, "dq_stride", dq_stride, wq));
    TRY(check_rows(fn, "dk_stride", dk_stride, wk));
    TRY(check_rows(fn, "dv_stride", dv_stride, wk));
    TRY(check_grid(fn, total_T, num_seqs, num_heads));
    if (num_seqs == 0 || total_T == 0) return ok();
    TRY(check_ptr(fn, "q", q, 16));
    TRY(check_ptr(fn, "k", k, 16));
    TRY(check_ptr(fn, "v", v, 16));
    TRY(check_ptr(fn, "cu_seqlens", cu_seqlens, 4));
    TRY(check_ptr(fn, "out", out, 16));
    TRY(check_ptr(fn, "lse", lse, 4));
    TRY(check_ptr(fn, "d_out", d_out, 16));
    TRY(check_ptr(fn, "dq", dq, 16));
    TRY(check_ptr(fn, "dk", dk, 16));
    TRY(check_ptr(fn, "dv", dv, 16));
    const size_t need = lfm2sc_attn_backward_workspace_bytes(dtype, D, num_heads, num_kv_heads, total_T, num_seqs);
    TRY(check_workspace(fn, workspace, workspace_bytes, need, 16));
    hipStream_t s = static_cast<hipStream_t>(stream);
    TRY(check_cu(fn, s, cu_seqlens, num_seqs, total_T));
    AttnGradArgs a;
    a.f.q = static_cast<const uint16_t*>(q); a.f.q_stride = q_stride;
    a.f.k = static_cast<const uint16_t*>(k); a.f.k_stride = k_stride;
    a.f.v = static_cast<const uint16_t*>(v); a.f.v_stride = v_stride;
    a.f.total_T = total_T; a.f.cu = cu_seqlens; a.f.N = num_seqs;
    a.f.Hq = num_heads; a.f.Hkv = num_kv_heads; a.f.scale = scale;
    a.f.out = static_cast<uint16_t*>(const_cast<void*>(out)); a.f.out_stride = out_stride;
    a.f.lse = const_cast<float*>(lse);
    a.dout = static_cast<const uint16_t*>(d_out); a.dout_stride = d_out_stride;
    a.dq = static_cast<uint16_t*>(dq); a.dq_stride = dq_stride;
    a.dk = static_cast<uint16_t*>(dk); a.dk_stride = dk_stride;
    a.dv = static_cast<uint16_t*>(dv); a.dv_stride = dv_stride;
    a.delta = static_cast<float*>(workspace);
    const size_t rows = round_up((size_t)num_heads * (size_t)total_T * 4);
    a.lse2 = reinterpret_cast<float*>(static_cast<char*>(workspace) + rows);
    a.splits = attn_backward_splits(num_heads, num_kv_heads, total_T, num_seqs);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + 2 * rows);
    return submitted(fn, launch_attn_backward(a, D, s));
}

size_t lfm2sc_attn_cached_workspace_bytes(int dtype, int D, int num_heads, int num_kv_heads, int num_seqs, int L,
                                          int prefix_len, int max_pages, int page_size) {
    if (dtype != LFM2SC_BF16 || (D != 64 && D != 128) || num_kv_heads < 1 || num_heads < num_kv_heads ||
        num_heads % num_kv_heads != 0 || num_heads > kMaxHeads || num_seqs <= 0 || L <= 0 ||
        !cached_rows_fit(num_seqs, L, num_heads) || prefix_len < 0 || prefix_len >= kMaxKeys ||
        page_size < 1 || (page_size & (page_size - 1)) != 0 || max_pages < 0 || (int64_t)max_pages * page_size >= kMaxKeys)
        return 0;
    return cached_bytes(D, num_heads, num_kv_heads, num_seqs, L, prefix_len, max_pages * page_size);
}

int lfm2sc_attn_cached(int dtype, int D, int num_heads, int num_kv_heads, const void* q, int64_t q_stride, int num_seqs,
                       int L, const void* k_pages, const void* v_pages, int64_t kv_stride, int num_pages, int page_size,
                       const int32_t* prefix_pages, int prefix_len, const int32_t* page_table, int max_pages,
                       const int32_t* suffix_len, float scale, void* out, int64_t out_stride, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const char* fn = "lfm2sc_attn_cached";
    TRY(check_heads(fn, dtype, D, num_heads, num_kv_heads));
    TRY(check_scale(fn, scale));
    TRY(check_cached_sizes(fn, num_seqs, L, num_heads, prefix_len, max_pages, page_size));
    TRY(check_rows(fn, "q_stride", q_stride, (int64_t)num_heads * D));
    TRY(check_rows(fn, "kv_stride", kv_stride, (int64_t)num_kv_heads * D));
    TRY(check_rows(fn, "out_stride", out_stride, (int64_t)num_heads * D));
    if (num_seqs == 0 || L == 0) return ok();
    if ((prefix_len > 0 || max_pages > 0) && (num_pages < 1 || (int64_t)num_pages * page_size >= kMaxRows))
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: num_pages=%d of %d tokens outside [1, 2^31)", fn, num_pages, page_size);
    TRY(check_ptr(fn, "q", q, 16));
    if (prefix_len > 0 || max_pages > 0) {
        TRY(check_ptr(fn, "k_pages", k_pages, 16));
        TRY(check_ptr(fn, "v_pages", v_pages, 16));
    }
    if (prefix_len > 0) TRY(check_ptr(fn, "prefix_pages", prefix_pages, 4));
    if (max_pages > 0) TRY(check_ptr(fn, "page_table", page_table, 4));
    TRY(check_ptr(fn, "suffix_len", suffix_len, 4));
    TRY(check_ptr(fn, "out", out, 16));
    const size_t need = cached_bytes(D, num_heads, num_kv_heads, num_seqs, L, prefix_len, max_pages * page_size);
    TRY(check_workspace(fn, workspace, workspace_bytes, need, 16));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const RangeCheck ranges[] = {
        {prefix_pages, prefix_len > 0 ? ((int64_t)prefix_len + page_size - 1) / page_size : 0, 0, (int64_t)num_pages - 1},
        {page_table, (int64_t)num_seqs * max_pages, 0, (int64_t)num_pages - 1, suffix_len, max_pages, page_size},
        {suffix_len, num_seqs, 0, (int64_t)max_pages * page_size}};
    const char* const names[] = {"a prefix page", "a page of page_table", "a suffix length"};
    TRY(check_ranges(fn, s, ranges, names, 3));
    CachedArgs a;
    a.q = static_cast<const uint16_t*>(q); a.q_stride = q_stride; a.N = num_seqs; a.L = L;
    a.Hq = num_heads; a.Hkv = num_kv_heads;
    a.k = static_cast<const uint16_t*>(k_pages); a.v = static_cast<const uint16_t*>(v_pages); a.kv_stride = kv_stride;
    a.num_pages = num_pages; a.page_shift = __builtin_ctz((unsigned)page_size);
    a.prefix_pages = prefix_pages; a.prefix_len = prefix_len;
    a.page_table = page_table; a.max_pages = max_pages; a.suffix_len = suffix_len;
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out); a.out_stride = out_stride;
    const CachedPlan p = cached_plan(D, num_heads, num_kv_heads, num_seqs, L, prefix_len, max_pages * page_size);
    const size_t rows = (size_t)num_seqs * (size_t)L * (size_t)num_heads * (size_t)(p.prefix_splits + p.suffix_splits);
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + round_up(rows * (size_t)D * 4));
    a.prefix_splits = a.prefix_chunk = a.suffix_splits = 0;
    a.prefix_blocks = 0;
    return submitted(fn, launch_attn_cached(a, D, s));
}

size_t lfm2sc_accept_drafts_workspace_bytes(int num_seqs, int L, int V) {
    if (num_seqs <= 0 || L < 0 || L > 64 || V < 1 || V >= kMaxV) return 0;
    return round_up((size_t)num_seqs * 2 * (size_t)draft_chunks(V) * 8);
}

int lfm2sc_accept_drafts(int dtype, int V, int num_seqs, int L, const void* target_probs, int64_t target_stride,
                         const void* draft_probs, int64_t draft_stride, const int32_t* draft_tokens,
                         const int32_t* num_drafts, const float* u_accept, const float* u_sample, int32_t* accept_len,
                         int32_t* keep_len, int32_t* next_token, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "lfm2sc_accept_drafts";
    if (dtype != LFM2SC_BF16 && dtype != LFM2SC_F32)
        return fail(LFM2SC_ERR_UNSUPPORTED, "%s: dtype %d is neither LFM2SC_BF16 (0) nor LFM2SC_F32 (1)", fn, dtype);
    if (V < 1 || V >= kMaxV) return fail(LFM2SC_ERR_BAD_SHAPE, "%s: V=%d outside [1, 2^30)", fn, V);
    if (L < 0 || L > 64) return fail(LFM2SC_ERR_BAD_SHAPE, "%s: L=%d outside [0, 64]", fn, L);
    if (num_seqs < 0) return fail(LFM2SC_ERR_BAD_SHAPE, "%s: num_seqs=%d is negative", fn, num_seqs);
    if ((int64_t)num_seqs * draft_chunks(V) >= kMaxRows)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: too many sequences of V=%d for one launch", fn, V);
    if (target_stride < V)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: target_stride=%lld is below V=%d", fn, (long long)target_stride, V);
    const bool rows = L > 0 && draft_probs != nullptr;
    if (rows && draft_stride < V)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: draft_stride=%lld is below V=%d", fn, (long long)draft_stride, V);
    if (num_seqs == 0) return ok();
    const uintptr_t e = dtype == LFM2SC_BF16 ? 2 : 4;
    TRY(check_ptr(fn, "target_probs", target_probs, e));
    if (rows) TRY(check_ptr(fn, "draft_probs", draft_probs, e));
    if (L > 0) {
        TRY(check_ptr(fn, "draft_tokens", draft_tokens, 4));
        TRY(check_ptr(fn, "u_accept", u_accept, 4));
    }
    if (num_drafts != nullptr) TRY(check_ptr(fn, "num_drafts", num_drafts, 4));
    TRY(check_ptr(fn, "u_sample", u_sample, 4));
    TRY(check_ptr(fn, "accept_len", accept_len, 4));
    if (keep_len != nullptr) TRY(check_ptr(fn, "keep_len", keep_len, 4));
    TRY(check_ptr(fn, "next_token", next_token, 4));
    TRY(check_workspace(fn, workspace, workspace_bytes, lfm2sc_accept_drafts_workspace_bytes(num_seqs, L, V), 8));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const RangeCheck ranges[] = {{L > 0 ? draft_tokens : nullptr, (int64_t)num_seqs * L, 0, (int64_t)V - 1, num_drafts, L},
                                 {num_drafts, num_seqs, 0, L}};
    const char* const names[] = {"a draft token", "a number of drafts"};
    TRY(check_ranges(fn, s, ranges, names, 2));
    auto fill = [&](auto& a) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(a.target)>>;
        a.target = static_cast<const E*>(target_probs); a.target_stride = target_stride;
        a.draft = rows ? static_cast<const E*>(draft_probs) : nullptr; a.draft_stride = draft_stride;
        a.V = V; a.N = num_seqs; a.L = L;
        a.tokens = draft_tokens; a.num_drafts = num_drafts;
        a.u_accept = u_accept; a.u_sample = u_sample;
        a.accept_len = accept_len; a.keep_len = keep_len; a.next_token = next_token;
        a.sums = static_cast<double*>(workspace);
        return submitted(fn, launch_drafts(a, s));
    };
    if (dtype == LFM2SC_BF16) {
        DraftArgs<uint16_t> a;
        return fill(a);
    }
    DraftArgs<float> a;
    return fill(a);
}

}  // extern "C"
