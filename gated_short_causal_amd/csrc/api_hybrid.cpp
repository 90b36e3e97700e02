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
constexpr int64_t kMaxPoolStride = (int64_t)1 << 31;
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

// Never less for larger sizes.
size_t cached8_bytes(int D, int Hq, int Hkv, int N, int L, int prefix_len, int max_suffix) {
    const size_t rows = (size_t)cached8_part_rows(D, Hq, Hkv, N, L, prefix_len, max_suffix);
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

constexpr int64_t kMaxPageBytes = (int64_t)1 << 30;   // offsets within a page are 32-bit

// A pool of 8-bit codes: format, head dimension, page geometry.
int check_pool8(const char* fn, int format, int D, int Hkv, int64_t page_stride, int64_t scale_stride, int page_size,
                int scale_tokens, int max_pages) {
    if (format != LFM2SC_CACHE_E4M3 && format != LFM2SC_CACHE_INT8)
        return fail(LFM2SC_ERR_UNSUPPORTED, "%s: format %d is neither LFM2SC_CACHE_E4M3 (0) nor LFM2SC_CACHE_INT8 (1)", fn,
                    format);
    if (D != 64 && D != 128) return fail(LFM2SC_ERR_UNSUPPORTED, "%s: D=%d is neither 64 nor 128", fn, D);
    if (Hkv < 1 || Hkv > kMaxHeads)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: num_kv_heads=%d outside [1, %d]", fn, Hkv, kMaxHeads);
    if (page_size < 16 || (page_size & (page_size - 1)) != 0)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: page_size=%d is not a power of two of at least 16", fn, page_size);
    if (scale_tokens != 1 && (scale_tokens < 16 || scale_tokens > 128 || (scale_tokens & (scale_tokens - 1)) != 0 ||
                              scale_tokens > page_size))
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: scale_tokens=%d is neither 1 nor a power of two in [16, 128] up to page_size=%d",
                    fn, scale_tokens, page_size);
    const int64_t page = (int64_t)Hkv * page_size * D, scales = (int64_t)Hkv * (page_size / scale_tokens);
    if (page >= kMaxPageBytes)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: a page of num_kv_heads * page_size * D is 2^30 bytes or more", fn);
    if (page_stride < page)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: page_stride=%lld is below a page's %lld bytes", fn, (long long)page_stride,
                    (long long)page);
    if (page_stride % 16 != 0)
        return fail(LFM2SC_ERR_ALIGNMENT, "%s: page_stride=%lld is not a multiple of 16 bytes", fn, (long long)page_stride);
    if (scale_stride < scales)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: scale_stride=%lld is below a page's %lld scales", fn, (long long)scale_stride,
                    (long long)scales);
    if (page_stride >= kMaxPoolStride || scale_stride >= kMaxPoolStride)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: page_stride or scale_stride is 2^31 or more", fn);
    if (max_pages < 0 || (int64_t)max_pages * page_size >= kMaxKeys)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: max_pages=%d of %d tokens outside [0, 2^30)", fn, max_pages, page_size);
    return LFM2SC_OK;
}

int check_pool8_pages(const char* fn, const void* k_pages, const void* v_pages, const float* k_scales, const float* v_scales,
                      int num_pages, int page_size) {
    if (num_pages < 1 || (int64_t)num_pages * page_size >= kMaxRows)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: num_pages=%d of %d tokens outside [1, 2^31)", fn, num_pages, page_size);
    TRY(check_ptr(fn, "k_pages", k_pages, 16));
    TRY(check_ptr(fn, "v_pages", v_pages, 16));
    TRY(check_ptr(fn, "k_scales", k_scales, 4));
    return check_ptr(fn, "v_scales", v_scales, 4);
}

// lfm2sc_cache8_write and lfm2sc_cache8_read differ in what they launch.
int cache8(const char* fn, bool write, int dtype, int format, int D, int Hkv, void* k, int64_t k_stride, void* v,
           int64_t v_stride, int64_t total_T, const int32_t* cu, int N, void* k_pages, void* v_pages, int64_t page_stride,
           float* k_scales, float* v_scales, int64_t scale_stride, int num_pages, int page_size, int scale_tokens,
           const int32_t* page_table, int max_pages, const int32_t* seq_len, void* stream) {
    if (dtype != LFM2SC_BF16 && dtype != LFM2SC_F32)
        return fail(LFM2SC_ERR_UNSUPPORTED, "%s: dtype %d is neither LFM2SC_BF16 (0) nor LFM2SC_F32 (1)", fn, dtype);
    TRY(check_pool8(fn, format, D, Hkv, page_stride, scale_stride, page_size, scale_tokens, max_pages));
    TRY(check_tokens(fn, total_T, N));
    TRY(check_rows(fn, "k_stride", k_stride, (int64_t)Hkv * D));
    TRY(check_rows(fn, "v_stride", v_stride, (int64_t)Hkv * D));
    if (cu == nullptr && (N == 0 ? total_T != 0 : total_T % N != 0))
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: total_T=%lld is not a multiple of num_seqs=%d, and cu_seqlens is NULL", fn,
                    (long long)total_T, N);
    if (N == 0 || total_T == 0 || max_pages == 0) return ok();
    TRY(check_ptr(fn, write ? "k" : "k_out", k, 16));
    TRY(check_ptr(fn, write ? "v" : "v_out", v, 16));
    if (cu != nullptr) TRY(check_ptr(fn, "cu_seqlens", cu, 4));
    TRY(check_pool8_pages(fn, k_pages, v_pages, k_scales, v_scales, num_pages, page_size));
    TRY(check_ptr(fn, "page_table", page_table, 4));
    TRY(check_ptr(fn, "seq_len", seq_len, 4));
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (cu != nullptr) TRY(check_cu(fn, s, cu, N, total_T));
    const RangeCheck ranges[] = {
        {page_table, (int64_t)N * max_pages, 0, (int64_t)num_pages - 1, seq_len, max_pages, page_size},
        {seq_len, N, 0, (int64_t)max_pages * page_size}};
    const char* const names[] = {"a page of page_table", "a sequence length"};
    TRY(check_ranges(fn, s, ranges, names, 2));
    Cache8Args a;
    a.rows.T = total_T; a.rows.N = N; a.rows.L = cu == nullptr ? (int)(total_T / N) : 0; a.rows.cu = cu;
    a.rows.page_table = page_table; a.rows.max_pages = max_pages; a.rows.seq_len = seq_len;
    a.rows.page_shift = __builtin_ctz((unsigned)page_size);
    a.Hkv = Hkv;
    a.k_rows = k; a.k_row_stride = k_stride; a.v_rows = v; a.v_row_stride = v_stride;
    a.k_pages = static_cast<uint8_t*>(k_pages); a.v_pages = static_cast<uint8_t*>(v_pages); a.page_stride = page_stride;
    a.k_scales = k_scales; a.v_scales = v_scales; a.scale_stride = scale_stride;
    a.num_pages = num_pages; a.block_shift = __builtin_ctz((unsigned)scale_tokens);
    a.units = 0;
    return submitted(fn, launch_cache8(a, D, format == LFM2SC_CACHE_INT8, dtype == LFM2SC_F32, write, s));
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

int lfm2sc_rotary_freqs(int rotary_dim, double base, int scaling, double factor, double original_len, double low,
                        double high, float* freqs) {
    const char* fn = "lfm2sc_rotary_freqs";
    const int R = rotary_dim;
    if (R < 2 || R > kRotaryMaxD || R % 2 != 0)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: rotary_dim=%d is not an even number in [2, %d]", fn, R, kRotaryMaxD);
    if (scaling < LFM2SC_ROPE_PLAIN || scaling > LFM2SC_ROPE_PARTS)
        return fail(LFM2SC_ERR_UNSUPPORTED, "%s: scaling %d is not one of LFM2SC_ROPE_*", fn, scaling);
    if (!(base > 1.) || !std::isfinite(base))
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: base=%g is not finite and above 1", fn, base);
    if (scaling != LFM2SC_ROPE_PLAIN && (!(factor >= 1.) || !std::isfinite(factor)))
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: factor=%g is not finite and at least 1", fn, factor);
    if (scaling == LFM2SC_ROPE_BASE && R < 4)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: LFM2SC_ROPE_BASE needs rotary_dim of at least 4", fn);
    if (scaling == LFM2SC_ROPE_PARTS && (!(original_len > 0.) || !std::isfinite(original_len) || !(low >= 0.) || !(high > low) ||
                                         !std::isfinite(high)))
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: original_len=%g is not positive, or not 0 <= low=%g < high=%g", fn, original_len,
                    low, high);
    TRY(check_ptr(fn, "freqs", freqs, 4));
    const double b = scaling == LFM2SC_ROPE_BASE ? base * std::pow(factor, (double)R / (R - 2)) : base;
    for (int i = 0; i < R / 2; ++i) {
        double f = std::pow(b, -2. * i / R);
        if (scaling == LFM2SC_ROPE_LINEAR) f /= factor;
        if (scaling == LFM2SC_ROPE_PARTS) {
            const double turns = original_len * f / 6.283185307179586476925, w = (turns - low) / (high - low);
            const double keep = w < 0. ? 0. : w > 1. ? 1. : w;
            f *= keep + (1. - keep) / factor;
        }
        freqs[i] = (float)f;
    }
    return ok();
}

int lfm2sc_rotary(int dtype, int D, int rotary_dim, int interleaved, int inverse, const void* q, int64_t q_stride, void* q_out,
                  int64_t q_out_stride, int num_heads, const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride,
                  int num_kv_heads, int64_t total_T, const int32_t* positions, const int32_t* cu_seqlens, int num_seqs,
                  const float* freqs, float magnitude, void* stream) {
    const char* fn = "lfm2sc_rotary";
    if (dtype != LFM2SC_BF16 && dtype != LFM2SC_F32)
        return fail(LFM2SC_ERR_UNSUPPORTED, "%s: dtype %d is neither LFM2SC_BF16 (0) nor LFM2SC_F32 (1)", fn, dtype);
    if (D < 8 || D > kRotaryMaxD || D % 8 != 0)
        return fail(LFM2SC_ERR_UNSUPPORTED, "%s: D=%d is not a multiple of 8 in [8, %d]", fn, D, kRotaryMaxD);
    if (rotary_dim < 2 || rotary_dim > D || rotary_dim % 2 != 0)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: rotary_dim=%d is not an even number in [2, D=%d]", fn, rotary_dim, D);
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
        return fail(LFM2SC_ERR_UNSUPPORTED, "%s: interleaved=%d and inverse=%d are 0 or 1", fn, interleaved, inverse);
    if (num_heads < 1 || num_heads > kMaxHeads || num_kv_heads < 0 || num_kv_heads > kMaxHeads)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: num_heads=%d outside [1, %d], or num_kv_heads=%d outside [0, %d]", fn, num_heads,
                    kMaxHeads, num_kv_heads, kMaxHeads);
    if (!std::isfinite(magnitude))
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: magnitude=%g is not finite", fn, (double)magnitude);
    TRY(check_tokens(fn, total_T, num_seqs));
    TRY(check_rows(fn, "q_stride", q_stride, (int64_t)num_heads * D));
    TRY(check_rows(fn, "q_out_stride", q_out_stride, (int64_t)num_heads * D));
    const bool both = num_kv_heads > 0;
    if (both) {
        TRY(check_rows(fn, "k_stride", k_stride, (int64_t)num_kv_heads * D));
        TRY(check_rows(fn, "k_out_stride", k_out_stride, (int64_t)num_kv_heads * D));
    }
    if (total_T == 0 || (cu_seqlens != nullptr && num_seqs == 0)) return ok();
    TRY(check_ptr(fn, "q", q, 16));
    TRY(check_ptr(fn, "q_out", q_out, 16));
    if (both) {
        TRY(check_ptr(fn, "k", k, 16));
        TRY(check_ptr(fn, "k_out", k_out, 16));
    }
    if (q_out == q && q_out_stride != q_stride)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: q_out is q, with another stride", fn);
    if (both && k_out == k && k_out_stride != k_stride)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: k_out is k, with another stride", fn);
    if (cu_seqlens != nullptr) TRY(check_ptr(fn, "cu_seqlens", cu_seqlens, 4));
    if (cu_seqlens == nullptr || positions != nullptr) TRY(check_ptr(fn, "positions", positions, 4));
    TRY(check_ptr(fn, "freqs", freqs, 4));
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (cu_seqlens != nullptr) TRY(check_cu(fn, s, cu_seqlens, num_seqs, total_T));
    auto fill = [&](auto& a) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(a.q)>>;
        a.r.T = total_T; a.r.positions = positions; a.r.cu = cu_seqlens; a.r.N = num_seqs;
        a.D = D; a.R = rotary_dim; a.Hq = num_heads; a.Hkv = num_kv_heads;
        a.q = static_cast<const E*>(q); a.q_stride = q_stride;
        a.q_out = static_cast<E*>(q_out); a.q_out_stride = q_out_stride;
        a.k = static_cast<const E*>(k); a.k_stride = k_stride;
        a.k_out = static_cast<E*>(k_out); a.k_out_stride = k_out_stride;
        a.freqs = freqs; a.magnitude = magnitude; a.turn = inverse ? -magnitude : magnitude;
        a.per_head = a.items = a.parts = a.part_items = 0;
        return submitted(fn, launch_rotary(a, interleaved != 0, s));
    };
    if (dtype == LFM2SC_BF16) {
        RotaryArgs<uint16_t> a;
        return fill(a);
    }
    RotaryArgs<float> a;
    return fill(a);
}

int lfm2sc_cache8_write(int dtype, int format, int D, int num_kv_heads, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, int64_t total_T, const int32_t* cu_seqlens, int num_seqs, void* k_pages, void* v_pages,
                        int64_t page_stride, float* k_scales, float* v_scales, int64_t scale_stride, int num_pages,
                        int page_size, int scale_tokens, const int32_t* page_table, int max_pages, const int32_t* seq_len,
                        void* stream) {
    return cache8("lfm2sc_cache8_write", true, dtype, format, D, num_kv_heads, const_cast<void*>(k), k_stride,
                  const_cast<void*>(v), v_stride, total_T, cu_seqlens, num_seqs, k_pages, v_pages, page_stride, k_scales,
                  v_scales, scale_stride, num_pages, page_size, scale_tokens, page_table, max_pages, seq_len, stream);
}

int lfm2sc_cache8_read(int dtype, int format, int D, int num_kv_heads, const void* k_pages, const void* v_pages,
                       int64_t page_stride, const float* k_scales, const float* v_scales, int64_t scale_stride, int num_pages,
                       int page_size, int scale_tokens, const int32_t* page_table, int max_pages, const int32_t* seq_len,
                       void* k_out, int64_t k_stride, void* v_out, int64_t v_stride, int64_t total_T, const int32_t* cu_seqlens,
                       int num_seqs, void* stream) {
    return cache8("lfm2sc_cache8_read", false, dtype, format, D, num_kv_heads, k_out, k_stride, v_out, v_stride, total_T,
                  cu_seqlens, num_seqs, const_cast<void*>(k_pages), const_cast<void*>(v_pages), page_stride,
                  const_cast<float*>(k_scales), const_cast<float*>(v_scales), scale_stride, num_pages, page_size, scale_tokens,
                  page_table, max_pages, seq_len, stream);
}

size_t lfm2sc_attn_cached8_workspace_bytes(int dtype, int D, int num_heads, int num_kv_heads, int num_seqs, int L,
                                           int prefix_len, int max_suffix_len) {
    if (dtype != LFM2SC_BF16 || (D != 64 && D != 128) || num_kv_heads < 1 || num_heads < num_kv_heads ||
        num_heads % num_kv_heads != 0 || num_heads > kMaxHeads || num_seqs <= 0 || L <= 0 ||
        !cached_rows_fit(num_seqs, L, num_heads) || prefix_len < 0 || prefix_len >= kMaxKeys || max_suffix_len < 0 ||
        max_suffix_len >= kMaxKeys)
        return 0;
    return cached8_bytes(D, num_heads, num_kv_heads, num_seqs, L, prefix_len, max_suffix_len);
}

int lfm2sc_attn_cached8(int dtype, int format, int D, int num_heads, int num_kv_heads, const void* q, int64_t q_stride,
                        int num_seqs, int L, const void* k_pages, const void* v_pages, int64_t page_stride,
                        const float* k_scales, const float* v_scales, int64_t scale_stride, int num_pages, int page_size,
                        int scale_tokens, const int32_t* prefix_pages, int prefix_len, const int32_t* page_table, int max_pages,
                        const int32_t* suffix_len, int max_suffix_len, float scale, void* out, int64_t out_stride,
                        void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "lfm2sc_attn_cached8";
    TRY(check_heads(fn, dtype, D, num_heads, num_kv_heads));
    TRY(check_scale(fn, scale));
    TRY(check_pool8(fn, format, D, num_kv_heads, page_stride, scale_stride, page_size, scale_tokens, max_pages));
    TRY(check_cached_sizes(fn, num_seqs, L, num_heads, prefix_len, max_pages, page_size));
    if (max_suffix_len < 0 || max_suffix_len > max_pages * page_size)
        return fail(LFM2SC_ERR_BAD_SHAPE, "%s: max_suffix_len=%d outside [0, max_pages * page_size = %d]", fn, max_suffix_len,
                    max_pages * page_size);
    TRY(check_rows(fn, "q_stride", q_stride, (int64_t)num_heads * D));
    TRY(check_rows(fn, "out_stride", out_stride, (int64_t)num_heads * D));
    if (num_seqs == 0 || L == 0) return ok();
    TRY(check_ptr(fn, "q", q, 16));
    if (prefix_len > 0 || max_suffix_len > 0)
        TRY(check_pool8_pages(fn, k_pages, v_pages, k_scales, v_scales, num_pages, page_size));
    if (prefix_len > 0) TRY(check_ptr(fn, "prefix_pages", prefix_pages, 4));
    if (max_suffix_len > 0) TRY(check_ptr(fn, "page_table", page_table, 4));
    TRY(check_ptr(fn, "suffix_len", suffix_len, 4));
    TRY(check_ptr(fn, "out", out, 16));
    const Cached8Plan p = cached8_plan(D, num_heads, num_kv_heads, num_seqs, L, prefix_len, max_suffix_len);
    const bool joins = p.prefix_splits + p.suffix_splits > 1;            // else the rows go straight to `out`
    const size_t need = joins ? cached8_bytes(D, num_heads, num_kv_heads, num_seqs, L, prefix_len, max_suffix_len) : 0;
    TRY(check_workspace(fn, workspace, workspace_bytes, need, 16));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const RangeCheck ranges[] = {
        {prefix_pages, prefix_len > 0 ? ((int64_t)prefix_len + page_size - 1) / page_size : 0, 0, (int64_t)num_pages - 1},
        {page_table, max_suffix_len > 0 ? (int64_t)num_seqs * max_pages : 0, 0, (int64_t)num_pages - 1, suffix_len, max_pages,
         page_size},
        {suffix_len, num_seqs, 0, max_suffix_len}};
    const char* const names[] = {"a prefix page", "a page of page_table", "a suffix length"};
    TRY(check_ranges(fn, s, ranges, names, 3));
    Cached8Args a;
    CachedArgs& c = a.c;
    c.q = static_cast<const uint16_t*>(q); c.q_stride = q_stride; c.N = num_seqs; c.L = L;
    c.Hq = num_heads; c.Hkv = num_kv_heads;
    c.k = c.v = nullptr; c.kv_stride = 0;
    c.num_pages = num_pages; c.page_shift = __builtin_ctz((unsigned)page_size);
    c.prefix_pages = prefix_pages; c.prefix_len = prefix_len;
    c.page_table = page_table; c.max_pages = max_pages; c.suffix_len = suffix_len;
    c.scale = scale;
    c.out = static_cast<uint16_t*>(out); c.out_stride = out_stride;
    const size_t rows = (size_t)num_seqs * (size_t)L * (size_t)num_heads * (size_t)(p.prefix_splits + p.suffix_splits);
    c.part_o = static_cast<float*>(workspace);
    c.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + round_up(rows * (size_t)D * 4));
    c.prefix_splits = c.prefix_chunk = c.suffix_splits = 0;
    c.prefix_blocks = 0;
    a.k = static_cast<const uint8_t*>(k_pages); a.v = static_cast<const uint8_t*>(v_pages); a.page_stride = page_stride;
    a.k_scales = k_scales; a.v_scales = v_scales; a.scale_stride = scale_stride;
    a.block_shift = __builtin_ctz((unsigned)scale_tokens);
    a.max_suffix = max_suffix_len;
    return submitted(fn, launch_attn_cached8(a, D, format == LFM2SC_CACHE_INT8, s));
}

}  // extern "C"
