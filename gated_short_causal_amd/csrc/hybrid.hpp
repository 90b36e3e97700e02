// hybrid.hpp -- argument blocks and launchers of the operators around the
// ShortConv in the hybrid decoder (include/lfm2sc_hybrid.h): attention over
// packed prompts (attn_fwd.hip, attn_bwd.hip), attention over a paged cache
// with a shared prefix (attn_cached.hip) and draft verification (drafts.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lfm2sc {

struct AttnArgs {
    const uint16_t* q; int64_t q_stride;
    const uint16_t* k; int64_t k_stride;
    const uint16_t* v; int64_t v_stride;
    int64_t total_T;
    const int32_t* cu; int N;
    int Hq, Hkv;
    float scale;
    uint16_t* out; int64_t out_stride;   // read by the backward
    float* lse;                          // [Hq][total_T]; nullptr: not written
};

struct AttnGradArgs {
    AttnArgs f;
    const uint16_t* dout; int64_t dout_stride;
    uint16_t* dq; int64_t dq_stride;
    uint16_t* dk; int64_t dk_stride;
    uint16_t* dv; int64_t dv_stride;
    float* delta;                        // workspace, [Hq][total_T]
    float* lse2;                         // workspace, [Hq][total_T]
    float* part;                         // workspace, [splits][2][total_T][Hkv * D] when splits > 1
    int splits;                          // workgroups that share a key block's query heads
};

struct CachedArgs {
    const uint16_t* q; int64_t q_stride; int N, L;
    int Hq, Hkv;
    const uint16_t* k; const uint16_t* v; int64_t kv_stride;   // pools [num_pages << page_shift] rows
    int num_pages, page_shift;
    const int32_t* prefix_pages; int prefix_len;
    const int32_t* page_table; int max_pages; const int32_t* suffix_len;
    float scale;
    uint16_t* out; int64_t out_stride;
    float* part_o;                       // workspace [splits][N * L][Hq][D]
    float* part_ml;                      // workspace [splits][N * L][Hq][2]
    int prefix_splits, prefix_chunk, suffix_splits;   // set by the launcher, as is
    int64_t prefix_blocks;                            // the number of prefix workgroups
};
struct CachedPlan {
    bool direct;                         // one workgroup per sequence, head and 32 rows; no workspace
    int prefix_splits, prefix_chunk, suffix_splits;
    int64_t prefix_blocks, suffix_blocks;
};
CachedPlan cached_plan(int D, int Hq, int Hkv, int N, int L, int prefix_len, int max_keys);

template <typename E>
struct DraftArgs {
    const E* target; int64_t target_stride;      // [N * (L + 1)] rows of V
    const E* draft; int64_t draft_stride;        // [N * L] rows of V, or nullptr
    int V, N, L;
    const int32_t* tokens;                       // [N][L]
    const int32_t* num_drafts;                   // [N] or nullptr
    const float* u_accept; const float* u_sample;
    int32_t* accept_len; int32_t* keep_len; int32_t* next_token;
    double* sums;                                // workspace [N][2][chunks]
};
constexpr int kDraftChunk = 4096;                // tokens per chunk of the split form
int draft_chunks(int V);

// Host check of int32 device data (check.hip): n entries within [lo, hi].  With
// `len`, the entries are runs of `row`, of which run i uses the first
// ceil(len[i] / per); the others may hold anything.
struct RangeCheck {
    const int32_t* v;
    int64_t n, lo, hi;
    const int32_t* len = nullptr;
    int64_t row = 1, per = 1;
};
int check_device_ranges(hipStream_t s, const RangeCheck* checks, int count, hipError_t* err);

// A launch holds fewer than 2^32 work-items a dimension.  The launchers below return
// hipErrorInvalidConfiguration, before they launch anything, where a call needs more.
inline bool too_many(int64_t blocks, int threads) { return blocks * threads >= (int64_t)1 << 32; }

hipError_t launch_attn_prefill(const AttnArgs& a, int D, hipStream_t s);
int attn_backward_splits(int Hq, int Hkv, int64_t total_T, int N);
hipError_t launch_attn_backward(const AttnGradArgs& a, int D, hipStream_t s);
hipError_t launch_attn_cached(CachedArgs a, int D, hipStream_t s);
template <typename E>
hipError_t launch_drafts(const DraftArgs<E>& a, hipStream_t s);

}  // namespace lfm2sc
