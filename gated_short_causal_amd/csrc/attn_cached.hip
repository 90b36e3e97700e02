// attn_cached.hip -- attention of new tokens over a paged cache whose first
// keys, the prefix, are shared by the whole batch.
//
// The prefix's keys are read once for all sequences: every query row of the
// batch that uses a key/value head (num_seqs * L * G of them) is a row of one
// product with them.  A sequence's own keys (the suffix) serve its L * G rows
// of that head.  Both are split along the keys, so that a few sequences still
// fill the card; each split leaves its rows' running maximum m, sum l and
// unnormalised output in the workspace, and a second kernel joins them:
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,   m = max m_i.
// One launch holds the workgroups of both kinds, the prefix's first (they run
// longest).  All sums are fp32; p is rounded to bf16 for the product with v.
#include "attn_common.hpp"
#include "hybrid.hpp"

namespace lfm2sc {

constexpr int kCW = 4;                        // waves per workgroup
constexpr int kCRows = 32 * kCW;              // query rows of a prefix workgroup
constexpr int kPrefixTile = 64;               // keys per staged tile, prefix
template <int D> constexpr int kSuffixTile = 4096 / D;   // keys per wave's tile, suffix: 8 KiB of K, 8 KiB of V

// Row number in the pool of key idx of a page list; idx < 2^31.  A page number
// outside the pool reads as the nearest page of it.
__device__ __forceinline__ uint32_t pool_row(const CachedArgs& a, const int32_t* pages, int idx) {
    const int p = min(max(pages[idx >> a.page_shift], 0), a.num_pages - 1);
    return ((uint32_t)p << a.page_shift) + (uint32_t)(idx & ((1 << a.page_shift) - 1));
}

// Copies n KiB of a tile whose row r lies at pool row `rows` of lane r.
template <int D, int N>
__device__ __forceinline__ void copy_paged(const uint16_t* pool, int64_t stride, uint32_t rows, uint8_t* lds, int first,
                                           int lane) {
    using T = Tile<D>;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = (first + i) * T::kRowsPerDma + lane / T::kChunks;
        const uint32_t at = (uint32_t)__shfl((int)rows, r, 64);
        const uint16_t* p = pool + (int64_t)at * stride + ((lane % T::kChunks) ^ T::rot(r)) * 8;
        __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) const void*)p,
                                         (lds_ptr_t)(lds + (first + i) * 1024), 16, 0, 0);
    }
}

// Running softmax state of a wave's 32 query rows (one per lane pair c, c + 32).
template <int D>
struct Rows {
    float m, l;
    f32x16 o[D / 32];
    __device__ void clear() {
        m = kNegInf;
        l = 0.f;
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[b][i] = 0.f;
    }
};

// One staged tile of KT keys against the wave's rows.  Keys numbered above
// `seen` (the lane's row's last visible key within the tile) are masked.
template <int D, int KT>
__device__ __forceinline__ void attend(Rows<D>& r, const bf16x8 (&qf)[D / 16], const uint8_t* kb, const uint8_t* vb,
                                       const LaneOffsets<D>& lo, float cs, bool masked, int seen, int h) {
    using T = Tile<D>;
    f32x16 s[KT / 32];
#pragma unroll
    for (int n = 0; n < KT / 32; ++n) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[n][i] = 0.f;
#pragma unroll
        for (int ds = 0; ds < D / 16; ++ds) s[n] = mfma32(lds_row(kb + n * 32 * T::kRowB, lo.row[ds]), qf[ds], s[n]);
    }
    if (masked) {
#pragma unroll
        for (int n = 0; n < KT / 32; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (n * 32 + 4 * h + (i & 3) + 8 * (i >> 2) > seen) s[n][i] = kNegInf;
    }
    float mx = s[0][0];
#pragma unroll
    for (int n = 0; n < KT / 32; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[n][i]);
    const float mn = fmaxf(r.m, max_halves(mx) * cs);
    const float ref = mn == kNegInf ? 0.f : mn;      // a row that has seen no key yet: every p is 0
    const float alpha = exp2_fast(r.m - ref);
    r.m = mn;
    r.l *= alpha;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) r.o[b][i] *= alpha;
#pragma unroll
    for (int n = 0; n < KT / 32; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[n][i] = exp2_fast(__builtin_fmaf(s[n][i], cs, -ref));
            r.l += s[n][i];
        }
#pragma unroll
    for (int n = 0; n < KT / 32; ++n)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const bf16x8 p = to_operand(s[n], ks);
#pragma unroll
            for (int b = 0; b < D / 32; ++b)
                r.o[b] = mfma32(lds_transposed(vb + (n * 32 + ks * 16) * T::kRowB, lo.tr[0][b], lo.tr[1][b]), p, r.o[b]);
        }
}

// Query row x of a key/value head: x = (token row) * G + head in the group.
struct QueryRow {
    int64_t token;
    int head;
};
__device__ __forceinline__ QueryRow query_row(const CachedArgs& a, int G, int kvh, int64_t x) {
    return QueryRow{x / G, kvh * G + (int)(x % G)};
}

// Leaves a row's state (after sum_halves of l) in split `split` of the workspace.
template <int D>
__device__ __forceinline__ void store_part(const CachedArgs& a, int split, const QueryRow& q, const Rows<D>& r, float l, int h) {
    const int64_t at = ((int64_t)split * a.N * a.L + q.token) * a.Hq + q.head;
    float* o = a.part_o + at * D + 4 * h;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(o + 32 * b + 2 * i) = make_float4(r.o[b][i], r.o[b][i + 1], r.o[b][i + 2], r.o[b][i + 3]);
    if (h == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(r.m, l);
}

template <int D>
__device__ void prefix_part(const CachedArgs& a, uint8_t* lds, int block, int wave, int lane) {
    using T = Tile<D>;
    constexpr int kTileB = kPrefixTile * T::kRowB;
    constexpr int kDma = kTileB / 1024 / kCW;
    const int c = lane & 31, h = lane >> 5, G = a.Hq / a.Hkv;
    const int kvh = block % a.Hkv, rest = block / a.Hkv;
    const int split = rest % a.prefix_splits;
    const int64_t rows = (int64_t)a.N * a.L * G;
    const int64_t x = (int64_t)(rest / a.prefix_splits) * kCRows + wave * 32 + c;
    const int k0 = split * a.prefix_chunk, k1 = min(k0 + a.prefix_chunk, a.prefix_len);   // k0 < k1
    const int tiles = (k1 - k0 + kPrefixTile - 1) / kPrefixTile;
    const bool busy = x - c < rows;              // the wave has a row

    auto rows_of = [&](int t) { return pool_row(a, a.prefix_pages, min(k0 + t * kPrefixTile + lane, k1 - 1)); };
    auto issue = [&](uint8_t* buf, uint32_t pr) {
        copy_paged<D, kDma>(a.k + (int64_t)kvh * D, a.kv_stride, pr, buf, wave * kDma, lane);
        copy_paged<D, kDma>(a.v + (int64_t)kvh * D, a.kv_stride, pr, buf + kTileB, wave * kDma, lane);
    };
    issue(lds, rows_of(0));
    uint32_t next = rows_of(min(1, tiles - 1));

    const QueryRow q = query_row(a, G, kvh, min(x, rows - 1));
    bf16x8 qf[D / 16];
    load_row_operand<D>(qf, a.q + q.token * a.q_stride + (int64_t)q.head * D, h, x < rows);
    const LaneOffsets<D> lo(lane);
    const float cs = a.scale * kLog2e;
    Rows<D> r;
    r.clear();
    for (int t = 0; t < tiles; ++t) {
        uint8_t* cur = lds + (t & 1) * 2 * kTileB;
        wait_vm<0>();
        stage_barrier();
        if (t + 1 < tiles) {
            issue(lds + ((t + 1) & 1) * 2 * kTileB, next);
            next = rows_of(min(t + 2, tiles - 1));
        }
        const int seen = k1 - 1 - k0 - t * kPrefixTile;
        if (busy) attend<D, kPrefixTile>(r, qf, cur, cur + kTileB, lo, cs, seen < kPrefixTile - 1, seen, h);
    }
    const float l = sum_halves(r.l);
    if (x < rows) store_part<D>(a, split, q, r, l, h);
}

// The suffix keys of one sequence for 32 of its rows of one head: the waves
// take every kCW-th tile, each with its own staging buffer, and join through LDS.
template <int D>
__device__ void suffix_part(const CachedArgs& a, uint8_t* lds, int block, int wave, int lane) {
    using T = Tile<D>;
    constexpr int KT = kSuffixTile<D>;
    constexpr int kTileB = KT * T::kRowB;        // 8 KiB
    const int c = lane & 31, h = lane >> 5, G = a.Hq / a.Hkv;
    const int kvh = block % a.Hkv;
    int rest = block / a.Hkv;
    const int split = rest % a.suffix_splits;
    rest /= a.suffix_splits;
    const int blocks = (a.L * G + 31) / 32;
    const int seq = rest / blocks, rb = rest % blocks;
    const int32_t* pages = a.page_table + (int64_t)seq * a.max_pages;
    const int len = min(max(a.suffix_len[seq], 0), a.max_pages << a.page_shift);
    const int all = (len + KT - 1) / KT, per = (all + a.suffix_splits - 1) / a.suffix_splits;
    const int t0 = min(split * per, all), t1 = min(t0 + per, all);

    const int y = rb * 32 + c;                   // row among the sequence's L * G
    const bool exists = y < a.L * G;
    const QueryRow q = query_row(a, G, kvh, (int64_t)seq * a.L * G + min(y, a.L * G - 1));
    const int last = len - a.L + min(y, a.L * G - 1) / G;    // the row's last visible key
    bf16x8 qf[D / 16];
    load_row_operand<D>(qf, a.q + q.token * a.q_stride + (int64_t)q.head * D, h, exists);
    const LaneOffsets<D> lo(lane);
    const float cs = a.scale * kLog2e;
    Rows<D> r;
    r.clear();
    uint8_t* buf = lds + wave * 2 * kTileB;
    auto rows_of = [&](int t) { return pool_row(a, pages, min(t * KT + lane % KT, len - 1)); };
    const int mine = t0 + wave;
    if (mine < t1) {
        uint32_t cur = rows_of(mine);
        for (int t = mine; t < t1; t += kCW) {
            copy_paged<D, kTileB / 1024>(a.k + (int64_t)kvh * D, a.kv_stride, cur, buf, 0, lane);
            copy_paged<D, kTileB / 1024>(a.v + (int64_t)kvh * D, a.kv_stride, cur, buf + kTileB, 0, lane);
            if (t + kCW < t1) cur = rows_of(t + kCW);
            wait_vm<0>();
            attend<D, KT>(r, qf, buf, buf + kTileB, lo, cs, t * KT + KT - 1 > len - a.L, last - t * KT, h);
        }
    }
    // join the waves: their m, l and o in LDS, then wave 0 adds them up
    const float l = sum_halves(r.l);
    lds_barrier();
    float* fo = reinterpret_cast<float*>(lds);                   // [wave][D / 32 * 4][64 lanes][4]
    float* fm = fo + (kCW - 1) * D * 32;
    if (wave > 0) {
        float* p = fo + (wave - 1) * D * 32;
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(p + ((b * 4 + i / 4) * 64 + lane) * 4) =
                    make_float4(r.o[b][i], r.o[b][i + 1], r.o[b][i + 2], r.o[b][i + 3]);
        fm[(wave - 1) * 128 + lane] = r.m;
        fm[(wave - 1) * 128 + 64 + lane] = l;
    }
    lds_barrier();
    if (wave > 0) return;
    float top = r.m, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kCW - 1; ++w) top = fmaxf(top, fm[w * 128 + lane]);
    const float ref = top == kNegInf ? 0.f : top;
    const float own = exp2_fast(r.m - ref);
    sum = own * l;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) r.o[b][i] *= own;
#pragma unroll
    for (int w = 0; w < kCW - 1; ++w) {
        const float f = exp2_fast(fm[w * 128 + lane] - ref);
        sum += f * fm[w * 128 + 64 + lane];
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(fo + w * D * 32 + ((b * 4 + i / 4) * 64 + lane) * 4);
                r.o[b][i] += f * v.x; r.o[b][i + 1] += f * v.y; r.o[b][i + 2] += f * v.z; r.o[b][i + 3] += f * v.w;
            }
    }
    r.m = top;
    if (exists) store_part<D>(a, a.prefix_splits + split, q, r, sum, h);
}

template <int D>
__global__ __launch_bounds__(64 * kCW, 2) void attn_cached_kernel(CachedArgs a) {
    constexpr int kPrefixB = 2 * 2 * kPrefixTile * 2 * D;                       // two tiles of K and V
    constexpr int kSuffixB = kCW * 2 * 8192;                                    // a tile of K and V per wave
    constexpr int kJoinB = (kCW - 1) * (D * 32 + 128) * 4;
    constexpr int kA = kPrefixB > kSuffixB ? kPrefixB : kSuffixB;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kA > kJoinB ? kA : kJoinB];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if ((int)blockIdx.x < a.prefix_blocks) prefix_part<D>(a, lds, blockIdx.x, wave, lane);
    else suffix_part<D>(a, lds, blockIdx.x - a.prefix_blocks, wave, lane);
}

// Joins the splits: D / 4 lanes per (token row, head).
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(CachedArgs a) {
    constexpr int kLanes = D / 4;
    const int64_t rows = (int64_t)a.N * a.L * a.Hq;
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / kLanes;
    const int j = threadIdx.x % kLanes;
    if (row >= rows) return;
    const int splits = a.prefix_splits + a.suffix_splits;
    float m = kNegInf, l = 0.f;
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s) {
        const int64_t at = s * rows + row;
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
        const float4 x = *reinterpret_cast<const float4*>(a.part_o + at * D + 4 * j);
        const float mn = fmaxf(m, ml.x), ref = mn == kNegInf ? 0.f : mn;
        const float f0 = exp2_fast(m - ref), f1 = exp2_fast(ml.x - ref);
        m = mn;
        l = l * f0 + ml.y * f1;
        o[0] = o[0] * f0 + x.x * f1;
        o[1] = o[1] * f0 + x.y * f1;
        o[2] = o[2] * f0 + x.z * f1;
        o[3] = o[3] * f0 + x.w * f1;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);      // no visible key: 0; NaN stays
    uint2 v;
    v.x = Elem<uint16_t>::pack2(o[0] * inv, o[1] * inv);
    v.y = Elem<uint16_t>::pack2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(a.out + row / a.Hq * a.out_stride + (row % a.Hq) * D + 4 * j) = v;
}

// Splits.  The card has 256 CUs, two workgroups each: the prefix gets as many
// splits of at least 64 keys as one round of 512 workgroups holds, the suffixes
// as many of at least one tile per wave as two rounds hold.
CachedPlan cached_plan(int D, int Hq, int Hkv, int N, int L, int prefix_len, int max_keys) {
    CachedPlan p;
    const int G = Hq / Hkv;
    const int64_t rows = (int64_t)N * L * G;
    const int64_t row_blocks = (rows + kCRows - 1) / kCRows;
    p.prefix_splits = 0;
    p.prefix_chunk = 0;
    p.prefix_blocks = 0;
    if (prefix_len > 0) {
        const int tiles = (prefix_len + kPrefixTile - 1) / kPrefixTile;
        const int64_t want = 512 / (row_blocks * Hkv);
        const int splits = (int)(want < 1 ? 1 : want < tiles ? want : tiles);
        const int per = (tiles + splits - 1) / splits;
        p.prefix_chunk = per * kPrefixTile;
        p.prefix_splits = (tiles + per - 1) / per;
        p.prefix_blocks = row_blocks * Hkv * p.prefix_splits;
    }
    const int64_t base = (int64_t)N * ((L * G + 31) / 32) * Hkv;
    const int64_t per_wg = (int64_t)kCW * 4096 / D;
    const int64_t most = (max_keys + per_wg - 1) / per_wg, want = 1024 / base;
    p.suffix_splits = (int)(want < 1 ? 1 : want < most ? want : most);
    if (p.suffix_splits < 1) p.suffix_splits = 1;
    p.suffix_blocks = base * p.suffix_splits;
    return p;
}

template <int D>
static hipError_t launch_cached(const CachedArgs& a, int64_t suffix_blocks, hipStream_t s) {
    const int64_t blocks = a.prefix_blocks + suffix_blocks;
    const int64_t joins = ((int64_t)a.N * a.L * a.Hq * (D / 4) + 255) / 256;
    if (blocks >= ((int64_t)1 << 31) || joins >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((attn_cached_kernel<D>), dim3((uint32_t)blocks), dim3(64 * kCW), 0, s, a);
    hipLaunchKernelGGL((attn_join_kernel<D>), dim3((uint32_t)joins), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_attn_cached(CachedArgs a, int D, hipStream_t s) {
    const CachedPlan p = cached_plan(D, a.Hq, a.Hkv, a.N, a.L, a.prefix_len, a.max_pages << a.page_shift);
    a.prefix_splits = p.prefix_splits;
    a.prefix_chunk = p.prefix_chunk;
    a.prefix_blocks = p.prefix_blocks;
    a.suffix_splits = p.suffix_splits;
    return D == 64 ? launch_cached<64>(a, p.suffix_blocks, s) : launch_cached<128>(a, p.suffix_blocks, s);
}

}  // namespace lfm2sc
