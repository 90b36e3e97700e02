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
// longest).  All sums are fp32; p is rounded to bf16 once, as the matrix unit's
// operand of the product with v (outputs 2.2-2.3e-3 off, 1.7e-3 from their own
// rounding alone); the splits' partial outputs stay fp32.
#include "attn_common.hpp"
#include "hybrid.hpp"

namespace lfm2sc {

constexpr int kCW = 4;                        // waves per workgroup of the split form
constexpr int kCRows = 32 * kCW;              // query rows of a prefix workgroup
constexpr int kPrefixTile = 64;               // keys per staged tile, prefix
constexpr int kOwnTile = 32;                  // keys per wave's tile, suffix
constexpr int kDirectW = 8;                   // waves per workgroup of the direct form

// Row number in the pool of key idx (< 2^31), whose page number is `page`.  A
// page number outside the pool reads as the nearest page of it.  The number is
// loaded a tile ahead and only looked at when it is used: clamping it at once
// would wait for it, and with it for the copies issued before it.
__device__ __forceinline__ uint32_t pool_row(const CachedArgs& a, int32_t page, int idx) {
    const int p = min(max(page, 0), a.num_pages - 1);
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

// Running softmax state of a wave's 32 query rows (one per lane pair c, c + 32):
// the reference m, sum l and output o, all relative to 2^m.
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

// One staged tile of KT keys against the wave's rows.  If `masked` (uniform),
// keys numbered above `seen`, the lane's row's last visible key within the
// tile, are masked.  A row that has seen no key keeps m = -inf and o = l = 0.
// after_k runs when the K tile has been read, before_v before the V tile is.
template <int D, int KT, typename F1, typename F2>
__device__ __forceinline__ void attend(Rows<D>& r, const bf16x8 (&qf)[D / 16], const uint8_t* kb, const uint8_t* vb,
                                       const LaneOffsets<D>& lo, float cs, bool masked, int seen, int h, F1 after_k,
                                       F2 before_v) {
    using T = Tile<D>;
    f32x16 s[KT / 32];
#pragma unroll
    for (int n = 0; n < KT / 32; ++n) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[n][i] = 0.f;
#pragma unroll
        for (int ds = 0; ds < D / 16; ++ds) s[n] = mfma32(lds_row(kb + n * 32 * T::kRowB, lo.row[ds]), qf[ds], s[n]);
    }
    after_k();
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
    const float mn = max_halves(mx) * cs;
    if (__any(mn > r.m + kLazy)) {
        const float m = fmaxf(r.m, mn), alpha = exp2_fast(r.m - (m == kNegInf ? 0.f : m));
        r.m = m;
        r.l *= alpha;
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) r.o[b][i] *= alpha;
    }
    const float ref = r.m == kNegInf ? 0.f : r.m;
    float sum = 0.f;
#pragma unroll
    for (int n = 0; n < KT / 32; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[n][i] = exp2_fast(__builtin_fmaf(s[n][i], cs, -ref));
            sum += s[n][i];
        }
    r.l += sum;
    before_v();
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

// The prefix's keys [split] for 128 query rows of one head; the waves share the
// staged tiles, two buffers of K and V.
template <int D>
__device__ __forceinline__ void prefix_part(const CachedArgs& a, uint8_t* buf0, uint8_t* buf1, int block, int wave, int lane) {
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

    auto key_of = [&](int t) { return min(k0 + t * kPrefixTile + lane, k1 - 1); };
    auto page_of = [&](int t) { return a.prefix_pages[key_of(t) >> a.page_shift]; };
    auto issue = [&](uint8_t* buf, uint32_t pr) {
        copy_paged<D, kDma>(a.k + (int64_t)kvh * D, a.kv_stride, pr, buf, wave * kDma, lane);
        copy_paged<D, kDma>(a.v + (int64_t)kvh * D, a.kv_stride, pr, buf + kTileB, wave * kDma, lane);
    };
    issue(buf0, pool_row(a, page_of(0), key_of(0)));
    int32_t next = page_of(min(1, tiles - 1));

    const QueryRow q = query_row(a, G, kvh, min(x, rows - 1));
    bf16x8 qf[D / 16];
    load_row_operand<D>(qf, a.q + q.token * a.q_stride + (int64_t)q.head * D, h, x < rows);
    const LaneOffsets<D> lo(lane);
    const float cs = a.scale * kLog2e;
    Rows<D> r;
    r.clear();
    auto step = [&](const uint8_t* cur, uint8_t* other, int t) {
        wait_vm<0>();
        stage_barrier();
        if (t + 1 < tiles) {
            issue(other, pool_row(a, next, key_of(t + 1)));
            next = page_of(min(t + 2, tiles - 1));
        }
        const int seen = k1 - 1 - k0 - t * kPrefixTile;
        if (busy) attend<D, kPrefixTile>(r, qf, cur, cur + kTileB, lo, cs, seen < kPrefixTile - 1, seen, h, [] {}, [] {});
    };
    for (int t = 0; t < tiles; t += 2) {
        step(buf0, buf1, t);
        if (t + 1 < tiles) step(buf1, buf0, t + 1);
    }
    const float l = sum_halves(r.l);
    if (x < rows) store_part<D>(a, split, q, r, l, h);
}

// Keys of one sequence for 32 of its rows of one head: its own (kDirect: the
// prefix's as well).  The W waves take every W-th tile of KT keys, each with a
// staging buffer of its own, and join through LDS: wave w then adds up pieces
// w, w + W, .. (4 values of each row) of all waves.  kDirect, or the only
// split of all keys: the sum is the output; else it is left in the workspace.
template <int D, int W, int KT, bool kDirect>
__device__ __forceinline__ void own_part(const CachedArgs& a, uint8_t* buf0, uint8_t* buf1, float (*ml)[2][64], int block,
                                         int wave, int lane) {
    using T = Tile<D>;
    constexpr int kTileB = KT * T::kRowB;
    constexpr int kWaveB = 2 * kTileB;
    static_assert(kWaveB >= D * 32 * 4, "a wave's o fits its staging buffer");
    const int c = lane & 31, h = lane >> 5, G = a.Hq / a.Hkv;
    const int kvh = block % a.Hkv;
    int rest = block / a.Hkv;
    const int splits = kDirect ? 1 : a.suffix_splits, split = rest % splits;
    rest /= splits;
    const int blocks = (a.L * G + 31) / 32;
    const int seq = rest / blocks, rb = rest % blocks;
    const int32_t* pages = a.page_table + (int64_t)seq * a.max_pages;
    const int len = min(max(a.suffix_len[seq], 0), a.max_pages << a.page_shift);
    const int prefix = kDirect ? a.prefix_len : 0, pt = (prefix + KT - 1) / KT;     // tiles of the prefix come first
    const int all = pt + (len + KT - 1) / KT, per = (all + splits - 1) / splits;
    const int t0 = min(split * per, all), t1 = min(t0 + per, all);

    const int y = rb * 32 + c;                   // row among the sequence's L * G
    const bool exists = y < a.L * G;
    const QueryRow q = query_row(a, G, kvh, (int64_t)seq * a.L * G + min(y, a.L * G - 1));
    const int last = len - a.L + min(y, a.L * G - 1) / G;    // the row's last visible own key
    const LaneOffsets<D> lo(lane);
    const float cs = a.scale * kLog2e;
    Rows<D> r;
    r.clear();
    auto region = [&](int w) { return (w < W / 2 ? buf0 : buf1) + (w % (W / 2)) * kWaveB; };
    uint8_t* kb = buf0 + wave * kTileB;
    uint8_t* vb = buf1 + wave * kTileB;
    auto key_of = [&](int t) {
        return kDirect && t < pt ? min(t * KT + lane % KT, prefix - 1) : min((t - pt) * KT + lane % KT, len - 1);
    };
    auto page_of = [&](int t) { return (kDirect && t < pt ? a.prefix_pages : pages)[key_of(t) >> a.page_shift]; };
    // The wave's next K tile is copied as soon as the scores of this one are formed, the next V tile after the
    // products with this one, and the page numbers a tile before that; so its waits leave the copies issued later in
    // flight.  Order of its vector memory operations: pages(t + 1), K(t), V(t), [pages(t + 2), K(t + 1)], V(t + 1), ..
    // Each wait leaves exactly the copies of one tile in flight, so it holds however many loads the compiler makes of
    // the page numbers; the one before V therefore waits for pages(t + 2) too.
    constexpr int kN = kTileB / 1024;
    const uint16_t* kp = a.k + (int64_t)kvh * D;
    const uint16_t* vp = a.v + (int64_t)kvh * D;
    const int mine = t0 + wave;
    bf16x8 qf[D / 16];
    load_row_operand<D>(qf, a.q + q.token * a.q_stride + (int64_t)q.head * D, h, exists);
    int32_t next = 0;
    uint32_t rows = 0;
    if (mine < t1) {
        rows = pool_row(a, page_of(mine), key_of(mine));
        next = page_of(min(mine + W, t1 - 1));
        copy_paged<D, kN>(kp, a.kv_stride, rows, kb, 0, lane);
        copy_paged<D, kN>(vp, a.kv_stride, rows, vb, 0, lane);
    }
    auto tile = [&](auto more_c, int t) {        // more: the wave has another tile after this one
        constexpr bool more = decltype(more_c)::value;
        wait_vm<kN>();
        asm volatile("" ::: "memory");
        auto after_k = [&] {
            if constexpr (more) {
                rows = pool_row(a, next, key_of(t + W));
                next = page_of(min(t + 2 * W, t1 - 1));
                lds_reads_done();                // of this K tile
                copy_paged<D, kN>(kp, a.kv_stride, rows, kb, 0, lane);
            }
        };
        auto before_v = [&] {
            wait_vm<more ? kN : 0>();
            asm volatile("" ::: "memory");
        };
        const int k0 = (t - pt) * KT;            // first own key of the tile; negative: a tile of the prefix
        const bool shared = kDirect && t < pt;
        attend<D, KT>(r, qf, kb, vb, lo, cs, shared ? t * KT + KT > prefix : k0 + KT - 1 > len - a.L,
                      shared ? prefix - 1 - t * KT : last - k0, h, after_k, before_v);
        if constexpr (more) {
            lds_reads_done();                    // of this V tile
            copy_paged<D, kN>(vp, a.kv_stride, rows, vb, 0, lane);
        }
    };
    if (mine < t1) {
        int t = mine;
        for (; t + W < t1; t += W) tile(std::true_type{}, t);
        tile(std::false_type{}, t);
    }
    const float l = sum_halves(r.l);
    lds_barrier();
    float* mine_o = reinterpret_cast<float*>(region(wave));      // [D / 8 pieces][64 lanes][4]
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(mine_o + ((b * 4 + i / 4) * 64 + lane) * 4) =
                make_float4(r.o[b][i], r.o[b][i + 1], r.o[b][i + 2], r.o[b][i + 3]);
    ml[wave][0][lane] = r.m;
    ml[wave][1][lane] = l;
    lds_barrier();
    float top = kNegInf, sum = 0.f, f[W];
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w][0][lane]);
    const float ref = top == kNegInf ? 0.f : top;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        f[w] = exp2_fast(ml[w][0][lane] - ref);
        sum += f[w] * ml[w][1][lane];
    }
    const bool whole = kDirect || a.prefix_splits + splits == 1;
    // no visible key: 0; a NaN stays
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const int64_t at = ((int64_t)(a.prefix_splits + split) * a.N * a.L + q.token) * a.Hq + q.head;
#pragma unroll
    for (int g = wave; g < D / 8; g += W) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(region(w)) + (g * 64 + lane) * 4);
            x.x = __builtin_fmaf(f[w], v.x, x.x);
            x.y = __builtin_fmaf(f[w], v.y, x.y);
            x.z = __builtin_fmaf(f[w], v.z, x.z);
            x.w = __builtin_fmaf(f[w], v.w, x.w);
        }
        const int col = 8 * g + 4 * h;           // values 32 b + 8 (i / 4) + 4 h ..
        if (!exists) continue;
        if (whole) {
            *reinterpret_cast<uint2*>(a.out + q.token * a.out_stride + (int64_t)q.head * D + col) =
                make_uint2(Elem<uint16_t>::pack2(x.x * inv, x.y * inv), Elem<uint16_t>::pack2(x.z * inv, x.w * inv));
        } else {
            *reinterpret_cast<float4*>(a.part_o + at * D + col) = x;
        }
    }
    if (!whole && exists && wave == 0 && h == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(top, sum);
}

// Split form: the prefix's workgroups first, which run longest, then the
// suffixes'.
template <int D>
__global__ __launch_bounds__(64 * kCW, D == 64 ? 4 : 2) void attn_cached_kernel(CachedArgs a) {
    constexpr int kBufB = 2 * kPrefixTile * Tile<D>::kRowB;
    static_assert(kBufB == 2 * 2 * kOwnTile * Tile<D>::kRowB, "two waves' staging per buffer");
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[kBufB], buf1[kBufB];
    __shared__ float ml[kCW][2][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int b = blockIdx.x, p = (int)a.prefix_blocks;
    if (b < p) prefix_part<D>(a, buf0, buf1, b, wave, lane);
    else own_part<D, kCW, kOwnTile, false>(a, buf0, buf1, ml, b - p, wave, lane);
}

// Direct form, for few keys: one workgroup per sequence, head and 32 rows reads
// prefix and suffix and writes the output.
template <int D>
__global__ __launch_bounds__(64 * kDirectW) void attn_cached_direct_kernel(CachedArgs a) {
    constexpr int KT = 4096 / D, kBufB = kDirectW / 2 * 2 * KT * Tile<D>::kRowB;
    __shared__ __attribute__((aligned(1024))) uint8_t buf0[kBufB], buf1[kBufB];
    __shared__ float ml[kDirectW][2][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    own_part<D, kDirectW, KT, true>(a, buf0, buf1, ml, blockIdx.x, wave, threadIdx.x & 63);
}

// Joins the splits: a wave per (token row, head).  First every lane takes a
// split's m and l, then D / 4 lanes times 256 / D groups of them add up o.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(CachedArgs a) {
    constexpr int kLanes = D / 4, kGroups = 64 / kLanes;
    const int64_t rows = (int64_t)a.N * a.L * a.Hq;
    const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, j = lane % kLanes, g = lane / kLanes;
    if (row >= rows) return;
    const int splits = a.prefix_splits + a.suffix_splits;
    float m = kNegInf, l = 0.f;
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < splits; s0 += 64) {
        float2 ml = make_float2(kNegInf, 0.f);
        if (s0 + lane < splits) ml = *reinterpret_cast<const float2*>(a.part_ml + ((s0 + lane) * rows + row) * 2);
        float mn = ml.x;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) mn = fmaxf(mn, __shfl_xor(mn, d, 64));
        mn = fmaxf(mn, m);
        const float ref = mn == kNegInf ? 0.f : mn;
        const float f = exp2_fast(ml.x - ref), old = exp2_fast(m - ref);
        float sum = f * ml.y;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
        m = mn;
        l = l * old + sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= old;
        const int n = min(64, splits - s0);
        for (int s = 0; s < n; s += kGroups) {
            const float w = __shfl(f, s + g, 64);
            if (s + g < n) {
                const float4 x = *reinterpret_cast<const float4*>(a.part_o + ((s0 + s + g) * rows + row) * D + 4 * j);
                o[0] = __builtin_fmaf(w, x.x, o[0]);
                o[1] = __builtin_fmaf(w, x.y, o[1]);
                o[2] = __builtin_fmaf(w, x.z, o[2]);
                o[3] = __builtin_fmaf(w, x.w, o[3]);
            }
        }
    }
#pragma unroll
    for (int d = kLanes; d < 64; d <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], d, 64);
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);      // no visible key: 0; a NaN stays
    uint2 v;
    v.x = Elem<uint16_t>::pack2(o[0] * inv, o[1] * inv);
    v.y = Elem<uint16_t>::pack2(o[2] * inv, o[3] * inv);
    if (g == 0) *reinterpret_cast<uint2*>(a.out + row / a.Hq * a.out_stride + (row % a.Hq) * D + 4 * j) = v;
}

// The direct form where a workgroup per (sequence, head) covers all keys in two
// rounds of its waves and the card holds them all at once.  us in a graph, direct /
// split, 32 / 8 heads of 64: one sequence, prefix 500, suffix 37: 6.1 / 6.9; 32
// sequences 6.5 / 8.2; without a prefix 250 keys 4.5 / 6.6, 1000 keys 7.2 / 6.8 (32
// sequences 9.8 / 13.3).  Up to 128 keys without a prefix the split form is one
// launch too and 0.4 us faster (64 keys 4.1 / 3.8).  128-wide heads the same way
// (40 / 8, 250 keys: 5.9 / 7.8).
//
// Splits of the split form: the prefix gets workgroups of at least 64 keys, one
// per CU where the suffixes' bytes take longer than the prefix's products (the
// rest of the CU reads suffixes meanwhile), two where they do not; the suffixes
// as many of at least a tile per wave as two rounds of 512 hold.  Measured with
// 1 / 2 / 4 prefix workgroups per CU (* the rule's), us: 256 x 1 rows, 4096 + 600
// keys, 32 / 8 heads of 64: 54* / 59 / 67, of 128: 93* / 107 / 125; 64 x 8 rows, 2000 +
// 2000 keys: 57* / 63 / 72; 16384 + 999 keys: 141 / 117* / 110, with 40 / 8 heads of 128:
// 360 / 225* / 236; 16 x 4 rows, 32768 + 500: 42 / 40* / 46.  Four gain only in the one
// of these shapes.
//
// Lengths are device data, so the plan takes the page table's width for the
// suffixes' length.  A table much wider than the sequences costs a small batch the
// direct form and fills its splits with nothing (one sequence of 500 + 37 keys: a
// table of 3 pages of 16 6.1 us, 256 pages 8.0, 2048 pages 13.6); 64 and 256
// sequences measure the same at any width.
CachedPlan cached_plan(int D, int Hq, int Hkv, int N, int L, int prefix_len, int max_keys) {
    CachedPlan p;
    const int G = Hq / Hkv;
    const int64_t rows = (int64_t)N * L * G;
    const int64_t row_blocks = (rows + kCRows - 1) / kCRows;
    const int64_t base = (int64_t)N * ((L * G + 31) / 32) * Hkv;
    p.prefix_splits = 0;
    p.prefix_chunk = 0;
    p.prefix_blocks = 0;
    const int KT = 4096 / D;
    const int64_t rounds = ((prefix_len + KT - 1) / KT + (max_keys + KT - 1) / KT + kDirectW - 1) / kDirectW;
    p.direct = base <= 256 && rounds <= 2;
    if (p.direct) {
        p.suffix_splits = 0;
        p.suffix_blocks = base;
        return p;
    }
    if (prefix_len > 0) {
        const int tiles = (prefix_len + kPrefixTile - 1) / kPrefixTile;
        // seconds at 5e12 bytes/s and 8e14 flops/s; a batch fills about half of its page tables
        const double read = 2. * N * max_keys * Hkv * D / 5e12, product = 4. * rows * Hkv * D * prefix_len / 8e14;
        const int64_t want = (read > product ? 256 : 512) / (row_blocks * Hkv);
        const int splits = (int)(want < 1 ? 1 : want < tiles ? want : tiles);
        const int per = (tiles + splits - 1) / splits;
        p.prefix_chunk = per * kPrefixTile;
        p.prefix_splits = (tiles + per - 1) / per;
        p.prefix_blocks = row_blocks * Hkv * p.prefix_splits;
    }
    const int64_t per_wg = (int64_t)kCW * kOwnTile;
    const int64_t most = (max_keys + per_wg - 1) / per_wg, want = 1024 / base;
    p.suffix_splits = (int)(want < 1 ? 1 : want < most ? want : most);
    if (p.suffix_splits < 1) p.suffix_splits = 1;
    p.suffix_blocks = base * p.suffix_splits;
    return p;
}

template <int D>
static hipError_t launch_cached(const CachedArgs& a, const CachedPlan& p, hipStream_t s) {
    const int64_t blocks = p.prefix_blocks + p.suffix_blocks;
    const int64_t joins = p.prefix_splits + p.suffix_splits > 1 ? ((int64_t)a.N * a.L * a.Hq + 3) / 4 : 0;
    if (too_many(blocks, 64 * (p.direct ? kDirectW : kCW)) || too_many(joins, 256)) return hipErrorInvalidConfiguration;
    if (p.direct) {
        hipLaunchKernelGGL((attn_cached_direct_kernel<D>), dim3((uint32_t)blocks), dim3(64 * kDirectW), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((attn_cached_kernel<D>), dim3((uint32_t)blocks), dim3(64 * kCW), 0, s, a);
    if (joins > 0)
        hipLaunchKernelGGL((attn_join_kernel<D>), dim3((uint32_t)joins), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_attn_cached(CachedArgs a, int D, hipStream_t s) {
    const CachedPlan p = cached_plan(D, a.Hq, a.Hkv, a.N, a.L, a.prefix_len, a.max_pages << a.page_shift);
    a.prefix_splits = p.prefix_splits;
    a.prefix_chunk = p.prefix_chunk;
    a.prefix_blocks = p.prefix_blocks;
    a.suffix_splits = p.suffix_splits;
    return D == 64 ? launch_cached<64>(a, p, s) : launch_cached<128>(a, p, s);
}

}  // namespace lfm2sc
