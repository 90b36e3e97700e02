// attn_cached8.hpp -- attention of new tokens over a paged cache of 8-bit codes
// (lfm2sc_attn_cached8): the kernels, instantiated by attn_cached8_*.hip.
//
// With code ck, cv and scale ks, vs of a key's block of tokens,
//   score = scale ks (q . ck),  out = sum_j p_j vs_j cv_j / sum_j p_j.
// Decoding reads the whole cache once a step, so bytes bound it: codes stay 8 bits
// up to the registers, where they become bf16 operands (every code of either
// format is a bf16 value), the scale of a key multiplies its score, and that of a
// value its probability before p is rounded to bf16.  Sums and statistics are fp32.
//
// A wave takes 64 keys at a time.  Products run on v_mfma_f32_16x16x32_bf16; lane
// (c = lane & 15, g = lane >> 4) holds of the operands
//   A[m = c][k = 8 g + j],  B[k = 8 g + j][n = c],  j = 0..7,
// and of the result C[m = 4 g + i][n = c], i = 0..3.  Scores are S^T = K Q^T: row m
// of block t (of four) is key 16 (m >> 2) + 4 t + (m & 3), so that a lane ends up
// with the 16 neighbouring keys 16 g + 4 t + i of query row c, and two blocks,
// rounded, are at once the B operand of O^T += V^T P^T with k = 16 g + 8 u + j.  For
// its A operand the lane needs 16 neighbouring tokens of a channel: one 16-byte
// load of the V page.  K's k order is free as well: lane g takes bytes
// [D / 4 g, D / 4 (g + 1)) of a key's codes, and the query's operand the same.
// Nothing but the waves' join goes through LDS.
#pragma once

#include "attn_common.hpp"
#include "cache8.hpp"

namespace lfm2sc {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kC8Tile = 64;      // keys per tile

__device__ __forceinline__ f32x4 mfma16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 8 codes as bf16 values, exactly.
template <bool kInt8>
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t lo, uint32_t hi) {
    union { bf16x2 p[4]; uint32_t u[4]; bf16x8 v; } r;
    if constexpr (kInt8) {
        float f[8];
        decode4<true>(lo, f);
        decode4<true>(hi, f + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.u[i] = Elem<uint16_t>::pack2(f[2 * i], f[2 * i + 1]);
    } else {
        r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
        r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
        r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
        r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    }
    return r.v;
}

// Maximum and sum over the four lanes of a column (16 apart).
__device__ __forceinline__ float max_groups(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_groups(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// The value of lane i of the lane's row of 16.
template <int i>
__device__ __forceinline__ float row_lane(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + i, 0xf, 0xf, false));
}
template <int i = 0, typename F>
__device__ __forceinline__ void for_keys(F f) {
    if constexpr (i < 16) {
        f(IC<i>{});
        for_keys<i + 1>(f);
    }
}

// Codes and scales of a tile in a lane.
template <int D>
struct Tile8 {
    uint4 k[4][D / 64];      // block t: bytes D / 4 g .. of key 16 (c >> 2) + 4 t + (c & 3)
    uint4 v[D / 16];         // tokens 16 g .. 16 g + 15 of channel 16 b + c
    float ks, vs;            // kToken: of key 16 g + c; else of the 16 keys of g
};

// Where a wave's tiles lie: tile i of `first` prefix tiles, then the own ones.
struct Keys8 {
    const int32_t* prefix;   // page numbers
    const int32_t* own;
    int len;                 // own keys
    int p0, p1;              // prefix keys [p0, p1) of this workgroup, p0 a multiple of 64
    int ptiles;              // tiles of those
    int tile0;               // first own tile
};

template <int D, bool kInt8, bool kToken>
struct Loader8 {
    const Cached8Args& a;
    const Keys8& s;
    int kvh, lane;
    // a tile's first key, its part, and the keys of the part
    __device__ __forceinline__ bool is_prefix(int i) const { return i < s.ptiles; }
    __device__ __forceinline__ int first_key(int i) const {
        return i < s.ptiles ? s.p0 + i * kC8Tile : (s.tile0 + i - s.ptiles) * kC8Tile;
    }
    __device__ __forceinline__ int end_key(int i) const { return i < s.ptiles ? s.p1 : s.len; }
    // 16 tokens of a page: those of group x of tile i, or the last ones that exist
    __device__ __forceinline__ int group_key(int i, int x) const {
        return min(first_key(i) + 16 * x, (end_key(i) - 1) & ~15);
    }
    __device__ __forceinline__ int32_t page(int i, int x) const {
        return (is_prefix(i) ? s.prefix : s.own)[group_key(i, x) >> a.c.page_shift];
    }
    __device__ __forceinline__ int clamp_page(int32_t p) const { return min(max(p, 0), a.c.num_pages - 1); }
    __device__ __forceinline__ void load_k(Tile8<D>& t, int i, int32_t pk, int32_t pg) const {
        const int c = lane & 15, g = lane >> 4, S = 1 << a.c.page_shift;
        const int in = group_key(i, c >> 2) & (S - 1);
        const uint8_t* p = a.k + (int64_t)clamp_page(pk) * a.page_stride + ((int64_t)kvh * S + in + (c & 3)) * D + D / 4 * g;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) t.k[b][h] = *reinterpret_cast<const uint4*>(p + 4 * b * D + 16 * h);
        t.ks = scale(a.k_scales, i, pg);
    }
    __device__ __forceinline__ void load_v(Tile8<D>& t, int i, int32_t pg) const {
        const int c = lane & 15, g = lane >> 4, S = 1 << a.c.page_shift;
        const int in = group_key(i, g) & (S - 1);
        const uint8_t* p = a.v + (int64_t)clamp_page(pg) * a.page_stride + ((int64_t)kvh * S + in) * D + c * 16;
#pragma unroll
        for (int b = 0; b < D / 16; ++b) t.v[b] = *reinterpret_cast<const uint4*>(p + b * 256);
        t.vs = scale(a.v_scales, i, pg);
    }
    __device__ __forceinline__ float scale(const float* scales, int i, int32_t pg) const {
        const int c = lane & 15, g = lane >> 4, S = 1 << a.c.page_shift;
        const int in = (group_key(i, g) & (S - 1)) + (kToken ? c : 0);
        return scales[(int64_t)clamp_page(pg) * a.scale_stride + (((int64_t)kvh * S + in) >> a.block_shift)];
    }
};

// Running softmax state of 16 NT query rows (row 16 n + c): reference m, sum l
// (of the lane's own keys) and output o, relative to 2^m.
template <int D, int NT>
struct Rows8 {
    float m[NT], l[NT];
    f32x4 o[NT][D / 16];
    __device__ void clear() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = kNegInf;
            l[n] = 0.f;
#pragma unroll
            for (int b = 0; b < D / 16; ++b) o[n][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
};

// One tile against the wave's rows.  masked (uniform): keys numbered seen[n] + 1 and
// on within the tile are masked, and keys from `end` on do not exist: their codes
// and scales may be anything.
template <int D, int NT, bool kInt8, bool kToken, typename F1, typename F2>
__device__ __forceinline__ void attend8(Rows8<D, NT>& r, const bf16x8 (&q)[NT][D / 32], Tile8<D>& t, float cs, bool masked,
                                        const int (&seen)[NT], int end, int lane, F1 after_k, F2 after_v) {
    const int g = lane >> 4;
    f32x4 s[NT][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        bf16x8 k[D / 32];
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            k[2 * h] = codes_to_bf16<kInt8>(t.k[b][h].x, t.k[b][h].y);
            k[2 * h + 1] = codes_to_bf16<kInt8>(t.k[b][h].z, t.k[b][h].w);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            s[n][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int d = 0; d < D / 32; ++d) s[n][b] = mfma16(k[d], q[n][d], s[n][b]);
        }
    }
    float ks = t.ks * cs, vs = t.vs;
    after_k();
    if (masked) {
        const int at = 16 * g + (kToken ? lane & 15 : 0);
        if (at >= end) ks = vs = 0.f;
        if constexpr (!kInt8) {
            // codes of tokens that do not exist: a NaN among them would outlive its probability of 0
            const int have = min(max(end - 16 * g, 0), 16);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int bytes = min(max(have - 4 * w, 0), 4);
                const uint32_t m = bytes == 4 ? 0xffffffffu : (1u << (8 * bytes)) - 1u;
#pragma unroll
                for (int b = 0; b < D / 16; ++b) (&t.v[b].x)[w] &= m;
            }
        }
    }
    bf16x8 p[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float x[16];
        for_keys([&](auto i) {
            constexpr int e = decltype(i)::value;
            if constexpr (kToken) x[e] = s[n][e >> 2][e & 3] * row_lane<e>(ks);
            else x[e] = s[n][e >> 2][e & 3];
        });
        if (masked) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (16 * g + e > seen[n]) x[e] = kNegInf;
        }
        float mx = x[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) mx = fmaxf(mx, x[e]);
        // a masked lane's scale may be 0, and 0 times -inf is no maximum
        const float mn = max_groups(kToken ? mx : mx == kNegInf ? kNegInf : mx * ks);
        if (__any(mn > r.m[n] + kLazy)) {
            const float m = fmaxf(r.m[n], mn), alpha = exp2_fast(r.m[n] - (m == kNegInf ? 0.f : m));
            r.m[n] = m;
            r.l[n] *= alpha;
#pragma unroll
            for (int b = 0; b < D / 16; ++b) r.o[n][b] *= alpha;
        }
        const float ref = r.m[n] == kNegInf ? 0.f : r.m[n];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if constexpr (kToken) x[e] = exp2_fast(x[e] - ref);
            else x[e] = masked && x[e] == kNegInf ? 0.f : exp2_fast(__builtin_fmaf(x[e], ks, -ref));
            sum += x[e];
        }
        r.l[n] += sum;
        for_keys([&](auto i) {
            constexpr int e = decltype(i)::value;
            if constexpr (kToken) x[e] *= row_lane<e>(vs);
            else x[e] *= vs;
        });
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            union { uint32_t w[4]; bf16x8 v; } y;
#pragma unroll
            for (int j = 0; j < 4; ++j) y.w[j] = Elem<uint16_t>::pack2(x[8 * u + 2 * j], x[8 * u + 2 * j + 1]);
            p[n][u] = y.v;
        }
    }
#pragma unroll
    for (int b = 0; b < D / 16; ++b) {
        const bf16x8 v0 = codes_to_bf16<kInt8>(t.v[b].x, t.v[b].y), v1 = codes_to_bf16<kInt8>(t.v[b].z, t.v[b].w);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            r.o[n][b] = mfma16(v0, p[n][0], r.o[n][b]);
            r.o[n][b] = mfma16(v1, p[n][1], r.o[n][b]);
        }
    }
    after_v();
}

// Tiles mine, mine + step, .. < tiles of the workgroup's list.  The next tile's K
// is loaded as soon as the scores are formed, its V after the products, its page
// numbers a tile earlier.
template <int D, int NT, bool kInt8, bool kToken>
__device__ __forceinline__ void walk8(Rows8<D, NT>& r, const bf16x8 (&q)[NT][D / 32], const Cached8Args& a, const Keys8& s,
                                      int kvh, int tiles, int mine, int step, const int (&last)[NT], int least, int lane) {
    if (mine >= tiles) return;
    const int c = lane & 15, g = lane >> 4;
    const Loader8<D, kInt8, kToken> ld{a, s, kvh, lane};
    const float cs = a.c.scale * kLog2e;
    Tile8<D> t;
    int32_t pk = ld.page(mine, c >> 2), pg = ld.page(mine, g);
    ld.load_k(t, mine, pk, pg);
    ld.load_v(t, mine, pg);
    int32_t nk = 0, ng = 0;
    if (mine + step < tiles) {
        nk = ld.page(mine + step, c >> 2);
        ng = ld.page(mine + step, g);
    }
    for (int i = mine; i < tiles; i += step) {
        const bool prefix = ld.is_prefix(i);
        const int k0 = ld.first_key(i), end = ld.end_key(i) - k0;
        int seen[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) seen[n] = prefix ? end - 1 : last[n] - k0;
        const bool masked = prefix ? end < kC8Tile : k0 + kC8Tile - 1 > least;
        const int next = i + step;
        auto after_k = [&] {
            if (next >= tiles) return;
            pk = nk;
            pg = ng;
            const int then = min(next + step, tiles - 1);
            nk = ld.page(then, c >> 2);
            ng = ld.page(then, g);
            ld.load_k(t, next, pk, pg);
        };
        auto after_v = [&] {
            if (next < tiles) ld.load_v(t, next, pg);
        };
        attend8<D, NT, kInt8, kToken>(r, q, t, cs, masked, seen, end, lane, after_k, after_v);
    }
}

// The B operand of a query row: values D / 4 g + 8 s .. of step s; zeros where there is no row.
template <int D>
__device__ __forceinline__ void load_query8(bf16x8 (&f)[D / 32], const uint16_t* row, int g, bool exists) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (exists) x = *reinterpret_cast<const uint4*>(row + D / 4 * g + 8 * s);
        f[s] = __builtin_bit_cast(bf16x8, x);
    }
}

// A workgroup: 16 NT query rows of one key/value head against some of the keys.
// Own keys: rows of one sequence; prefix: rows of any.  The waves deal the tiles
// out among themselves and join through LDS, in halves.
template <int D, int NT, bool kInt8, bool kToken, int W>
__device__ __forceinline__ void keys8(const Cached8Args& a, const Keys8& s, int kvh, int64_t x0, int64_t rows, int len, int tiles,
                                      int split, bool whole, float* lds, int wave, int lane) {
    constexpr int kWaveF = NT * (D / 4 + 2) * 64;        // floats of a wave's state
    const CachedArgs& ca = a.c;
    const int c = lane & 15, g = lane >> 4, G = ca.Hq / ca.Hkv;
    int64_t token[NT];
    int head[NT], last[NT], least = 1 << 30;
    bool exists[NT];
    bf16x8 q[NT][D / 32];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int64_t x = min(x0 + 16 * n + c, rows - 1);
        exists[n] = x0 + 16 * n + c < rows;
        token[n] = x / G;
        head[n] = kvh * G + (int)(x % G);
        last[n] = len - ca.L + (int)(token[n] % ca.L);   // the row's last own key
        load_query8<D>(q[n], ca.q + token[n] * ca.q_stride + (int64_t)head[n] * D, g, exists[n]);
    }
    least = len - ca.L;
    Rows8<D, NT> r;
    r.clear();
    walk8<D, NT, kInt8, kToken>(r, q, a, s, kvh, tiles, wave, W, last, least, lane);
#pragma unroll
    for (int n = 0; n < NT; ++n) r.l[n] = sum_groups(r.l[n]);
#pragma unroll
    for (int half = W / 2; half >= 1; half >>= 1) {
        float* mine = lds + (wave % half) * kWaveF;
        if (half < W / 2) lds_barrier();                 // the last round's states are read
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int b = 0; b < D / 16; ++b)
                    *reinterpret_cast<f32x4*>(mine + ((n * (D / 16) + b) * 64 + lane) * 4) = r.o[n][b];
                mine[NT * D / 4 * 64 + (2 * n) * 64 + lane] = r.m[n];
                mine[NT * D / 4 * 64 + (2 * n + 1) * 64 + lane] = r.l[n];
            }
        }
        lds_barrier();
        if (wave < half) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float m2 = mine[NT * D / 4 * 64 + (2 * n) * 64 + lane], l2 = mine[NT * D / 4 * 64 + (2 * n + 1) * 64 + lane];
                const float m = fmaxf(r.m[n], m2), ref = m == kNegInf ? 0.f : m;
                const float f1 = exp2_fast(r.m[n] - ref), f2 = exp2_fast(m2 - ref);
                r.m[n] = m;
                r.l[n] = r.l[n] * f1 + l2 * f2;
#pragma unroll
                for (int b = 0; b < D / 16; ++b)
                    r.o[n][b] = r.o[n][b] * f1 + *reinterpret_cast<const f32x4*>(mine + ((n * (D / 16) + b) * 64 + lane) * 4) * f2;
            }
        }
    }
    if (wave != 0) return;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (!exists[n]) continue;
        if (whole) {
            // no visible key: 0; a NaN stays
            const float inv = r.l[n] > 0.f ? 1.f / r.l[n] : (r.l[n] == 0.f ? 0.f : r.l[n]);
            uint16_t* o = ca.out + token[n] * ca.out_stride + (int64_t)head[n] * D + 4 * g;
#pragma unroll
            for (int b = 0; b < D / 16; ++b)
                *reinterpret_cast<uint2*>(o + 16 * b) =
                    make_uint2(Elem<uint16_t>::pack2(r.o[n][b][0] * inv, r.o[n][b][1] * inv),
                               Elem<uint16_t>::pack2(r.o[n][b][2] * inv, r.o[n][b][3] * inv));
        } else {
            const int64_t at = ((int64_t)split * ca.N * ca.L + token[n]) * ca.Hq + head[n];
#pragma unroll
            for (int b = 0; b < D / 16; ++b) *reinterpret_cast<f32x4*>(ca.part_o + at * D + 16 * b + 4 * g) = r.o[n][b];
            if (g == 0) *reinterpret_cast<float2*>(ca.part_ml + at * 2) = make_float2(r.m[n], r.l[n]);
        }
    }
}

// Split form (direct = false): the prefix's workgroups first, then the suffixes'.
// Direct form: a workgroup reads prefix and suffix and writes the output.
template <int D, int NT, bool kInt8, bool kToken, int W>
__global__ __launch_bounds__(64 * W) void attn_cached8_kernel(Cached8Args a, bool direct) {
    __shared__ __attribute__((aligned(16))) float lds[W / 2 * NT * (D / 4 + 2) * 64];
    const CachedArgs& ca = a.c;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int G = ca.Hq / ca.Hkv, prefix_blocks = (int)ca.prefix_blocks;
    int block = blockIdx.x;
    Keys8 s;
    s.prefix = ca.prefix_pages;
    if (block < prefix_blocks) {
        const int kvh = block % ca.Hkv, rest = block / ca.Hkv, split = rest % ca.prefix_splits;
        s.own = nullptr;
        s.len = 0;
        s.p0 = split * ca.prefix_chunk;
        s.p1 = min(s.p0 + ca.prefix_chunk, ca.prefix_len);
        s.ptiles = (s.p1 - s.p0 + kC8Tile - 1) / kC8Tile;
        s.tile0 = 0;
        keys8<D, NT, kInt8, kToken, W>(a, s, kvh, (int64_t)(rest / ca.prefix_splits) * 16 * NT, (int64_t)ca.N * ca.L * G, 0,
                                       s.ptiles, split, false, lds, wave, lane);
        return;
    }
    block -= prefix_blocks;
    const int kvh = block % ca.Hkv;
    int rest = block / ca.Hkv;
    const int splits = direct ? 1 : ca.suffix_splits, split = rest % splits;
    rest /= splits;
    const int blocks = (ca.L * G + 16 * NT - 1) / (16 * NT);
    const int seq = rest / blocks, rb = rest % blocks;
    s.own = ca.page_table + (int64_t)seq * ca.max_pages;
    s.len = min(max(ca.suffix_len[seq], 0), a.max_suffix);
    s.p0 = 0;
    s.p1 = direct ? ca.prefix_len : 0;
    s.ptiles = (s.p1 + kC8Tile - 1) / kC8Tile;
    const int all = (s.len + kC8Tile - 1) / kC8Tile, per = (all + splits - 1) / splits;
    const int t0 = min(split * per, all), t1 = min(t0 + per, all);
    s.tile0 = t0;
    keys8<D, NT, kInt8, kToken, W>(a, s, kvh, (int64_t)seq * ca.L * G + (int64_t)rb * 16 * NT, (int64_t)(seq + 1) * ca.L * G, s.len,
                                   s.ptiles + t1 - t0, ca.prefix_splits + split, direct || ca.prefix_splits + splits == 1, lds, wave,
                                   lane);
}

constexpr int kC8Waves = 4, kC8DirectWaves = 8;
inline int cached8_row_tiles(int L, int G) { return (int64_t)L * G <= 16 ? 1 : 2; }

// Defined in the file of its format and head dimension.
template <int D, bool kInt8>
hipError_t launch_cached8(const Cached8Args& a, bool direct, int64_t blocks, hipStream_t s);

#ifdef LFM2SC_CACHED8_D
template <int D, bool kInt8>
hipError_t launch_cached8(const Cached8Args& a, bool direct, int64_t blocks, hipStream_t s) {
    const int nt = cached8_row_tiles(a.c.L, a.c.Hq / a.c.Hkv);
    auto go = [&](auto n, auto token) {
        constexpr int NT = decltype(n)::value;
        constexpr bool kToken = decltype(token)::value;
        if (direct)
            hipLaunchKernelGGL((attn_cached8_kernel<D, NT, kInt8, kToken, kC8DirectWaves>), dim3((uint32_t)blocks),
                               dim3(64 * kC8DirectWaves), 0, s, a, true);
        else
            hipLaunchKernelGGL((attn_cached8_kernel<D, NT, kInt8, kToken, kC8Waves>), dim3((uint32_t)blocks), dim3(64 * kC8Waves), 0,
                               s, a, false);
    };
    auto by_rows = [&](auto token) {
        if (nt == 1) go(IC<1>{}, token);
        else go(IC<2>{}, token);
    };
    if (a.block_shift == 0) by_rows(std::true_type{});
    else by_rows(std::false_type{});
    return hipGetLastError();
}
template hipError_t launch_cached8<LFM2SC_CACHED8_D, LFM2SC_CACHED8_INT8>(const Cached8Args&, bool, int64_t, hipStream_t);
#endif

}  // namespace lfm2sc
