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
// Where a wave reads tiles for its own rows, nothing but the waves' join goes through
// LDS; a prefix of many rows is staged there as operands (shared8).
//
// Measured (one MI355X, device time): 64 sequences of up to 16384 keys, 24/8 heads of
// 128, a scale a token: 212 us for 1.13 GB, 5.3 TB/s (1 GiB copies reach 5.1): reads
// bound it.  256 sequences of up to 600 (2000) keys behind no prefix, 32/8 heads of 64:
// 19.4 (61) us for 17 (51) at the copy's rate.  One user, 500 + 37 keys: 5.2 us, a chain
// of four dependent reads.  Three waves a SIMD for D = 128, with the registers that
// leaves, took 262 us instead of 217 (64 x 16384).
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

// Maximum over the four lanes of a column (16 apart).
__device__ __forceinline__ float max_groups(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
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

// Addresses of a tile.  A tile begins at a multiple of 64 keys, so its offset in a
// page is uniform (0 in pages of up to 64 tokens), and a lane's 16 tokens lie at the
// same distance from it in every tile: an address is a constant of the lane, one
// product with a page number and the uniform offset.  No branch on the page size:
// the loads in flight are then counted exactly, unless the form spills registers
// (form_per_simd).  Tokens past the end are read from the last page that exists.
template <int D, bool kToken>
struct Loader8 {
    const Cached8Args& a;
    const Keys8& s;
    int lane, shift;
    const uint8_t *k, *v;    // the lane's place in page 0
    const float *ks, *vs;
    __device__ __forceinline__ Loader8(const Cached8Args& a_, const Keys8& s_, int kvh, int lane_) : a(a_), s(s_), lane(lane_) {
        const int c = lane & 15, g = lane >> 4;
        shift = a.c.page_shift;
        const int S = 1 << shift, kin = (16 * key_group()) & (S - 1), vin = (16 * g) & (S - 1);
        k = a.k + (kvh * S + kin + (c & 3)) * D + D / 4 * g;
        v = a.v + (kvh * S + vin) * D + c * 16;
        const int at = (kvh * S + vin + (kToken ? c : 0)) >> a.block_shift;
        ks = a.k_scales + at;
        vs = a.v_scales + at;
    }
    // a tile's first key, its part, and the keys of the part
    __device__ __forceinline__ bool is_prefix(int i) const { return i < s.ptiles; }
    __device__ __forceinline__ int first_key(int i) const {
        return i < s.ptiles ? s.p0 + i * kC8Tile : (s.tile0 + i - s.ptiles) * kC8Tile;
    }
    __device__ __forceinline__ int end_key(int i) const { return i < s.ptiles ? s.p1 : s.len; }
    // groups of 16 tokens of the tile: of the lane's keys, of its values
    __device__ __forceinline__ int key_group() const { return (lane & 15) >> 2; }
    __device__ __forceinline__ int value_group() const { return lane >> 4; }
    // page numbers: of the lane's keys, of its values
    __device__ __forceinline__ int32_t key_page(int i) const { return page(i, key_group()); }
    __device__ __forceinline__ int32_t value_page(int i) const { return page(i, value_group()); }
    __device__ __forceinline__ int32_t page(int i, int group) const {
        const int32_t* table = is_prefix(i) ? s.prefix : s.own;
        return table[(uint32_t)min((first_key(i) + 16 * group) >> shift, (end_key(i) - 1) >> shift)];
    }
    __device__ __forceinline__ uint32_t in_page(int i) const { return (uint32_t)(first_key(i) & ((1 << shift) - 1)); }
    __device__ __forceinline__ uint64_t in_pool(int32_t p) const { return (uint32_t)min(max(p, 0), a.c.num_pages - 1); }
    __device__ __forceinline__ const uint8_t* key_at(int i, int32_t p) const {
        return k + in_pool(p) * (uint32_t)a.page_stride + in_page(i) * D;
    }
    __device__ __forceinline__ const uint8_t* value_at(int i, int32_t p) const {
        return v + in_pool(p) * (uint32_t)a.page_stride + in_page(i) * D;
    }
    __device__ __forceinline__ void load_k(Tile8<D>& t, int i, int32_t pk) const {
        const uint8_t* p = key_at(i, pk);
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) t.k[b][h] = *reinterpret_cast<const uint4*>(p + 4 * b * D + 16 * h);
    }
    __device__ __forceinline__ void load_v(Tile8<D>& t, int i, int32_t pv) const {
        const uint8_t* p = value_at(i, pv);
#pragma unroll
        for (int b = 0; b < D / 16; ++b) t.v[b] = *reinterpret_cast<const uint4*>(p + b * 256);
    }
    __device__ __forceinline__ void load_scales(float& k1, float& v1, int i, int32_t pv) const {
        // The offset, a multiple of 64, and the lane's tokens below 64 do not carry into each other's part of the block number.
        const uint64_t at = in_pool(pv) * (uint32_t)a.scale_stride + (in_page(i) >> a.block_shift);
        k1 = ks[at];
        v1 = vs[at];
    }
};

// Running softmax state of 16 NT query rows (row 16 n + c): reference m, sum l and
// output o, relative to 2^m.  l is a result of the matrix unit like o, with 1 / vs in
// place of a channel's code (rows 0 and 1: its two bf16 parts, 2^-17 of it off),
// because p carries vs: so it adds up the very p that o does, rounded, which takes
// most of that rounding out of o / l (1.9e-3 of an output off, 2.4e-3 with a sum of
// unrounded p), and costs nothing of the vector unit, which bounds the kernel where
// many rows share a tile.
template <int D, int NT>
struct Rows8 {
    float m[NT];
    f32x4 l[NT], o[NT][D / 16];
    __device__ void clear() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = kNegInf;
            l[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < D / 16; ++b) o[n][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
    // the row's sum, in all of its lanes
    __device__ __forceinline__ float sum(int n) const { return __shfl(l[n][0] + l[n][1], threadIdx.x & 15, 64); }
};

// Scales as the kernels take them.  A scale below 2^-100 (0: a block of zeros)
// counts as 2^-100, so that its logarithm and reciprocal exist, and its product with
// the scale of scores as at least 2^-126, as 0 times a masked score of -inf would be a
// NaN; a NaN stays.
__device__ __forceinline__ float at_least(float least, float x) { return x < least ? least : x; }
__device__ __forceinline__ float usable(float scale) { return at_least(kMinScale, scale); }

// Few tiles are masked: what only they need is a branch of its own, not selects in
// every tile (30 instructions of each row tile's 150).
__device__ __forceinline__ void masked_side() { asm volatile("; masked" ::: "memory"); }

// Keys that do not exist, from `end` on within the tile: no scale, and (e4m3, where
// they are in registers) zeros for their values' codes: a NaN among them would
// outlive its probability of 0.
template <bool kToken>
__device__ __forceinline__ void drop_scales(float& ks, float& vs, int end, int lane) {
    if (16 * (lane >> 4) + (kToken ? lane & 15 : 0) >= end) ks = vs = 1.f;
}
__device__ __forceinline__ void drop_codes(uint4& v, int have) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int bytes = min(max(have - 4 * w, 0), 4);
        (&v.x)[w] &= bytes == 4 ? 0xffffffffu : (1u << (8 * bytes)) - 1u;
    }
}

// The scales of a tile in a lane: of its keys' scores (times scale log2 e) and
// values; kToken: of key 16 g + c, else of the 16 keys of g.
template <bool kToken>
struct Scales8 {
    float k, v;
    float log_v;                 // not kToken: log2 v,
    uint32_t one;                // and two values of the operand of l
    __device__ __forceinline__ void set(float ks, float vs, float cs, bool masked, int end, int lane) {
        if (masked) drop_scales<kToken>(ks, vs, end, lane);
        k = at_least(__FLT_MIN__, usable(ks) * cs);
        v = usable(vs);
        if constexpr (!kToken) {
            log_v = __builtin_amdgcn_logf(v);
            const float r = __builtin_amdgcn_rcpf(v), hi = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
            const int c = lane & 15;
            one = c < 2 ? Elem<uint16_t>::pack2(c ? r - hi : hi, c ? r - hi : hi) : 0u;
        }
    }
};

// The scores of a tile, s[t][i] of key 16 g + 4 t + i: the rows' maxima, times log2 e,
// of row tile n.  masked (uniform): keys numbered above `seen` within the tile are
// -inf from here on.
template <int NT, bool kToken>
__device__ __forceinline__ float peak8(f32x4 (&s)[NT][4], int n, const Scales8<kToken>& sc, bool masked, int seen, int g) {
    if constexpr (kToken)
        for_keys([&](auto i) {
            constexpr int e = decltype(i)::value;
            s[n][e >> 2][e & 3] *= row_lane<e>(sc.k);
        });
    if (masked) {
        masked_side();
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (16 * g + e > seen) s[n][e >> 2][e & 3] = kNegInf;
    }
    float mx = s[n][0][0];
#pragma unroll
    for (int e = 1; e < 16; ++e) mx = fmaxf(mx, s[n][e >> 2][e & 3]);
    return max_groups(kToken ? mx : mx * sc.k);
}

// The rows' reference moves where a maximum passes it by 2^kLazy.
template <int D, int NT>
__device__ __forceinline__ void refer8(Rows8<D, NT>& r, const float (&mn)[NT]) {
    bool move = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) move |= mn[n] > r.m[n] + kLazy;
    if (__any(move)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float m = mn[n] > r.m[n] + kLazy ? mn[n] : r.m[n];
            const float alpha = exp2_fast(r.m[n] - (m == kNegInf ? 0.f : m));
            r.m[n] = m;
            r.l[n] *= alpha;
#pragma unroll
            for (int b = 0; b < D / 16; ++b) r.o[n][b] *= alpha;
        }
    }
}

// Then the scores of block b become probabilities times their values' scales, words
// 2 (b & 1) and + 1 of operand b >> 1 of the second product.  They are rounded to
// bf16 because that is what the matrix unit multiplies: an output is then 1.8e-3 to
// 2.0e-3 off in the 2-norm, where its own rounding is 1.6e-3; what is left of p as a
// second operand would double the second product.  between() runs when the scores
// have been read.
template <int b, int D, int NT, bool kToken, typename F>
__device__ __forceinline__ void weigh8(Rows8<D, NT>& r, f32x4 (&s)[NT][4], bf16x8 (&p)[NT][2], const Scales8<kToken>& sc, F between) {
    float x[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float ref = r.m[n] == kNegInf ? 0.f : r.m[n], at = kToken ? -ref : sc.log_v - ref;
#pragma unroll
        for (int i = 0; i < 4; ++i)              // else: p vs = 2^(score - ref + log2 vs)
            x[n][i] = kToken ? s[n][b][i] + at : __builtin_fmaf(s[n][b][i], sc.k, at);
    }
    between();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = exp2_fast(x[n][i]);
        if constexpr (kToken) {
            x[n][0] *= row_lane<4 * b>(sc.v);
            x[n][1] *= row_lane<4 * b + 1>(sc.v);
            x[n][2] *= row_lane<4 * b + 2>(sc.v);
            x[n][3] *= row_lane<4 * b + 3>(sc.v);
        }
        union { uint32_t w[4]; bf16x8 v; } y;
        y.v = p[n][b >> 1];
        y.w[2 * (b & 1)] = Elem<uint16_t>::pack2(x[n][0], x[n][1]);
        y.w[2 * (b & 1) + 1] = Elem<uint16_t>::pack2(x[n][2], x[n][3]);
        p[n][b >> 1] = y.v;
    }
}

// Adds a tile's p to the rows' sums.  The operand: 1 / v of keys 16 g + 8 u + j, of
// which row 0 (lanes c = 0) holds the upper 8 digits and row 1 the next, the others 0.
template <int D, int NT, bool kToken>
__device__ __forceinline__ void sum8(Rows8<D, NT>& r, const bf16x8 (&p)[NT][2], const Scales8<kToken>& sc, int lane) {
    bf16x8 x[2];
    if constexpr (kToken) {
        const float one = __builtin_amdgcn_rcpf(sc.v), hi = __uint_as_float(__float_as_uint(one) & 0xffff0000u);
        const int c = lane & 15;
        const float both = __uint_as_float(__float_as_uint(hi) | bf16_bits(one - hi));       // of key 16 g + c
        const uint32_t pick = c == 0 ? 0x07060302u : c == 1 ? 0x05040100u : 0x0c0c0c0cu;     // halves of two keys', or zeros
        uint32_t w[8];
        for_keys([&](auto i) {
            constexpr int e = decltype(i)::value;
            if constexpr (e % 2 == 0)
                w[e / 2] = __builtin_amdgcn_perm(__float_as_uint(row_lane<(e + 1) % 16>(both)), __float_as_uint(row_lane<e>(both)), pick);
        });
        x[0] = __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
        x[1] = __builtin_bit_cast(bf16x8, make_uint4(w[4], w[5], w[6], w[7]));
    } else {
        x[0] = x[1] = __builtin_bit_cast(bf16x8, make_uint4(sc.one, sc.one, sc.one, sc.one));
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) r.l[n] = mfma16(x[u], p[n][u], r.l[n]);
}

// One tile, in registers, against the wave's rows.
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
    Scales8<kToken> sc;
    sc.set(t.ks, t.vs, cs, masked, end, lane);
    after_k();
    if (!kInt8 && masked) {
        masked_side();
#pragma unroll
        for (int b = 0; b < D / 16; ++b) drop_codes(t.v[b], end - 16 * g);
    }
    float mn[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) mn[n] = peak8(s, n, sc, masked, seen[n], g);
    refer8(r, mn);
    bf16x8 p[NT][2];
    weigh8<0>(r, s, p, sc, [] {});
    weigh8<1>(r, s, p, sc, [] {});
    weigh8<2>(r, s, p, sc, [] {});
    weigh8<3>(r, s, p, sc, [] {});
    sum8(r, p, sc, lane);
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
    const Loader8<D, kToken> ld(a, s, kvh, lane);
    const float cs = a.c.scale * kLog2e;
    Tile8<D> t;
    int32_t nk = ld.key_page(mine), nv = ld.value_page(mine);        // page numbers of the tile that is loaded next
    ld.load_k(t, mine, nk);
    ld.load_scales(t.ks, t.vs, mine, nv);
    ld.load_v(t, mine, nv);
    if (mine + step < tiles) {
        nk = ld.key_page(mine + step);
        nv = ld.value_page(mine + step);
    }
    for (int i = mine; i < tiles; i += step) {
        const bool prefix = ld.is_prefix(i);
        const int k0 = ld.first_key(i), end = ld.end_key(i) - k0;
        int seen[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) seen[n] = prefix ? end - 1 : last[n] - k0;
        const int next = i + step;
        auto after_k = [&] {
            if (next >= tiles) return;
            ld.load_k(t, next, nk);
            nk = ld.key_page(min(next + step, tiles - 1));
            ld.load_scales(t.ks, t.vs, next, nv);
        };
        auto after_v = [&] {
            if (next >= tiles) return;
            ld.load_v(t, next, nv);
            nv = ld.value_page(min(next + step, tiles - 1));
        };
        const bool masked = prefix ? end < kC8Tile : k0 + kC8Tile - 1 > least;
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

// Query row x of a key/value head: x = (token row) * G + head in the group.
struct Query8 {
    int token, head;
    bool exists;
};
__device__ __forceinline__ Query8 query8(const CachedArgs& a, int kvh, int x, int rows) {
    const int G = a.Hq / a.Hkv, y = max(min(x, rows - 1), 0);
    return Query8{y / G, kvh * G + y % G, x < rows};
}

// Writes the output (whole) of the rows x0 + 16 n + c, or their state to split
// `split` of the workspace.
template <int D, int NT>
__device__ __forceinline__ void store8(const CachedArgs& a, const Rows8<D, NT>& r, const float (&l)[NT], int kvh, int x0,
                                       int rows, int split, bool whole, int lane) {
    const int c = lane & 15, g = lane >> 4;
    asm volatile("" : "+s"(x0));                         // worked out here, not kept in registers through the loop
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const Query8 y = query8(a, kvh, x0 + 16 * n + c, rows);
        if (!y.exists) continue;
        if (whole) {
            // no visible key: 0; a NaN stays
            const float inv = l[n] > 0.f ? 1.f / l[n] : (l[n] == 0.f ? 0.f : l[n]);
            uint16_t* o = a.out + y.token * a.out_stride + y.head * D + 4 * g;
#pragma unroll
            for (int b = 0; b < D / 16; ++b)
                *reinterpret_cast<uint2*>(o + 16 * b) =
                    make_uint2(Elem<uint16_t>::pack2(r.o[n][b][0] * inv, r.o[n][b][1] * inv),
                               Elem<uint16_t>::pack2(r.o[n][b][2] * inv, r.o[n][b][3] * inv));
        } else {
            const int64_t at = ((int64_t)split * a.N * a.L + y.token) * a.Hq + y.head;
#pragma unroll
            for (int b = 0; b < D / 16; ++b) *reinterpret_cast<f32x4*>(a.part_o + at * D + 16 * b + 4 * g) = r.o[n][b];
            if (g == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(r.m[n], l[n]);
        }
    }
}

// U waves: 16 NT query rows of one key/value head against some of the keys.  Own
// keys: rows of one sequence; prefix: rows of any.  The waves deal the tiles out
// among themselves and join through LDS, in halves.  All waves of the workgroup
// come here together.
template <int D, int NT>
constexpr int join_floats() { return NT * (D / 4 + 2) * 64; }      // a wave's state
template <int D, int NT, bool kInt8, bool kToken, int U>
__device__ __forceinline__ void keys8(const Cached8Args& a, const Keys8& s, int kvh, int x0, int rows, int len, int tiles, int split,
                                      bool whole, float* lds, int wave, int lane) {
    const CachedArgs& ca = a.c;
    bf16x8 q[NT][D / 32];
    int last[NT];                                        // the row's last own key
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const Query8 y = query8(ca, kvh, x0 + 16 * n + (lane & 15), rows);
        load_query8<D>(q[n], ca.q + y.token * ca.q_stride + y.head * D, lane >> 4, y.exists);
        last[n] = len - ca.L + y.token % ca.L;
    }
    Rows8<D, NT> r;
    r.clear();
    walk8<D, NT, kInt8, kToken>(r, q, a, s, kvh, tiles, wave, U, last, len - ca.L, lane);
    float l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) l[n] = r.sum(n);
#pragma unroll
    for (int half = U / 2; half >= 1; half >>= 1) {
        float* mine = lds + (wave % half) * join_floats<D, NT>();
        if (half < U / 2) lds_barrier();                 // the last round's states are read
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int b = 0; b < D / 16; ++b)
                    *reinterpret_cast<f32x4*>(mine + ((n * (D / 16) + b) * 64 + lane) * 4) = r.o[n][b];
                mine[NT * D / 4 * 64 + (2 * n) * 64 + lane] = r.m[n];
                mine[NT * D / 4 * 64 + (2 * n + 1) * 64 + lane] = l[n];
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
                l[n] = l[n] * f1 + l2 * f2;
#pragma unroll
                for (int b = 0; b < D / 16; ++b)
                    r.o[n][b] = r.o[n][b] * f1 + *reinterpret_cast<const f32x4*>(mine + ((n * (D / 16) + b) * 64 + lane) * 4) * f2;
            }
        }
    }
    if (wave == 0) store8<D, NT>(ca, r, l, kvh, x0, rows, split, whole, lane);
}

// Prefix keys for many rows: 4 waves of 32 query rows share each tile.  They turn
// its codes into bf16 operands once, in LDS in the order in which the products
// read them (operand, lane: 16 bytes each, no bank conflict), two buffers of K and
// of V, one barrier a tile.  With two or three waves a SIMD the vector unit has to
// work beside the matrix unit within a wave: between two barriers the scores of tile i
// turn into p while those of tile i + 1 are formed, and the codes of K in tile
// i + 2 and of V in tile i + 1 are staged while p V is added up.
//
// 64 x 8 rows of 5 heads of 128 behind 16384 keys (a whole library product of that many
// flops: 131 us): 194 us with the join (10 us), 185 for e4m3; with suffixes of up to 999
// keys 210 and 196.  A tile takes two waves of a SIMD 2000 cycles each: 1090 of matrix
// and 1540 of vector instructions, which overlap in part.  Left out one at a time: code
// conversion -27 us, loads -22, half of p V -21, exponentials -8, reads of LDS -1 to -4;
// zeros for data -18 (power).  Not kept: 32 x 32 x 16 products (218 us with suffixes: their
// vector work hides better by itself, 1.5 cycles of 8 against 4, but not here), and K's codes
// read as runs of memory through places traded in LDS (220); 8 waves sharing a tile (224), or
// with half of them half a step behind (240: the suffixes' waves find no room beside).
constexpr int kSharedRows = 32 * 4;
template <int D>
constexpr int shared_bytes() { return 4 * kC8Tile * D * 2; }
template <int D, bool kInt8, bool kToken>
__device__ __forceinline__ void shared8(const Cached8Args& a, const Keys8& s, int kvh, int x0, int rows, int split, uint4* lds, int wave,
                                        int lane) {
    constexpr int NT = 2, kBuf = kC8Tile * D * 2 / 16;
    const CachedArgs& ca = a.c;
    const int c = lane & 15, g = lane >> 4;
    x0 += 32 * wave;
    const bool busy = x0 < rows;
    bf16x8 q[NT][D / 32];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const Query8 y = query8(ca, kvh, x0 + 16 * n + c, rows);
        load_query8<D>(q[n], ca.q + y.token * ca.q_stride + y.head * D, g, y.exists);
    }
    const Loader8<D, kToken> ld(a, s, kvh, lane);
    const float cs = ca.scale * kLog2e;
    const int tiles = s.ptiles;
    Rows8<D, NT> r;
    r.clear();
    // Wave w brings block w of the keys, and of V channels D / 4 w ..; C times 16 codes a lane of each, 2 C operands.
    constexpr int C = D / 64;
    uint4 kc[C], vc[C];                                  // codes of K and V on their way to LDS
    float ks, vs;
    auto tile = [&](int i) { return min(i, tiles - 1); };
    auto load_k = [&](int i, int32_t p) {
#pragma unroll
        for (int h = 0; h < C; ++h) kc[h] = *reinterpret_cast<const uint4*>(ld.key_at(i, p) + 4 * wave * D + 16 * h);
    };
    auto load_v = [&](int i, int32_t p) {
#pragma unroll
        for (int h = 0; h < C; ++h) vc[h] = *reinterpret_cast<const uint4*>(ld.value_at(i, p) + 256 * (C * wave + h));
    };
    auto operand = [&](const uint4& x, int u) {
        return __builtin_bit_cast(uint4, u ? codes_to_bf16<kInt8>(x.z, x.w) : codes_to_bf16<kInt8>(x.x, x.y));
    };
    auto stage_k = [&](int i, int u) { lds[(i & 1) * kBuf + (2 * C * wave + u) * 64 + lane] = operand(kc[u >> 1], u & 1); };
    auto stage_v = [&](int i, int u) { lds[(2 + (i & 1)) * kBuf + (2 * C * wave + u) * 64 + lane] = operand(vc[u >> 1], u & 1); };
    auto clean_v = [&](int i) {                          // e4m3: no NaN from tokens that do not exist
        const int end = ld.end_key(i) - ld.first_key(i);
        if (!kInt8 && end < kC8Tile) {
            masked_side();
#pragma unroll
            for (int h = 0; h < C; ++h) drop_codes(vc[h], end - 16 * g);
        }
    };
    auto read_k = [&](bf16x8 (&k)[D / 32], int i, int b) {
#pragma unroll
        for (int d = 0; d < D / 32; ++d) k[d] = __builtin_bit_cast(bf16x8, lds[(i & 1) * kBuf + (b * (D / 32) + d) * 64 + lane]);
    };
    auto read_v = [&](bf16x8 (&v)[2], int i, int b) {
#pragma unroll
        for (int u = 0; u < 2; ++u) v[u] = __builtin_bit_cast(bf16x8, lds[(2 + (i & 1)) * kBuf + (b * 2 + u) * 64 + lane]);
    };
    auto products = [&](f32x4 (&sc)[NT][4], const bf16x8 (&k)[D / 32], int b) {
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[n][b] = mfma16(k[d], q[n][d], sc[n][b]);
    };
    // Before step i: the scores of tile i with their maxima, its scales and those of tile i + 1, the codes of K in tile
    // i + 2 and of V in tile i + 1, and the page numbers of K in tile i + 3 and of V in tile
    // i + 2 are in registers; K of tile i + 1 and V of
    // tile i are staged.  Tiles past the last are the last once more.
    const int32_t k0 = ld.key_page(0), k1 = ld.key_page(tile(1)), k2 = ld.key_page(tile(2)), v0 = ld.value_page(0),
                  v1 = ld.value_page(tile(1));
    int32_t nk = ld.key_page(tile(3)), nv = ld.value_page(tile(2));
    Scales8<kToken> f;
    load_k(0, k0);
    load_v(0, v0);
    ld.load_scales(ks, vs, 0, v0);
#pragma unroll
    for (int u = 0; u < 2 * C; ++u) stage_k(0, u);
    load_k(tile(1), k1);
    clean_v(0);
#pragma unroll
    for (int u = 0; u < 2 * C; ++u) stage_v(0, u);
    load_v(tile(1), v1);
#pragma unroll
    for (int u = 0; u < 2 * C; ++u) stage_k(1, u);
    load_k(tile(2), k2);
    int end = min(ld.end_key(0) - ld.first_key(0), kC8Tile);         // keys of the tile
    f.set(ks, vs, cs, end < kC8Tile, end, lane);
    ld.load_scales(ks, vs, tile(1), v1);
    lds_barrier();
    f32x4 sc[NT][4];
    float mn[NT];
    if (busy) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            bf16x8 k[D / 32];
            read_k(k, 0, b);
            products(sc, k, b);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) mn[n] = peak8(sc, n, f, end < kC8Tile, end - 1, g);
    }
    lds_barrier();                                       // K of tile 0 is read: its buffer takes tile 2
    // kMore: tiles that follow, 2 for two or more; only the last may end within the tile.
    // busy_c: the wave has rows.  The others only stage, in a loop of their own: in one with both, the compiler would wait
    // for either's loads.
    auto step = [&](auto busy_c, auto more_c, int i) {
        constexpr int kMore = decltype(more_c)::value;
        constexpr bool has = decltype(busy_c)::value;
        bf16x8 p[NT][2], k[D / 32], v[2], w[2];
        Scales8<kToken> g1;
        float m1[NT];
        if constexpr (kMore == 1) {
            end = min(ld.end_key(i + 1) - ld.first_key(i + 1), kC8Tile);
            clean_v(i + 1);
        }
        // What is done beside the product with V: one part a region.  A register is loaded in a later region than its last
        // use: in the same one the compiler may load first, into another register, and wait for the load to copy it.  (Where
        // it spills an address instead, form_per_simd, the reload waits for the loads before it all the same.)
        auto part = [&](auto b_c) {
            constexpr int b = decltype(b_c)::value, q = D / 64;      // q regions for each of four parts
            const bool masked = kMore == 1 && end < kC8Tile;
            if constexpr (kMore == 0) return;
            if constexpr (b < q) {                           // tile i + 2 in tile i's buffer
                stage_k(i, 2 * b);
                stage_k(i, 2 * b + 1);
            }
            if constexpr (b == q) load_k(tile(i + 3), nk);
            if constexpr (b >= q && b < 2 * q) {
                stage_v(i + 1, 2 * (b - q));
                stage_v(i + 1, 2 * (b - q) + 1);
            }
            if constexpr (b == 2 * q) {
                nk = ld.key_page(tile(i + 4));
                load_v(tile(i + 2), nv);
                g1.set(ks, vs, cs, masked, end, lane);
            }
            if constexpr (b == 3 * q) {
                ld.load_scales(ks, vs, tile(i + 2), nv);
                if constexpr (has) m1[0] = peak8(sc, 0, g1, masked, end - 1, g);
            }
            if constexpr (b == 4 * q - 1) {
                if (q == 1) __builtin_amdgcn_sched_barrier(0);
                nv = ld.value_page(tile(i + 3));
                if constexpr (has) m1[1] = peak8(sc, 1, g1, masked, end - 1, g);
            }
        };
        auto parts = [&](auto... b) { (part(b), ...); };
        if constexpr (!has) {
            if constexpr (D == 128) parts(IC<0>{}, IC<1>{}, IC<2>{}, IC<3>{}, IC<4>{}, IC<5>{}, IC<6>{}, IC<7>{});
            else parts(IC<0>{}, IC<1>{}, IC<2>{}, IC<3>{});
            if constexpr (kMore > 0) lds_barrier();
            return;
        }
        if constexpr (kMore > 0) read_k(k, i + 1, 0);
        refer8(r, mn);
        // Operands are read a block (of K) or two (of V) ahead of their products; the regions keep the compiler from reading them all first.
        auto quarter = [&](auto b_c) {
            constexpr int b = decltype(b_c)::value;
            bf16x8 next[D / 32];
            if constexpr (kMore > 0 && b < 3) read_k(next, i + 1, b + 1);
            if constexpr (b == 2) read_v(v, i, 0);
            if constexpr (b == 3) read_v(w, i, 1);
            weigh8<b>(r, sc, p, f, [&] {
                if constexpr (kMore > 0) products(sc, k, b);
            });
            if constexpr (kMore > 0 && b < 3)
#pragma unroll
                for (int d = 0; d < D / 32; ++d) k[d] = next[d];
            __builtin_amdgcn_sched_barrier(0);
        };
        quarter(IC<0>{});
        quarter(IC<1>{});
        quarter(IC<2>{});
        quarter(IC<3>{});
        sum8(r, p, f, lane);
        auto region = [&](auto b_c) {
            constexpr int b = decltype(b_c)::value;
            bf16x8 next[2];
            if constexpr (b + 2 < D / 16) read_v(next, i, b + 2);
            part(b_c);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n) r.o[n][b] = mfma16(v[u], p[n][u], r.o[n][b]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                v[u] = w[u];
                if constexpr (b + 2 < D / 16) w[u] = next[u];
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        region(IC<0>{});
        region(IC<1>{});
        region(IC<2>{});
        region(IC<3>{});
        if constexpr (D == 128) {
            region(IC<4>{});
            region(IC<5>{});
            region(IC<6>{});
            region(IC<7>{});
        }
        if constexpr (kMore > 0) {
            f = g1;
            mn[0] = m1[0];
            mn[1] = m1[1];
            lds_barrier();
        }
    };
    auto walk = [&](auto busy_c) {
        for (int i = 0; i + 2 < tiles; ++i) step(busy_c, IC<2>{}, i);
        if (tiles > 1) step(busy_c, IC<1>{}, tiles - 2);
        step(busy_c, IC<0>{}, tiles - 1);
    };
    if (!busy) {
        walk(std::false_type{});
        return;
    }
    walk(std::true_type{});
    float l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) l[n] = r.sum(n);
    store8<D, NT>(ca, r, l, kvh, x0, rows, split, false, lane);
}

// Forms of a call (see cached8_plan).
//   kDirect  a workgroup of 8 waves reads prefix and suffix of its rows and writes the output
//   kSplit   workgroups of 4 waves, the prefix's first (few rows), then the suffixes'
//   kShared  workgroups of 4 waves: the prefix's (many rows, shared8), then four units of a wave each of the suffixes
//            (1024 rows behind 4096 + 600: 33 us; with a workgroup to a suffix, 54)
enum Form8 { kDirect8, kSplit8, kShared8 };
constexpr int form_waves(int form) { return form == kDirect8 ? 8 : 4; }
// waves a SIMD, which bounds their registers: 128, 168 or 256 of 512.  Registers that the compiler spills within that:
// 16 rows a unit: none for D = 128; D = 64 none direct, 0 or 1 split, shared 2 (block scales) or 9 to 11 (a scale a token);
// 32 rows: D = 64 none direct, 13 to 21 split, 8 to 23 shared; D = 128 1 to 7 direct, 13 to 23 split, 4 to 8 shared.
// A spilled address is reloaded in the loop, and as a wave's memory operations are waited for in order, the wait covers
// the tile's loads too: part of why 256 tokens behind 4096 + 600 keys take 38 us with block scales and 53 with a scale a
// token (64 x 8 behind 16384 + 999, 32 / 8 heads of 64: 114 to 122 and 160).
constexpr int form_per_simd(int D, int NT, int form) {
    if (D == 128) return 2;
    if (form == kSplit8) return NT == 1 ? 4 : 3;
    return form == kShared8 ? 3 : NT == 1 ? 4 : 2;
}
constexpr int own_waves(int form) { return form == kDirect8 ? 8 : form == kSplit8 ? 4 : 1; }

template <int D, int NT, bool kInt8, bool kToken, int kForm>
__global__ __launch_bounds__(64 * form_waves(kForm), form_per_simd(D, NT, kForm)) void attn_cached8_kernel(Cached8Args a) {
    constexpr int W = form_waves(kForm), U = own_waves(kForm);
    constexpr int kLds = kForm == kShared8 ? shared_bytes<D>() : W / 2 * join_floats<D, NT>() * 4;
    __shared__ uint4 lds[kLds / 16];
    const CachedArgs& ca = a.c;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int G = ca.Hq / ca.Hkv, prefix_blocks = (int)ca.prefix_blocks;
    int block = blockIdx.x;
    Keys8 s;
    s.prefix = ca.prefix_pages;
    if (kForm != kDirect8 && block < prefix_blocks) {
        const int kvh = block % ca.Hkv, rest = block / ca.Hkv, split = rest % ca.prefix_splits;
        s.own = nullptr;
        s.len = 0;
        s.p0 = split * ca.prefix_chunk;
        s.p1 = min(s.p0 + ca.prefix_chunk, ca.prefix_len);
        s.ptiles = (s.p1 - s.p0 + kC8Tile - 1) / kC8Tile;
        s.tile0 = 0;
        const int rows = ca.N * ca.L * G;
        if constexpr (kForm == kShared8)
            shared8<D, kInt8, kToken>(a, s, kvh, rest / ca.prefix_splits * kSharedRows, rows, split, lds, wave, lane);
        else
            keys8<D, NT, kInt8, kToken, U>(a, s, kvh, rest / ca.prefix_splits * 16 * NT, rows, 0, s.ptiles, split, false,
                                           reinterpret_cast<float*>(lds), wave, lane);
        return;
    }
    const int unit_wave = wave % U;
    const int64_t units = (int64_t)ca.N * ((ca.L * G + 16 * NT - 1) / (16 * NT)) * ca.Hkv * (kForm == kDirect8 ? 1 : ca.suffix_splits);
    const int64_t mine = (int64_t)(block - prefix_blocks) * (W / U) + wave / U;
    const bool none = mine >= units;             // the last workgroup's second unit
    int rest = (int)(none ? units - 1 : mine);
    const int kvh = rest % ca.Hkv;
    rest /= ca.Hkv;
    const int splits = kForm == kDirect8 ? 1 : ca.suffix_splits, split = rest % splits;
    rest /= splits;
    const int blocks = (ca.L * G + 16 * NT - 1) / (16 * NT);
    const int seq = rest / blocks, rb = rest % blocks;
    s.own = ca.page_table + (int64_t)seq * ca.max_pages;
    s.len = none ? 0 : min(max(ca.suffix_len[seq], 0), a.max_suffix);
    s.p0 = 0;
    s.p1 = kForm == kDirect8 ? ca.prefix_len : 0;
    s.ptiles = (s.p1 + kC8Tile - 1) / kC8Tile;
    const int all = (s.len + kC8Tile - 1) / kC8Tile, per = (all + splits - 1) / splits;
    const int t0 = min(split * per, all), t1 = min(t0 + per, all);
    s.tile0 = t0;
    const int end = none ? 0 : (seq + 1) * ca.L * G;        // no row exists for `none`
    keys8<D, NT, kInt8, kToken, U>(a, s, kvh, seq * ca.L * G + rb * 16 * NT, end, s.len, s.ptiles + t1 - t0,
                                   ca.prefix_splits + split, kForm == kDirect8 || ca.prefix_splits + splits == 1,
                                   reinterpret_cast<float*>(lds) + (wave / U) * (U / 2) * join_floats<D, NT>(), unit_wave, lane);
}

inline int cached8_row_tiles(int L, int G) { return (int64_t)L * G <= 16 ? 1 : 2; }

// Defined in the file of its format and head dimension.
template <int D, bool kInt8>
hipError_t launch_cached8(const Cached8Args& a, int form, int64_t blocks, hipStream_t s);

#ifdef LFM2SC_CACHED8_D
template <int D, bool kInt8>
hipError_t launch_cached8(const Cached8Args& a, int form, int64_t blocks, hipStream_t s) {
    auto go = [&](auto n, auto token, auto f) {
        constexpr int kForm = decltype(f)::value;
        hipLaunchKernelGGL((attn_cached8_kernel<D, decltype(n)::value, kInt8, decltype(token)::value, kForm>), dim3((uint32_t)blocks),
                           dim3(64 * form_waves(kForm)), 0, s, a);
    };
    auto by_form = [&](auto n, auto token) {
        if (form == kDirect8) go(n, token, IC<kDirect8>{});
        else if (form == kSplit8) go(n, token, IC<kSplit8>{});
        else go(n, token, IC<kShared8>{});
    };
    auto by_token = [&](auto n) {
        if (a.block_shift == 0) by_form(n, std::true_type{});
        else by_form(n, std::false_type{});
    };
    if (cached8_row_tiles(a.c.L, a.c.Hq / a.c.Hkv) == 1) by_token(IC<1>{});
    else by_token(IC<2>{});
    return hipGetLastError();
}
template hipError_t launch_cached8<LFM2SC_CACHED8_D, LFM2SC_CACHED8_INT8>(const Cached8Args&, int, int64_t, hipStream_t);
#endif

}  // namespace lfm2sc
