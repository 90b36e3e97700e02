// cache8.hpp -- the paged cache of 8-bit codes: its layout and the conversions
// that the write, the read (cache8.hip) and the attention (attn_cached8.hip) share.
//
// A page holds S = page_size tokens of every key/value head.
//   K page  [Hkv][S][D]         a token's codes are D bytes
//   V page  [Hkv][S / 16][D][16]  a channel's codes of 16 tokens are 16 bytes
// A head's 16 tokens are 16 D contiguous bytes in both.  V lies as the matrix
// unit takes it in the product with the probabilities (a channel, and tokens in
// a row), so the attention loads both straight into registers, with no transposing
// read (and through LDS only where many rows share a tile).  Scales
// [Hkv][S / scale_tokens] fp32 a page, a value is its code times the scale of its
// block of tokens.
#pragma once

#include "common.hpp"
#include "hybrid.hpp"

namespace lfm2sc {

constexpr int kTileTokens = 16;
constexpr float kMinScale = 7.88860905e-31f;     // 2^-100: its reciprocal, and products with it, are normal numbers

template <bool kInt8>
__device__ __forceinline__ float code_max() { return kInt8 ? 127.f : 448.f; }

// Four codes as fp32 values.
template <bool kInt8>
__device__ __forceinline__ void decode4(uint32_t c, float* f) {
    if constexpr (kInt8) {
        f[0] = (float)(int8_t)c;
        f[1] = (float)(int8_t)(c >> 8);
        f[2] = (float)(int8_t)(c >> 16);
        f[3] = (float)(int8_t)(c >> 24);
    } else {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
        f[0] = a[0];
        f[1] = a[1];
        f[2] = b[0];
        f[3] = b[1];
    }
}

// Four values, in steps of their scale, as codes: rounded to nearest even,
// beyond the largest code the largest; a NaN is 0 (int8) or stays NaN (e4m3).
template <bool kInt8>
__device__ __forceinline__ uint32_t encode4_any(const float* f) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float c = __builtin_amdgcn_fmed3f(f[i], -code_max<kInt8>(), code_max<kInt8>());
        x[i] = f[i] != f[i] ? (kInt8 ? 0.f : f[i]) : c;
    }
    if constexpr (kInt8) {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) r |= ((uint32_t)(int)__builtin_rintf(x[i]) & 0xffu) << (8 * i);
        return r;
    } else {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
    }
}

// The same for values that are numbers and whose codes the scale holds (below
// 127.5, 464): 11 instead of 30 instructions for int8.  x + 1.5 * 2^23 rounds x to a
// whole number (nearest even) whose low byte is the code; not fused with the product
// that x came from, which is rounded first.
template <bool kInt8>
__device__ __forceinline__ uint32_t encode4(const float* f) {
#pragma clang fp contract(off)
    if constexpr (kInt8) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __float_as_uint(f[i] + 12582912.f);
        const uint32_t lo = __builtin_amdgcn_perm(x[1], x[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(x[3], x[2], 0x04000c0cu);
        return lo | hi;
    } else {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
    }
}

// Magnitude of x as the bits of a float >= 0 (they order as the values do);
// 0 for an infinity or a NaN, which do not count for a scale.
__device__ __forceinline__ uint32_t finite_magnitude(float x) {
    const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
    return a < 0x7f800000u ? a : 0u;
}

// Scale of a block whose largest magnitude is `top`, without earlier tokens: int8
// top / 127; e4m3 the lowest power of two with top <= 448 scales, so that codes of
// a larger scale are the same digits (a code is a float itself: a finer scale
// would gain nothing).  0 for a block of zeros.
template <bool kInt8>
__device__ __forceinline__ float fresh_scale(float top) {
    if (!(top > 0.f)) return 0.f;
    if constexpr (kInt8) return fmaxf(top / 127.f, kMinScale);
    const uint32_t b = __float_as_uint(top);     // 448 = 1.75 * 2^8
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(e < 27 ? 27 : e) << 23);     // 2^-100 or more
}

// The scale of a block that keeps tokens of scale `old` when new ones of largest
// magnitude `top` join: old times the lowest power of two that holds them.  So
// the kept codes, rounded again at each doubling, stay within one step of their
// value however many tokens join: half a step for the last rounding, a quarter
// of today's step for the one before, and so on.  `ratio`: old / new.
template <bool kInt8>
__device__ __forceinline__ float joined_scale(float old, float top, float& ratio) {
    ratio = 0.f;
    if (!(old >= kMinScale && old < __builtin_inff())) return fresh_scale<kInt8>(top);     // the kept values are zeros
    const float need = top * (1.f / old);
    if (!(need < 1.1e12f)) return fresh_scale<kInt8>(top);         // 2^40 steps and more: the kept codes round to 0
    constexpr int kTopExp = kInt8 ? 6 : 8;       // floor(log2 of the largest code)
    int n = (int)(__float_as_uint(need) >> 23) - 127 - kTopExp;
    n = n < 0 ? 0 : n;
    ratio = __uint_as_float((uint32_t)(127 - n) << 23);
    if (kInt8 ? !(need * ratio < 127.5f) : !(need * ratio <= 448.f)) {
        ++n;
        ratio *= 0.5f;
    }
    return old * __uint_as_float((uint32_t)(127 + n) << 23);
}

}  // namespace lfm2sc
