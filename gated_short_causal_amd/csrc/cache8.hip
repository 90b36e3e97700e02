// cache8.hip -- k and v rows quantised into a paged cache of 8-bit codes as they
// are written (lfm2sc_cache8_write), and read back (lfm2sc_cache8_read).
//
// Both are streams: 2 bytes an element on the rows' side, 1 on the cache's.  A
// wave takes 16 tokens (a tile) of one head's keys or values; the waves of a
// block of scale_tokens tokens sit in one workgroup and agree on its scale
// through LDS, with the rows in registers meanwhile, so rows are read once.
//
// The tiles of a call are found on the device, as lengths are device data.
// Sequence i of a packed call has at most (n_i - 1) / U + 2 units of U tokens;
// on a virtual axis it begins at cu[i] / U + 2 i, so units [0, T / U + 2 N) hold
// every sequence's, and a wave finds its own by a search over that monotone key.
#include "attn_common.hpp"
#include "cache8.hpp"

namespace lfm2sc {

// Units of 2^shift tokens that n >= 1 neighbouring tokens may touch.
__host__ __device__ inline int64_t units_of(int64_t n, int shift) { return ((n - 2 + (1 << shift)) >> shift) + 1; }

struct Unit {
    int seq;          // -1: none
    int64_t row;      // packed row of token `start`
    int start, len;   // the call's tokens of the sequence: [start, len); may begin below 0
    int first;        // first token of the unit
};

// The unit-th unit of `U` tokens (a power of two).
__device__ __forceinline__ Unit find_unit(const Cache8Rows& a, uint32_t unit, int shift) {
    const int lane = threadIdx.x & 63;
    Unit u;
    int64_t begin, end;
    int j;
    if (a.cu == nullptr) {
        const uint32_t per = (uint32_t)units_of(a.L, shift);
        u.seq = (int)(unit / per);
        j = (int)(unit % per);
        begin = (int64_t)u.seq * a.L;
        end = begin + a.L;
    } else {
        auto key = [&](int i) { return (min(max((int64_t)a.cu[i], (int64_t)0), a.T) >> shift) + 2 * (int64_t)i; };
        int lo = 0, hi = a.N;                    // key(lo) <= unit (or lo == 0), key(hi) > unit (or hi == N)
        while (hi - lo > 1) {                    // 64 parts a step
            const int step = (hi - lo + 63) / 64, at = lo + (lane + 1) * step;
            const int part = __popcll(__ballot(at < hi && key(min(at, a.N)) <= unit));
            const int next = lo + part * step;
            hi = min(next + step, hi);
            lo = next;
        }
        u.seq = lo;
        begin = min(max((int64_t)a.cu[lo], (int64_t)0), a.T);
        end = min(max((int64_t)a.cu[lo + 1], begin), a.T);
        const int64_t d = unit - ((begin >> shift) + 2 * (int64_t)lo);
        j = d < 0 || d > (1 << 30) ? (1 << 30) : (int)d;
    }
    u.len = min(max(a.seq_len[u.seq], 0), a.max_pages << a.page_shift);
    u.start = u.len - (int)(end - begin);
    u.row = begin;
    const int64_t first = (((int64_t)max(u.start, 0) >> shift) + j) << shift;
    if (end == begin || first >= u.len) u.seq = -1;
    u.first = (int)min(first, (int64_t)1 << 30);
    return u;
}

// The workgroup's waves, `tiles` to a unit, and the wave's share of the call.
struct Share {
    Unit u;
    int head, tile;   // tile: first token
    bool v;
    int32_t page;
};
__device__ __forceinline__ Share find_share(const Cache8Args& a, int shift, int tiles, int wave, int waves) {
    Share s;
    const uint32_t task = blockIdx.x * (uint32_t)(waves / tiles) + (uint32_t)(wave / tiles);     // < 2^26, see the launcher
    const uint32_t unit = task / (uint32_t)(2 * a.Hkv);
    const int rest = (int)(task % (uint32_t)(2 * a.Hkv));
    s.v = rest >= a.Hkv;
    s.head = s.v ? rest - a.Hkv : rest;
    s.u.seq = -1;
    if (unit < a.units) s.u = find_unit(a.rows, unit, shift);
    s.tile = s.u.seq < 0 ? 0 : s.u.first + wave % tiles * kTileTokens;
    s.page = s.u.seq < 0 ? 0 : a.rows.page_table[(int64_t)s.u.seq * a.rows.max_pages + (s.u.first >> a.rows.page_shift)];
    return s;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x = max(x, (uint32_t)__shfl_xor((int)x, d, 64));
    return x;
}

// ---------------------------------------------------------------- write
// kToken: a scale for every token; else one for the unit's tokens.
//
// K: a lane holds 8 channels of a token, 64 / (D / 8) tokens an access.  V: a lane
// holds two channels of 16 D / 128 tokens, half of them (D = 64) or all.
template <typename E, int D, bool kInt8, bool kToken>
__global__ __launch_bounds__(512) void cache8_write_kernel(Cache8Args a) {
    constexpr int kLanesRow = D / 8, kRowsAcc = 64 / kLanesRow, kAcc = kTileTokens / kRowsAcc;
    constexpr int kVTok = D == 64 ? 8 : 16;      // tokens of a lane's two V channels
    __shared__ uint32_t tops[8];
    __shared__ float vsc[8][kTileTokens];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6, tiles = kToken ? 1 : 1 << (a.block_shift - 4);
    const Share s = find_share(a, kToken ? 4 : a.block_shift, tiles, wave, waves);
    const Cache8Rows& r = a.rows;
    const Unit& u = s.u;
    const bool busy = u.seq >= 0 && s.page >= 0 && s.page < a.num_pages;
    const int t0 = max(u.start, 0);              // tokens [t0, len) are written
    const int in_page = s.tile & ((1 << r.page_shift) - 1);
    const int64_t head_at = (int64_t)s.page * a.page_stride + (((int64_t)s.head << r.page_shift) + in_page) * D;
    const int64_t scale_at = (int64_t)s.page * a.scale_stride + ((int64_t)s.head << (r.page_shift - a.block_shift)) +
                             (in_page >> a.block_shift);
    const int vt0 = D == 64 ? (lane >> 5) * 8 : 0, vc = D == 64 ? lane & 31 : lane;

    float x[kAcc * 8 > 2 * kVTok ? kAcc * 8 : 2 * kVTok];
    uint32_t top[kToken ? kVTok : 1];
    float old = 0.f;
    static_assert(kAcc * 8 == 2 * kVTok, "16 D / 64 elements a lane");
    constexpr int kX = kAcc * 8;
    const bool keeps = !kToken && busy && u.first < t0;      // tokens of the unit stay from before
    if (busy) {
        if (keeps) old = (s.v ? a.v_scales : a.k_scales)[scale_at];
        const E* rows = (const E*)(s.v ? a.v_rows : a.k_rows) + (int64_t)s.head * D;
        const int64_t stride = s.v ? a.v_row_stride : a.k_row_stride;
        if (!s.v) {
            Raw8<E> raw[kAcc];
#pragma unroll
            for (int i = 0; i < kAcc; ++i) {
                const int t = s.tile + i * kRowsAcc + lane / kLanesRow;
                raw[i] = Raw8<E>{};
                if (t >= t0 && t < u.len) raw[i] = ld8s<E, 1>(rows + (u.row + (t - u.start)) * stride + lane % kLanesRow * 8);
            }
#pragma unroll
            for (int i = 0; i < kAcc; ++i) to_f32(raw[i], x + 8 * i);
        } else {
            // x[2 j + c]: token vt0 + j, channel 2 vc + c
            uint32_t raw[kVTok * (sizeof(E) / 2)];
#pragma unroll
            for (int j = 0; j < kVTok; ++j) {
                const int t = s.tile + vt0 + j;
                const bool in = t >= t0 && t < u.len;
                const E* p = rows + (u.row + (t - u.start)) * stride + 2 * vc;
                if constexpr (sizeof(E) == 2) {
                    raw[j] = 0;
                    if (in) raw[j] = *reinterpret_cast<const uint32_t*>(p);
                } else {
                    uint2 w = make_uint2(0, 0);
                    if (in) w = *reinterpret_cast<const uint2*>(p);
                    raw[2 * j] = w.x;
                    raw[2 * j + 1] = w.y;
                }
            }
#pragma unroll
            for (int j = 0; j < kVTok; ++j) {
                if constexpr (sizeof(E) == 2) {
                    x[2 * j] = __uint_as_float(raw[j] << 16);
                    x[2 * j + 1] = __uint_as_float(raw[j] & 0xffff0000u);
                } else {
                    x[2 * j] = __uint_as_float(raw[2 * j]);
                    x[2 * j + 1] = __uint_as_float(raw[2 * j + 1]);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kX; ++i) x[i] = 0.f;
    }

    float ratio = 1.f;
    float inv[kToken ? kX : 1];                  // 1 / scale: of each value, or of the unit
    if constexpr (!kToken) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kX; ++i) m = max(m, finite_magnitude(x[i]));
        m = wave_max(m);
        if (tiles > 1) {
            asm volatile("" ::"v"(old));         // every wave has the old scale before one writes the new
            if (lane == 0) tops[wave] = m;
            __syncthreads();
            for (int w = wave / tiles * tiles; w < (wave / tiles + 1) * tiles; ++w) m = max(m, tops[w]);
        }
        const float t = __uint_as_float(m);
        const float scale = keeps ? joined_scale<kInt8>(old, t, ratio) : fresh_scale<kInt8>(t);
        inv[0] = scale > 0.f ? 1.f / scale : 0.f;
        if (busy && wave % tiles == 0 && lane == 0) (s.v ? a.v_scales : a.k_scales)[scale_at] = scale;
    } else {
        if (!s.v) {
#pragma unroll
            for (int i = 0; i < kAcc; ++i) {
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = max(m, finite_magnitude(x[8 * i + e]));
#pragma unroll
                for (int d = 1; d < kLanesRow; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
                const float scale = fresh_scale<kInt8>(__uint_as_float(m));
#pragma unroll
                for (int e = 0; e < 8; ++e) inv[8 * i + e] = scale > 0.f ? 1.f / scale : 0.f;
                const int tt = i * kRowsAcc + lane / kLanesRow, t = s.tile + tt;
                if (busy && lane % kLanesRow == 0 && t >= t0 && t < u.len) a.k_scales[scale_at + tt] = scale;
            }
        } else {
            // the lanes of a token: halving the tokens that a lane keeps, then the lanes left with one
#pragma unroll
            for (int j = 0; j < kVTok; ++j) top[j] = max(finite_magnitude(x[2 * j]), finite_magnitude(x[2 * j + 1]));
            int kept = 0;
#pragma unroll
            for (int n = kVTok / 2, d = 1; n >= 1; n >>= 1, d <<= 1) {
                const bool upper = (lane & d) != 0;
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const uint32_t mine = upper ? top[j + n] : top[j], other = upper ? top[j] : top[j + n];
                    top[j] = max(mine, (uint32_t)__shfl_xor((int)other, d, 64));
                }
                kept += upper ? n : 0;
            }
            uint32_t m = top[0];
#pragma unroll
            for (int d = kVTok; d < (D == 64 ? 32 : 64); d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
            const float scale = fresh_scale<kInt8>(__uint_as_float(m));
            const int tt = vt0 + kept, t = s.tile + tt;
            if ((lane & (D == 64 ? 31 : 63)) < kVTok) {
                vsc[wave][tt] = scale > 0.f ? 1.f / scale : 0.f;
                if (busy && t >= t0 && t < u.len) a.v_scales[scale_at + tt] = scale;
            }
            lds_reads_done();                    // and writes
#pragma unroll
            for (int j = 0; j < kVTok; ++j) inv[2 * j] = inv[2 * j + 1] = vsc[wave][vt0 + j];
        }
    }
    if (!busy) return;

    // kept tokens of the unit: their codes in steps of the new scale
    const bool again = keeps && ratio != 1.f;
    if (!s.v) {
        uint8_t* at = a.k_pages + head_at + lane % kLanesRow * 8;
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int tt = i * kRowsAcc + lane / kLanesRow, t = s.tile + tt;
            float f[8];
            if (t >= t0 && t < u.len) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = x[8 * i + e] * (kToken ? inv[kToken ? 8 * i + e : 0] : inv[0]);
            } else if (again && t < t0) {
                const uint2 c = *reinterpret_cast<const uint2*>(at + tt * D);
                decode4<kInt8>(c.x, f);
                decode4<kInt8>(c.y, f + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= ratio;
            } else {
                continue;
            }
            *reinterpret_cast<uint2*>(at + tt * D) = make_uint2(encode4<kInt8>(f), encode4<kInt8>(f + 4));
        }
        return;
    }
    if (s.tile >= u.len || (s.tile + kTileTokens <= t0 && !again)) return;
    // V: a channel's tokens are neighbours
    uint32_t c[2][kVTok / 4];
#pragma unroll
    for (int ch = 0; ch < 2; ++ch)
#pragma unroll
        for (int g = 0; g < kVTok / 4; ++g) {
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 2 * (4 * g + e) + ch;
                f[e] = x[i] * (kToken ? inv[kToken ? i : 0] : inv[0]);
            }
            c[ch][g] = encode4<kInt8>(f);
        }
    uint8_t* at = a.v_pages + head_at + 2 * vc * kTileTokens + vt0;
    const bool merge = s.tile < t0 || s.tile + kTileTokens > u.len;      // bytes of other tokens stay
    if (merge) {
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
            for (int g = 0; g < kVTok / 4; ++g) {
                const uint32_t was = *reinterpret_cast<const uint32_t*>(at + ch * kTileTokens + 4 * g);
                uint32_t keep = was;
                if (again) {
                    float f[4];
                    decode4<kInt8>(was, f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] *= ratio;
                    keep = encode4<kInt8>(f);
                }
                uint32_t now = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = s.tile + vt0 + 4 * g + e;
                    const uint32_t m = 0xffu << (8 * e);
                    now |= (t < t0 ? keep : t < u.len ? c[ch][g] : was) & m;
                }
                c[ch][g] = now;
            }
    }
    if constexpr (D == 64) {
        *reinterpret_cast<uint2*>(at) = make_uint2(c[0][0], c[0][1]);
        *reinterpret_cast<uint2*>(at + kTileTokens) = make_uint2(c[1][0], c[1][1]);
    } else {
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
            *reinterpret_cast<uint4*>(at + ch * kTileTokens) =
                make_uint4(c[ch][0], c[ch][1], c[ch][kVTok / 4 - 2], c[ch][kVTok / 4 - 1]);
    }
}

// ---------------------------------------------------------------- read
template <typename E, int D, bool kInt8>
__global__ __launch_bounds__(256) void cache8_read_kernel(Cache8Args a) {
    constexpr int kLanesRow = D / 8, kRowsAcc = 64 / kLanesRow, kAcc = kTileTokens / kRowsAcc;
    constexpr int kVTok = D == 64 ? 8 : 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Share s = find_share(a, 4, 1, wave, 4);
    const Cache8Rows& r = a.rows;
    const Unit& u = s.u;
    if (u.seq < 0) return;
    const int page = min(max(s.page, 0), a.num_pages - 1);
    const int t0 = max(u.start, 0);
    const int in_page = s.tile & ((1 << r.page_shift) - 1);
    const int64_t head_at = (int64_t)page * a.page_stride + (((int64_t)s.head << r.page_shift) + in_page) * D;
    const int64_t scale_at = (int64_t)page * a.scale_stride + ((int64_t)s.head << (r.page_shift - a.block_shift)) +
                             (in_page >> a.block_shift);
    const int bs = a.block_shift;                // 0 or at least 4: a tile has one scale, or 16
    E* rows = (E*)(s.v ? a.v_rows : a.k_rows) + (int64_t)s.head * D;
    const int64_t stride = s.v ? a.v_row_stride : a.k_row_stride;
    if (!s.v) {
        uint2 c[kAcc];
        float sc[kAcc];
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int tt = i * kRowsAcc + lane / kLanesRow;
            c[i] = *reinterpret_cast<const uint2*>(a.k_pages + head_at + tt * D + lane % kLanesRow * 8);
            sc[i] = a.k_scales[scale_at + (tt >> bs)];
        }
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int t = s.tile + i * kRowsAcc + lane / kLanesRow;
            float f[8];
            decode4<kInt8>(c[i].x, f);
            decode4<kInt8>(c[i].y, f + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= sc[i];
            if (t >= t0 && t < u.len)
                st8s<E, 2>(rows + (u.row + (t - u.start)) * stride + lane % kLanesRow * 8, from_f32<E>(f));
        }
        return;
    }
    const int vt0 = D == 64 ? (lane >> 5) * 8 : 0, vc = D == 64 ? lane & 31 : lane;
    const uint8_t* at = a.v_pages + head_at + 2 * vc * kTileTokens + vt0;
    uint32_t c[2][kVTok / 4];
    float sc[kVTok];
#pragma unroll
    for (int ch = 0; ch < 2; ++ch)
#pragma unroll
        for (int g = 0; g < kVTok / 8; ++g) {
            const uint2 w = *reinterpret_cast<const uint2*>(at + ch * kTileTokens + 8 * g);
            c[ch][2 * g] = w.x;
            c[ch][2 * g + 1] = w.y;
        }
#pragma unroll
    for (int j = 0; j < kVTok; ++j) sc[j] = a.v_scales[scale_at + ((vt0 + j) >> bs)];
#pragma unroll
    for (int g = 0; g < kVTok / 4; ++g) {
        float f[2][4];
        decode4<kInt8>(c[0][g], f[0]);
        decode4<kInt8>(c[1][g], f[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 4 * g + e, t = s.tile + vt0 + j;
            if (t < t0 || t >= u.len) continue;
            E* p = rows + (u.row + (t - u.start)) * stride + 2 * vc;
            const float y0 = f[0][e] * sc[j], y1 = f[1][e] * sc[j];
            if constexpr (sizeof(E) == 2) *reinterpret_cast<uint32_t*>(p) = Elem<uint16_t>::pack2(y0, y1);
            else *reinterpret_cast<float2*>(p) = make_float2(y0, y1);
        }
    }
}

// Units of 2^shift tokens that a call's sequences may touch.
static int64_t cache8_units(const Cache8Rows& r, int shift) {
    if (r.cu == nullptr) return (int64_t)r.N * units_of(r.L, shift);
    return (r.T >> shift) + 2 * (int64_t)r.N;
}

template <typename E, int D, bool kInt8>
static hipError_t launch_write(const Cache8Args& a, dim3 grid, dim3 block, hipStream_t s) {
    if (a.block_shift == 0) hipLaunchKernelGGL((cache8_write_kernel<E, D, kInt8, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((cache8_write_kernel<E, D, kInt8, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_cache8(Cache8Args a, int D, bool int8, bool f32, bool write, hipStream_t s) {
    const int shift = write && a.block_shift > 4 ? a.block_shift : 4, tiles = 1 << (shift - 4);
    const int waves = tiles > 4 ? tiles : 4;     // scale_tokens <= 128: at most 8
    a.units = cache8_units(a.rows, shift);
    const int64_t tasks = a.units * 2 * a.Hkv, blocks = (tasks + waves / tiles - 1) / (waves / tiles);
    if (too_many(blocks, 64 * waves)) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)blocks), block(64 * waves);
    auto go = [&](auto e) {
        using E = decltype(e);
        if (!write) {
            if (D == 64 && int8) hipLaunchKernelGGL((cache8_read_kernel<E, 64, true>), grid, block, 0, s, a);
            else if (D == 64) hipLaunchKernelGGL((cache8_read_kernel<E, 64, false>), grid, block, 0, s, a);
            else if (int8) hipLaunchKernelGGL((cache8_read_kernel<E, 128, true>), grid, block, 0, s, a);
            else hipLaunchKernelGGL((cache8_read_kernel<E, 128, false>), grid, block, 0, s, a);
            return hipGetLastError();
        }
        if (D == 64) return int8 ? launch_write<E, 64, true>(a, grid, block, s) : launch_write<E, 64, false>(a, grid, block, s);
        return int8 ? launch_write<E, 128, true>(a, grid, block, s) : launch_write<E, 128, false>(a, grid, block, s);
    };
    return f32 ? go(float{}) : go(uint16_t{});
}

}  // namespace lfm2sc
