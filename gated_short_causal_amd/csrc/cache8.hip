// cache8.hip -- k and v rows quantised into a paged cache of 8-bit codes as they
// are written (lfm2sc_cache8_write), and read back (lfm2sc_cache8_read).
//
// Both are streams: 2 bytes an element on the rows' side, 1 on the cache's.  A
// wave takes 16 tokens (a tile) of one head's keys and values; the waves of a
// block of scale_tokens tokens sit in one workgroup and agree on its scales
// through LDS, with the rows in registers meanwhile, so rows are read once.  Small
// calls are a chain of dependent reads (lengths, page number, cache), so each wave
// asks for the rows before it knows the page, and for K and V together.
//
// The tiles of a call are found on the device, as lengths are device data.
// Sequence i of a packed call has at most (n_i - 1) / U + 2 units of U tokens;
// on a virtual axis it begins at cu[i] / U + 2 i, so units [0, T / U + 2 N) hold
// every sequence's, and a wave finds its own by a search over that monotone key.
//
// Measured (one MI355X): 65536 tokens of 8 heads of 128 written in 80 to 86 us (4.7 TB/s of
// rows, codes and scales; copies reach 5.1; vector unit 38% busy), read back in 65 us
// behind the write, when part of the codes is in the last cache, else in 75 us, and in 93
// to 108 into columns of one buffer; fp32 rows 131 and, into such columns, 176 us (130 at
// the copy's rate).  8 x <= 2048 tokens of 64: 9.9 and 6.7 us; 8 x 1024 with a scale a
// token 10.5 and 7.1 us (fp32 11.9 and 10.6), a scale for 16 tokens 8.4 and 6.9 (10.3 and
// 11.0): a wave's loads, maxima over lanes and stores follow each other, in one round of
// the card.  64 x 8 drafted tokens: 9.1 and 9.5; 256 single tokens 4.9 to 5.9, the block
// that each joins 8.5: four dependent reads of about 1 us each (lengths, page number,
// codes and scales beside rows), not bytes.  With a wave for K and one for V, and earlier
// codes asked for after the scales: 14.4 us (64 x 8 written), 7.3 (256), 12.7 (8 x 2048).
#include "attn_common.hpp"
#include "cache8.hpp"
#include "seq_find.hpp"

namespace lfm2sc {

// Units of 2^shift tokens that n >= 1 neighbouring tokens may touch.
__host__ __device__ inline int64_t units_of(int64_t n, int shift) { return ((n - 2 + (1 << shift)) >> shift) + 1; }

struct Unit {
    int seq;          // -1: none
    int64_t row;      // packed row of token `start`
    int start, len;   // the call's tokens of the sequence: [start, len); may begin below 0
    int first;        // first token of the unit
};

// The unit-th unit of 2^shift tokens.
__device__ __forceinline__ Unit find_unit(const Cache8Rows& a, uint32_t unit, int shift) {
    Unit u;
    int64_t begin, end;
    int j, len;
    if (a.cu == nullptr) {
        const uint32_t per = (uint32_t)units_of(a.L, shift);
        u.seq = (int)(unit / per);
        j = (int)(unit % per);
        begin = (int64_t)u.seq * a.L;
        end = begin + a.L;
        len = a.seq_len[u.seq];
    } else {
        auto row = [&](int at) { return min(max((int64_t)at, (int64_t)0), a.T); };
        const SeqAt s = find_seq(a.cu, a.seq_len, a.N, [&](int i, int at) { return (row(at) >> shift) + 2 * (int64_t)i <= unit; });
        u.seq = s.seq;
        begin = row(s.begin);
        end = max(row(s.end), begin);
        len = s.extra;
        const int64_t d = unit - ((begin >> shift) + 2 * (int64_t)s.seq);
        j = d < 0 || d > (1 << 30) ? (1 << 30) : (int)d;
    }
    u.len = min(max(len, 0), a.max_pages << a.page_shift);
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
    int32_t page;     // -1 where there is no unit
};
__device__ __forceinline__ Share find_share(const Cache8Args& a, int shift, int tiles, int wave, int waves) {
    Share s;
    const uint32_t task = blockIdx.x * (uint32_t)(waves / tiles) + (uint32_t)(wave / tiles);     // < 2^26, see the launcher
    const uint32_t unit = task / (uint32_t)a.Hkv;
    s.head = (int)(task % (uint32_t)a.Hkv);
    s.u.seq = -1;
    s.page = -1;
    s.tile = 0;
    if (unit < a.units) s.u = find_unit(a.rows, unit, shift);
    if (s.u.seq < 0) return s;
    s.tile = s.u.first + wave % tiles * kTileTokens;
    s.page = a.rows.page_table[(int64_t)s.u.seq * a.rows.max_pages + (s.u.first >> a.rows.page_shift)];
    return s;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x = max(x, (uint32_t)__shfl_xor((int)x, d, 64));
    return x;
}

// A lane's place in a tile.  K: 8 channels of a token, 64 / (D / 8) tokens an access.  V: two
// channels of 16 D / 128 tokens: 8 of them (D = 64) or all.
template <int D>
struct Lane8 {
    static constexpr int kRow = D / 8, kRows = 64 / kRow, kAcc = kTileTokens / kRows;     // K: lanes a row, rows an access, accesses
    static constexpr int kTok = D == 64 ? 8 : 16;                                         // V: tokens of a channel
    int kc, kt, vc, vt;              // first channel and token
    __device__ __forceinline__ explicit Lane8(int lane)
        : kc(lane % kRow * 8), kt(lane / kRow), vc(D == 64 ? 2 * (lane & 31) : 2 * lane), vt(D == 64 ? (lane >> 5) * 8 : 0) {}
};

// ---------------------------------------------------------------- write
// kToken: a scale for every token; else one for the unit's tokens.
template <typename E, int D, bool kInt8, bool kToken>
__global__ __launch_bounds__(512) void cache8_write_kernel(Cache8Args a) {
    using Lane = Lane8<D>;
    constexpr int kAcc = Lane::kAcc, kTok = Lane::kTok, kX = 8 * kAcc;
    static_assert(kX == 2 * kTok, "16 D / 64 elements a lane");
    __shared__ uint32_t tops[2][8];
    __shared__ float vsc[8][kTileTokens];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6, tiles = kToken ? 1 : 1 << (a.block_shift - 4);
    const Lane at(lane);
    const Share s = find_share(a, kToken ? 4 : a.block_shift, tiles, wave, waves);
    const Cache8Rows& r = a.rows;
    const Unit& u = s.u;
    const int t0 = max(u.start, 0);              // tokens [t0, len) are written
    auto is_new = [&](int t) { return t >= t0 && t < u.len; };

    // rows: x of K, access i and channel kc + e at 8 i + e; of V, token vt + j and channel vc + c at 2 j + c
    Raw8<E> kraw[kAcc];
    E vraw[kX];
#pragma unroll
    for (int i = 0; i < kAcc; ++i) kraw[i] = Raw8<E>{};
#pragma unroll
    for (int i = 0; i < kX; ++i) vraw[i] = 0;
    if (u.seq >= 0) {
        const E* k = (const E*)a.k_rows + (int64_t)s.head * D + at.kc;
        const E* v = (const E*)a.v_rows + (int64_t)s.head * D + at.vc;
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int t = s.tile + i * Lane::kRows + at.kt;
            if (is_new(t)) kraw[i] = ld8s<E, 1>(k + (u.row + (t - u.start)) * a.k_row_stride);
        }
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
            const int t = s.tile + at.vt + j;
            if (is_new(t)) __builtin_memcpy(vraw + 2 * j, __builtin_assume_aligned(v + (u.row + (t - u.start)) * a.v_row_stride, 2 * sizeof(E)),
                                            2 * sizeof(E));
        }
    }
    const bool busy = s.page >= 0 && s.page < a.num_pages;
    const int in_page = s.tile & ((1 << r.page_shift) - 1);
    const int64_t head_at = (int64_t)s.page * a.page_stride + (((int64_t)s.head << r.page_shift) + in_page) * D;
    const int64_t scale_at = (int64_t)s.page * a.scale_stride + ((int64_t)s.head << (r.page_shift - a.block_shift)) +
                             (in_page >> a.block_shift);
    uint8_t* const kp = a.k_pages + head_at + at.kt * D + at.kc;             // access i: i * kRows * D further
    uint8_t* const vp = a.v_pages + head_at + at.vc * kTileTokens + at.vt;   // the second channel: kTileTokens further
    const bool keeps = !kToken && busy && u.first < t0;      // tokens of the unit stay from before
    const bool merge = busy && s.tile < u.len && (s.tile < t0 || s.tile + kTileTokens > u.len);      // bytes of V that stay
    // earlier codes, which the scales decide about
    float kold = 0.f, vold = 0.f;
    uint2 kwas[kAcc];
    uint32_t vwas[2][kTok / 4];
    if (keeps) {
        kold = a.k_scales[scale_at];
        vold = a.v_scales[scale_at];
#pragma unroll
        for (int i = 0; i < kAcc; ++i)
            if (s.tile + i * Lane::kRows + at.kt < t0) kwas[i] = *reinterpret_cast<const uint2*>(kp + i * Lane::kRows * D);
    }
    if (merge) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int g = 0; g < kTok / 8; ++g) {
                const uint2 w = *reinterpret_cast<const uint2*>(vp + c * kTileTokens + 8 * g);
                vwas[c][2 * g] = w.x;
                vwas[c][2 * g + 1] = w.y;
            }
    }
    float kx[kX], vx[kX];
#pragma unroll
    for (int i = 0; i < kAcc; ++i) to_f32(kraw[i], kx + 8 * i);
#pragma unroll
    for (int i = 0; i < kX; ++i) {
        if constexpr (sizeof(E) == 2) vx[i] = bf16_val(vraw[i]);
        else vx[i] = vraw[i];
    }

    // infinities and NaN among the wave's values, which do not count for a scale: rare, and handled apart
    float poison = 0.f;
#pragma unroll
    for (int i = 0; i < kX; ++i) poison = __builtin_fmaf(kx[i], 0.f, __builtin_fmaf(vx[i], 0.f, poison));
    const bool odd = __any(poison != 0.f);
    auto magnitude = [](auto odd_c, float x) {
        return decltype(odd_c)::value ? finite_magnitude(x) : __float_as_uint(x) & 0x7fffffffu;
    };
    auto either = [&](auto f) {
        if (odd) f(std::true_type{});
        else f(std::false_type{});
    };

    float kratio = 1.f, vratio = 1.f;            // old scale / new
    float kinv[kToken ? kAcc : 1], vinv[kToken ? kTok : 1];      // 1 / scale
    auto inverse = [](float scale) { return scale > 0.f ? 1.f / scale : 0.f; };
    if constexpr (!kToken) {
        uint32_t km = 0, vm = 0;
        either([&](auto o) {
#pragma unroll
            for (int i = 0; i < kX; ++i) {
                km = max(km, magnitude(o, kx[i]));
                vm = max(vm, magnitude(o, vx[i]));
            }
        });
        km = wave_max(km);
        vm = wave_max(vm);
        if (tiles > 1) {
            asm volatile("" ::"v"(kold), "v"(vold));     // every wave has the old scales before one writes the new
            if (lane == 0) {
                tops[0][wave] = km;
                tops[1][wave] = vm;
            }
            __syncthreads();
            for (int w = wave / tiles * tiles; w < (wave / tiles + 1) * tiles; ++w) {
                km = max(km, tops[0][w]);
                vm = max(vm, tops[1][w]);
            }
        }
        const float kt = __uint_as_float(km), vt = __uint_as_float(vm);
        const float kscale = keeps ? joined_scale<kInt8>(kold, kt, kratio) : fresh_scale<kInt8>(kt);
        const float vscale = keeps ? joined_scale<kInt8>(vold, vt, vratio) : fresh_scale<kInt8>(vt);
        kinv[0] = inverse(kscale);
        vinv[0] = inverse(vscale);
        if (busy && wave % tiles == 0 && lane == 0) {
            a.k_scales[scale_at] = kscale;
            a.v_scales[scale_at] = vscale;
        }
    } else {
        uint32_t top[kTok], row[kAcc];
        either([&](auto o) {
#pragma unroll
            for (int i = 0; i < kAcc; ++i) {
                row[i] = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) row[i] = max(row[i], magnitude(o, kx[8 * i + e]));
            }
#pragma unroll
            for (int j = 0; j < kTok; ++j) top[j] = max(magnitude(o, vx[2 * j]), magnitude(o, vx[2 * j + 1]));
        });
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            uint32_t m = row[i];
#pragma unroll
            for (int d = 1; d < Lane::kRow; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
            const float scale = fresh_scale<kInt8>(__uint_as_float(m));
            kinv[i] = inverse(scale);
            const int tt = i * Lane::kRows + at.kt;
            if (busy && at.kc == 0 && is_new(s.tile + tt)) a.k_scales[scale_at + tt] = scale;
        }
        // the lanes of a token of V: halving the tokens that a lane keeps, then the lanes left with one
        int kept = 0;
#pragma unroll
        for (int n = kTok / 2, d = 1; n >= 1; n >>= 1, d <<= 1) {
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
        for (int d = kTok; d < (D == 64 ? 32 : 64); d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
        const float scale = fresh_scale<kInt8>(__uint_as_float(m));
        const int tt = at.vt + kept;
        if ((lane & (D == 64 ? 31 : 63)) < kTok) {
            vsc[wave][tt] = inverse(scale);
            if (busy && is_new(s.tile + tt)) a.v_scales[scale_at + tt] = scale;
        }
        lds_reads_done();                        // and writes
#pragma unroll
        for (int j = 0; j < kTok; ++j) vinv[j] = vsc[wave][at.vt + j];
    }
    if (!busy || s.tile >= u.len) return;

    // the earlier codes of a word in steps of the new scale
    auto again = [](uint32_t was, float ratio) {
        float f[4];
        decode4<kInt8>(was, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] *= ratio;
        return encode4_any<kInt8>(f);
    };
    either([&](auto o) {
        auto encode = [](const float* f) { return decltype(o)::value ? encode4_any<kInt8>(f) : encode4<kInt8>(f); };
#pragma unroll
        for (int i = 0; i < kAcc; ++i) {
            const int t = s.tile + i * Lane::kRows + at.kt;
            if (!is_new(t)) continue;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = kx[8 * i + e] * kinv[kToken ? i : 0];
            *reinterpret_cast<uint2*>(kp + i * Lane::kRows * D) = make_uint2(encode(f), encode(f + 4));
        }
    });
    if (keeps && kratio != 1.f) {
#pragma unroll
        for (int i = 0; i < kAcc; ++i)
            if (s.tile + i * Lane::kRows + at.kt < t0)
                *reinterpret_cast<uint2*>(kp + i * Lane::kRows * D) = make_uint2(again(kwas[i].x, kratio), again(kwas[i].y, kratio));
    }
    if (s.tile + kTileTokens <= t0 && vratio == 1.f) return;
    // V: a channel's tokens are neighbours
    uint32_t c[2][kTok / 4];
    either([&](auto o) {
        auto encode = [](const float* f) { return decltype(o)::value ? encode4_any<kInt8>(f) : encode4<kInt8>(f); };
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
            for (int g = 0; g < kTok / 4; ++g) {
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = vx[2 * (4 * g + e) + ch] * vinv[kToken ? 4 * g + e : 0];
                c[ch][g] = encode(f);
            }
    });
    if (merge) {
#pragma unroll
        for (int ch = 0; ch < 2; ++ch)
#pragma unroll
            for (int g = 0; g < kTok / 4; ++g) {
                const uint32_t was = vwas[ch][g], kept = vratio != 1.f ? again(was, vratio) : was;
                uint32_t now = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = s.tile + at.vt + 4 * g + e;
                    now |= (t < t0 ? kept : t < u.len ? c[ch][g] : was) & (0xffu << (8 * e));
                }
                c[ch][g] = now;
            }
    }
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
        if constexpr (D == 64) *reinterpret_cast<uint2*>(vp + ch * kTileTokens) = make_uint2(c[ch][0], c[ch][1]);
        else *reinterpret_cast<uint4*>(vp + ch * kTileTokens) = make_uint4(c[ch][0], c[ch][1], c[ch][kTok / 4 - 2], c[ch][kTok / 4 - 1]);
    }
}

// ---------------------------------------------------------------- read
template <typename E, int D, bool kInt8>
__global__ __launch_bounds__(256) void cache8_read_kernel(Cache8Args a) {
    using Lane = Lane8<D>;
    constexpr int kAcc = Lane::kAcc, kTok = Lane::kTok;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Lane at(lane);
    const Share s = find_share(a, 4, 1, wave, 4);
    const Cache8Rows& r = a.rows;
    const Unit& u = s.u;
    if (u.seq < 0) return;
    const int page = min(max(s.page, 0), a.num_pages - 1);
    const int t0 = max(u.start, 0);
    auto is_asked = [&](int t) { return t >= t0 && t < u.len; };
    const int in_page = s.tile & ((1 << r.page_shift) - 1);
    const int64_t head_at = (int64_t)page * a.page_stride + (((int64_t)s.head << r.page_shift) + in_page) * D;
    const int64_t scale_at = (int64_t)page * a.scale_stride + ((int64_t)s.head << (r.page_shift - a.block_shift)) +
                             (in_page >> a.block_shift);
    const int bs = a.block_shift;                // 0 or at least 4: a tile has one scale, or 16
    uint2 kc[kAcc];
    uint32_t vc[2][kTok / 4];
    float ks[kAcc], vs[kTok];
    const uint8_t* kp = a.k_pages + head_at + at.kt * D + at.kc;
    const uint8_t* vp = a.v_pages + head_at + at.vc * kTileTokens + at.vt;
#pragma unroll
    for (int i = 0; i < kAcc; ++i) {
        kc[i] = *reinterpret_cast<const uint2*>(kp + i * Lane::kRows * D);
        ks[i] = a.k_scales[scale_at + ((i * Lane::kRows + at.kt) >> bs)];
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int g = 0; g < kTok / 8; ++g) {
            const uint2 w = *reinterpret_cast<const uint2*>(vp + c * kTileTokens + 8 * g);
            vc[c][2 * g] = w.x;
            vc[c][2 * g + 1] = w.y;
        }
#pragma unroll
    for (int j = 0; j < kTok; ++j) vs[j] = a.v_scales[scale_at + ((at.vt + j) >> bs)];
    E* k = (E*)a.k_rows + (int64_t)s.head * D + at.kc;
    E* v = (E*)a.v_rows + (int64_t)s.head * D + at.vc;
#pragma unroll
    for (int i = 0; i < kAcc; ++i) {
        const int t = s.tile + i * Lane::kRows + at.kt;
        float f[8];
        decode4<kInt8>(kc[i].x, f);
        decode4<kInt8>(kc[i].y, f + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= ks[i];
        if (is_asked(t)) st8s<E, 2>(k + (u.row + (t - u.start)) * a.k_row_stride, from_f32<E>(f));
    }
#pragma unroll
    for (int g = 0; g < kTok / 4; ++g) {
        float f[2][4];
        decode4<kInt8>(vc[0][g], f[0]);
        decode4<kInt8>(vc[1][g], f[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 4 * g + e, t = s.tile + at.vt + j;
            if (!is_asked(t)) continue;
            E* p = v + (u.row + (t - u.start)) * a.v_row_stride;
            const float y0 = f[0][e] * vs[j], y1 = f[1][e] * vs[j];
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
    const int64_t tasks = a.units * a.Hkv, blocks = (tasks + waves / tiles - 1) / (waves / tiles);
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
