// rotary.hip -- rotary positions of q and k rows (lfm2sc_rotary), forward and gradient.
//
// A pair (x, y) of a head's columns turns by a = position * freq:
//   (x, y) -> m (x cos a - y sin a, y cos a + x sin a),   gradient: sin a -> -sin a.
// A stream of rows: 2 x 2 bytes a bf16 element for 3 flops.  A row's angles serve all of its heads, so a wave takes
// one row (few rows: part of one): it issues the row's loads, forms the row's cos and sin in LDS while they are
// under way, and turns 16 elements a lane, two 16-byte accesses each way.
//
// Angles are reduced in 64 bits: position * freq loses the fraction of a turn in 32 bits from some thousands of
// positions on.  The remainder, at most an eighth of a turn, goes through the Taylor polynomials of sin and cos in
// fp32 (truncated below 2^-28).
//
// Measured (one MI355X; copies reach 5.1 TB/s): 8 x <= 2048 packed rows of 40 heads of 64 16.8 us (4.6 TB/s), 32768
// rows of 18 heads of 128, half of each interleaved, 50 us (rows of a call fit the last cache in part), the gradient of
// 13 x <= 1531 fp32 rows of 32 heads of 128 55 us (5.1 TB/s).  One row: 2.6 us, its launch and two reads.
#include "attn_common.hpp"
#include "hybrid.hpp"
#include "seq_find.hpp"

namespace lfm2sc {

constexpr int kRotW = 4;          // waves per workgroup, each with its own rows
constexpr int kRotU = 3;          // items whose loads a lane has in flight

// (cos, sin) of 2 pi (position * freq / 2 pi)
__device__ __forceinline__ float2 cos_sin(int position, float freq) {
    constexpr double kTurn = 0.15915494309189533576888;              // 1 / (2 pi)
    const double turns = (double)position * (double)freq * kTurn;
    const double quarters = 4.0 * (turns - __builtin_rint(turns));
    const double q = __builtin_rint(quarters);
    const float x = (float)((quarters - q) * 1.57079632679489661923);
    const int n = (int)q & 3;
    const float y = x * x;
    const float s = x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880))));
    const float c = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320 + y * (-1.f / 3628800)))));
    const float co = n & 1 ? s : c, si = n & 1 ? c : s;
    return make_float2(n == 1 || n == 2 ? -co : co, n >= 2 ? -si : si);
}

// The row's position; false: the row belongs to no sequence.
__device__ __forceinline__ bool row_position(const RotaryRows& a, int64_t row, int& position) {
    if (a.cu == nullptr) {
        position = a.positions[row];
        return true;
    }
    const SeqAt s = find_seq(a.cu, a.positions, a.N, [&](int, int at) { return at <= row; });
    position = (int)(row - max(s.begin, 0)) + s.extra;       // offsets count as clamped to [0, T]
    return row >= s.begin && row < s.end;
}

// How a layout falls into runs of 8 elements.  kAligned: every run is 16-byte aligned.  The others (half layout, R / 2 no
// multiple of 8) begin at any element.  kOverlap: the last run of a part begins early enough to be whole, so that some
// elements are computed and written twice, the same both times; not in place, where they may be rotated already.
// kShort: it has fewer elements, one access each (32768 rows of 18 heads of 128 with R = 100: 105 us, kOverlap 66).
// Runs off their alignment cost more the odder they lie, out of place (kOverlap; R = 12 kShort) and in place (kShort), us:
// R = 100 of 128 68 and 88, 126 148 and 143; 58 of 64 168 and 142, 12 159 and 113; 20 of 80 61 and 82; aligned, 64 of 128,
// 69 and 37.  A copy of those rows takes 59.
enum Runs { kAligned, kOverlap, kShort };

// n elements of a row: 8 or none, or for kShort any number up to 8.
template <typename E, int kRuns>
__device__ __forceinline__ Raw8<E> load_run(const E* p, int n) {
    Raw8<E> r{};
    if (n == 8) {
        if constexpr (kRuns == kAligned) r = ld8<E>(p);
        else __builtin_memcpy(&r, p, sizeof(r));
    } else if constexpr (kRuns == kShort) {
        E e[8] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) e[j] = p[j];
        __builtin_memcpy(&r, e, sizeof(r));
    }
    return r;
}
template <typename E, int kRuns>
__device__ __forceinline__ void store_run(E* p, int n, const Raw8<E>& r) {
    if (n == 8) {
        if constexpr (kRuns == kAligned) st8s<E, 2>(p, r);
        else __builtin_memcpy(p, &r, sizeof(r));
    } else if constexpr (kRuns == kShort) {
        E e[8];
        __builtin_memcpy(e, &r, sizeof(r));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = e[j];
    }
}

// A lane's item is two runs of up to 8 elements of one head, chosen so that neighbouring lanes' runs are neighbours
// (a lane with 16 neighbouring elements would use half of each line an access touches).  Half layout: columns c and R / 2 + c
// of the R rotated ones, then of the columns from R on one of either half; interleaved: a run of either half of the columns.
//
// Rows are stored past the caches' reach (nt) and read as usual: read nt too, 8 prompts take 20.3 instead of 16.8 us and
// 16384 rows 40 instead of 33 us; stored as usual, 65536 rows of 40 heads of 64 gain (144 -> 128 us: a run of R = 64 is half
// a line), everything else loses (32768 interleaved 50 -> 61 us).  Lanes trading runs so that a store fills its lines
// cost more than they gained (8 prompts 16.8 -> 27.5 us).
template <typename E, bool kInterleaved, int kRuns>
__global__ __launch_bounds__(64 * kRotW) void rotary_kernel(RotaryArgs<E> a) {
    __shared__ float2 table[kRotW][kRotaryMaxD / 2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t unit = blockIdx.x * (uint32_t)kRotW + (uint32_t)wave;       // < 2^26, see the launcher
    const int64_t row = unit / (uint32_t)a.parts;
    if (row >= a.r.T) return;
    const int R = a.R, half = R / 2, full = half / 8, tail = kRuns == kAligned ? 0 : 1;
    const int first = (int)(unit % (uint32_t)a.parts) * a.part_items, last = min(first + a.part_items, a.items);
    const uint32_t per_head = (uint32_t)a.per_head;
    float2* cs = table[wave];

    struct Item {
        const E* src;
        E* dst;
        int c[2], n[2], pair[2];     // pair: number of the first pair, of each run (half layout: of both; -1: columns that stay)
    };
    auto item = [&](int i) {
        Item x;
        const int head = (int)((uint32_t)i / per_head), j = i - head * (int)per_head;
        const bool k = head >= a.Hq;
        x.src = (k ? a.k + row * a.k_stride : a.q + row * a.q_stride) + (int64_t)(k ? head - a.Hq : head) * a.D;
        x.dst = (k ? a.k_out + row * a.k_out_stride : a.q_out + row * a.q_out_stride) + (int64_t)(k ? head - a.Hq : head) * a.D;
        if constexpr (kInterleaved) {
            x.c[0] = 8 * j;
            x.c[1] = 8 * (j + (int)per_head);
            x.n[0] = 8;
            x.n[1] = x.c[1] < a.D ? 8 : 0;
            x.pair[0] = x.c[0] / 2;
            x.pair[1] = x.c[1] / 2;
        } else if (j < full + tail) {
            x.pair[0] = kRuns == kOverlap ? min(8 * j, half - 8) : 8 * j;
            x.c[0] = x.pair[0];
            x.c[1] = half + x.pair[0];
            x.n[0] = x.n[1] = kRuns == kShort ? min(8, half - 8 * j) : 8;
        } else {
            const int m = j - full - tail;
            x.c[0] = R + 8 * m;
            x.c[1] = x.c[0] + 8 * ((int)per_head - full - tail);
            x.n[0] = kRuns == kShort ? min(8, a.D - x.c[0]) : 8;
            x.n[1] = kRuns == kShort ? max(0, min(8, a.D - x.c[1])) : x.c[1] < a.D ? 8 : 0;
            if (kRuns == kOverlap) {
                x.c[0] = min(x.c[0], a.D - 8);
                x.c[1] = min(x.c[1], a.D - 8);
            }
            x.pair[0] = -1;
        }
        return x;
    };

    bool ready = false;
    for (int i0 = first; i0 < last; i0 += 64 * kRotU) {
        Item x[kRotU];
        Raw8<E> v[kRotU][2];
#pragma unroll
        for (int u = 0; u < kRotU; ++u) {
            x[u] = item(min(i0 + u * 64 + lane, last - 1));
#pragma unroll
            for (int s = 0; s < 2; ++s) v[u][s] = load_run<E, kRuns>(x[u].src + x[u].c[s], x[u].n[s]);
        }
        if (!ready) {                                        // the first loads are under way
            ready = true;
            int position = 0;
            if (!row_position(a.r, row, position)) return;
            for (int p = lane; p < half; p += 64) {
                const float2 t = cos_sin(position, a.freqs[p]);
                cs[p] = make_float2(a.magnitude * t.x, a.turn * t.y);
            }
            lds_reads_done();                                // and writes: the wave reads what other lanes wrote
        }
#pragma unroll
        for (int u = 0; u < kRotU; ++u) {
            float f[2][8];
            to_f32(v[u][0], f[0]);
            to_f32(v[u][1], f[1]);
            if constexpr (kInterleaved) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int at = x[u].pair[s] + p;
                        const float2 t = cs[min(at, half - 1)];
                        const float b = f[s][2 * p], c = f[s][2 * p + 1];
                        const bool turns = at < half;
                        f[s][2 * p] = turns ? __builtin_fmaf(b, t.x, -c * t.y) : b;
                        f[s][2 * p + 1] = turns ? __builtin_fmaf(c, t.x, b * t.y) : c;
                    }
            } else {
                const bool turns = x[u].pair[0] >= 0;
                const int p0 = turns ? x[u].pair[0] : 0;
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    const float2 t = cs[kRuns == kShort ? min(p0 + p, half - 1) : p0 + p];
                    const float b = f[0][p], c = f[1][p];
                    f[0][p] = turns ? __builtin_fmaf(b, t.x, -c * t.y) : b;
                    f[1][p] = turns ? __builtin_fmaf(c, t.x, b * t.y) : c;
                }
            }
            if (i0 + u * 64 + lane < last) {
#pragma unroll
                for (int s = 0; s < 2; ++s) store_run<E, kRuns>(x[u].dst + x[u].c[s], x[u].n[s], from_f32<E>(f[s]));
            }
        }
    }
}

template <typename E>
hipError_t launch_rotary(RotaryArgs<E> a, bool interleaved, hipStream_t s) {
    const int half = a.R / 2;
    const bool in_place = (const E*)a.q_out == a.q || (a.Hkv > 0 && (const E*)a.k_out == a.k);
    const bool all_in_place = (const E*)a.q_out == a.q && (a.Hkv == 0 || (const E*)a.k_out == a.k);
    const int runs = interleaved || half % 8 == 0                                              ? kAligned
                     : !in_place && half >= 8 && (a.D == a.R || a.D - a.R >= 8) ? kOverlap
                                                                                : kShort;
    const int rest = all_in_place ? 0 : (a.D - a.R + 15) / 16;       // in place, the columns that stay are there
    a.per_head = interleaved ? ((all_in_place ? a.R : a.D) + 15) / 16 : half / 8 + (runs != kAligned ? 1 : 0) + rest;
    a.items = a.per_head * (a.Hq + a.Hkv);
    // few rows: a row's items go to several waves, so that the card has 2048 of them
    const int64_t want = 2048 / a.r.T, most = (a.items + 63) / 64;
    a.parts = (int)(want < 1 ? 1 : want < most ? want : most);
    a.part_items = ((a.items + a.parts - 1) / a.parts + 63) / 64 * 64;
    a.parts = (a.items + a.part_items - 1) / a.part_items;
    const int64_t blocks = (a.r.T * a.parts + kRotW - 1) / kRotW;
    if (too_many(blocks, 64 * kRotW)) return hipErrorInvalidConfiguration;
    const dim3 grid((uint32_t)blocks), block(64 * kRotW);
    if (interleaved) hipLaunchKernelGGL((rotary_kernel<E, true, kAligned>), grid, block, 0, s, a);
    else if (runs == kAligned) hipLaunchKernelGGL((rotary_kernel<E, false, kAligned>), grid, block, 0, s, a);
    else if (runs == kOverlap) hipLaunchKernelGGL((rotary_kernel<E, false, kOverlap>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rotary_kernel<E, false, kShort>), grid, block, 0, s, a);
    return hipGetLastError();
}
template hipError_t launch_rotary<uint16_t>(RotaryArgs<uint16_t>, bool, hipStream_t);
template hipError_t launch_rotary<float>(RotaryArgs<float>, bool, hipStream_t);

}  // namespace lfm2sc
