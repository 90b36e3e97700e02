// attn_common.hpp -- pieces shared by the attention kernels (bf16 in and out,
// fp32 sums, head dimension D = 64 or 128).
//
// All products run on v_mfma_f32_32x32x16_bf16.  A lane (c = lane & 31, half
// h = lane >> 5) holds of its operands
//   A[m = c][k = 8 h + j],  B[k = 8 h + j][n = c],  j = 0..7,
// and of the result
//   C[m = 4 h + (i & 3) + 8 (i >> 2)][n = c],  i = 0..15.
// The sum over k does not care in which order k runs, as long as A and B agree.
// So a result block converted to bf16 is at once the B operand of a following
// product over its rows m, without leaving its registers: elements
// i = 8 t .. 8 t + 7 of half h are the rows
//   16 t + 4 h + {0..3}, 16 t + 8 + 4 h + {0..3}
// of 16-row step t, and the A operand of that product takes its k in the same
// order (two transposing LDS reads of 4 rows each).
#pragma once

#include "fused_common.hpp"

namespace lfm2sc {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -__builtin_inff();

// How far (log2) a row's maximum may pass the reference m of its softmax before
// the reference moves: most tiles then rescale nothing, and p stays below
// 2^kLazy, whose bf16 and fp32 values are as exact as those below 1.
constexpr float kLazy = 8.f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The value of the lane 32 away, for a reduction over both halves of a wave.
__device__ __forceinline__ float max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Elements 8 t .. 8 t + 7 of a result block, rounded to bf16 (RNE): the B
// operand of step t of the product over the block's rows.
__device__ __forceinline__ bf16x8 to_operand(const f32x16& x, int t) {
    union { uint32_t u[4]; bf16x8 v; } r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.u[j] = Elem<uint16_t>::pack2(x[8 * t + 2 * j], x[8 * t + 2 * j + 1]);
    return r.v;
}

// A staged tile: rows of D bf16 values in LDS, 16-byte chunk c of row r at
// position c ^ rot(r).  Two access patterns have to reach all 64 banks:
//   * 16 lanes of a 16-byte read: 16 consecutive rows, one chunk;
//   * 32 lanes of a transposing 8-byte read: 4 consecutive rows, 4 consecutive
//     (aligned) chunks, of which each lane takes 8 bytes.
// The rows' low bits therefore go to the chunk's high bits.
template <int D>
struct Tile {
    static_assert(D == 64 || D == 128, "head dimension");
    static constexpr int kRowB = 2 * D;
    static constexpr int kChunks = kRowB / 16;
    static constexpr int kRowsPerDma = 1024 / kRowB;       // rows of one 64-lane x 16-byte copy to LDS
    __host__ __device__ static constexpr int rot(int r) {
        if (D == 64) {
            const int x = (r >> 1) & 7;
            return ((x & 1) << 2) | (x & 2) | (x >> 2);
        }
        return ((r & 3) << 2) | ((r >> 2) & 3);
    }
    __device__ static uint32_t at(int r, int c) { return (uint32_t)(r * kRowB + ((c ^ rot(r)) << 4)); }
};

// Offsets of a lane's operands within a staged tile.  rot() repeats after 16
// rows, so whole 16-row steps are plain byte offsets.
template <int D>
struct LaneOffsets {
    uint32_t row[D / 16];        // row operand: rows c (+ 32 b), values 16 s + 8 h ..
    uint32_t tr[2][D / 32];      // transposed operand: rows 4 h + .. (+ 8), column block of 32 values
    __device__ explicit LaneOffsets(int lane) {
        const int c = lane & 31, h = lane >> 5, g = (lane >> 4) & 1, i = lane & 15;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) row[s] = Tile<D>::at(c, 2 * s + h);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int b = 0; b < D / 32; ++b)
                tr[j][b] = Tile<D>::at(8 * j + 4 * h + (i >> 2), 4 * b + 2 * g + ((i & 3) >> 1)) + 8 * (i & 1);
    }
};

__device__ __forceinline__ bf16x8 lds_row(const uint8_t* tile, uint32_t off) {
    return *reinterpret_cast<const bf16x8*>(tile + off);
}

// A operand A[m = column][k = row] of a row-major tile: for each of 16 lanes,
// ds_read_b64_tr_b16 hands lane i column i of the 4 rows x 16 columns that the
// 16 lanes address (lane i: 4 values of row i >> 2, columns 4 (i & 3) ..).
__device__ __forceinline__ bf16x8 lds_transposed(const uint8_t* tile, uint32_t off0, uint32_t off1) {
    typedef __attribute__((address_space(3))) s16x4* p4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((p4)(tile + off0));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((p4)(tile + off1));
    const s16x8 r = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, r);
}

// The wave's LDS reads have returned.  A copy to LDS is not ordered behind reads
// issued before it, neither by the compiler nor by the hardware: a wave that
// refills a tile which it has just read waits here first.  (Slots shared by a
// workgroup are refilled behind a barrier, before which every read was consumed.)
__device__ __forceinline__ void lds_reads_done() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((63 & 15) | (7 << 4) | (0 << 8) | ((63 >> 4) << 14));   // lgkmcnt(0)
    asm volatile("" ::: "memory");
}

// Copies of R-row tiles (row r at byte (r * stride) * 2 from the tile's first
// row) to LDS, kDma KiB per wave; rows at or beyond the given count read as
// zeros (the buffer's range check).
template <int D, int W, int R = 64>
struct TileCopy {
    using T = Tile<D>;
    static constexpr int kDma = R * T::kRowB / 1024 / W;
    static_assert(kDma * W * 1024 == R * T::kRowB, "whole copies");
    uint32_t off[kDma];
    __device__ TileCopy(int wave, int lane, int64_t stride) {
#pragma unroll
        for (int i = 0; i < kDma; ++i) {
            const int r = (wave * kDma + i) * T::kRowsPerDma + lane / T::kChunks;
            off[i] = (uint32_t)(r * (int)stride * 2 + ((lane % T::kChunks) ^ T::rot(r)) * 16);
        }
    }
    // p: the tile's first row; rows >= 1 (uniform)
    __device__ void operator()(const uint16_t* p, int64_t stride, int rows, uint8_t* lds, int wave) const {
        const rsrc_t r = row_rsrc(p, __builtin_amdgcn_readfirstlane((uint32_t)(((rows - 1) * (int)stride + D) * 2)));
#pragma unroll
        for (int i = 0; i < kDma; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(lds + (wave * kDma + i) * 1024), 16, off[i], 0, 0, 0);
    }
};

// A ring of S (2 or 3) staged tiles: step(IC<u>, t) for t = 0 .. n - 1 with u = t % S.  The
// step waits for tile t, meets the workgroup, refills slot (u + S - 1) % S with
// tile min(t + S - 1, n - 1) (always, so that the number of copies in flight at
// every wait is a constant) and computes from slot u.
template <int u, typename T>
__device__ __forceinline__ T* pick_slot(T* a, T* b, T* c) {
    if constexpr (u == 0) return a;
    else if constexpr (u == 1) return b;
    else return c;
}
template <int S, typename F>
__device__ __forceinline__ void for_stages(int n, F step) {
    static_assert(S == 2 || S == 3, "slots");
    for (int t = 0; t < n; t += S) {
        step(IC<0>{}, t);
        if (t + 1 < n) step(IC<1>{}, t + 1);
        if constexpr (S > 2) {
            if (t + 2 < n) step(IC<2>{}, t + 2);
        }
    }
}

// Row operand (B[k = value][n = row]) of row c: values 16 s + 8 h .. of a row in
// global memory; zeros where the row does not exist.
template <int D>
__device__ __forceinline__ void load_row_operand(bf16x8 (&f)[D / 16], const uint16_t* row, int h, bool exists) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (exists) x = *reinterpret_cast<const uint4*>(row + 16 * s + 8 * h);
        f[s] = __builtin_bit_cast(bf16x8, x);
    }
}

// Stores a transposed result (x[db]: values 32 db + 4 h + (i & 3) + 8 (i >> 2)
// of row c), times f and rounded to bf16, as 16-byte pieces of the row: the two
// halves of the wave trade 4-value runs.
template <int D>
__device__ __forceinline__ void store_transposed(uint16_t* row, const f32x16 (&x)[D / 32], float f, int h, bool exists) {
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            const uint32_t a0 = Elem<uint16_t>::pack2(x[db][i] * f, x[db][i + 1] * f);
            const uint32_t a1 = Elem<uint16_t>::pack2(x[db][i + 2] * f, x[db][i + 3] * f);
            const uint32_t b0 = Elem<uint16_t>::pack2(x[db][i + 4] * f, x[db][i + 5] * f);
            const uint32_t b1 = Elem<uint16_t>::pack2(x[db][i + 6] * f, x[db][i + 7] * f);
            const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
            if (exists)
                *reinterpret_cast<uint4*>(row + 32 * db + 2 * i + 8 * h) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
        }
}

// Sum over the wave, the same in every lane (DPP row shifts, then row broadcasts).
__device__ __forceinline__ int wave_sum(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);    // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);    // row_shr:2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);    // row_shr:4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);    // row_shr:8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);    // row_bcast:15
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);    // row_bcast:31
    return __builtin_amdgcn_readlane(x, 63);
}

// Row blocks of packed sequences in order of falling work.  A sequence of len
// rows has nb = ceil(len / rows) blocks; rank r = 1 .. nb counts them from the
// end that costs least (forward: rank = block + 1, the keys it sees; key blocks
// of the backward: rank = nb - block, the queries that see it).  The tile-th
// block overall is found from F(r) = sum_i max(0, nb_i - r), the number of
// blocks of a rank above r: a binary search over r, all lanes of the wave
// summing over the sequences, 64 at a time.  Row offsets are clamped to
// [0, total_T].  len == 0: no such block.  Wave-uniform.
//
// Handing out the heaviest blocks first, whatever their sequence, keeps a long
// sequence at the end of the batch from running on alone.
struct SeqTile {
    int64_t start;    // first packed row of the sequence
    int len;          // its length
    int rank;         // 1 .. ceil(len / rows)
};
struct SeqRange {
    int start, len;
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* __restrict__ cu, int s, int N, int64_t total_T) {
    if (s >= N) return SeqRange{0, 0};
    const int64_t lo = min(max((int64_t)cu[s], (int64_t)0), total_T);
    const int64_t hi = min(max((int64_t)cu[s + 1], (int64_t)0), total_T);
    return SeqRange{(int)lo, hi > lo ? (int)(hi - lo) : 0};
}
__device__ __forceinline__ SeqTile find_seq_tile(const int32_t* __restrict__ cu, int N, int64_t total_T, int tile,
                                                 int rows) {
    const int lane = threadIdx.x & 63;
    const SeqRange own = seq_range(cu, lane, N, total_T);        // sequences 0 .. 63
    const int nb = (own.len + rows - 1) / rows;
    if (N == 1) {
        const int all = __builtin_amdgcn_readfirstlane(nb);
        if (tile >= all) return SeqTile{0, 0, 0};
        return SeqTile{__builtin_amdgcn_readfirstlane(own.start), __builtin_amdgcn_readfirstlane(own.len), all - tile};
    }
    auto above = [&](int r) {
        int n = max(nb - r, 0);
        for (int s = 64 + lane; s < N; s += 64) n += max((seq_range(cu, s, N, total_T).len + rows - 1) / rows - r, 0);
        return wave_sum(n);
    };
    if (tile >= above(0)) return SeqTile{0, 0, 0};
    int lo = 0, hi = 1;                          // F(lo) > tile >= F(hi)
    int at = above(1);
    while (at > tile) {
        lo = hi;
        hi *= 2;
        at = above(hi);
    }
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1, f = above(mid);
        if (f > tile) lo = mid;
        else {
            hi = mid;
            at = f;
        }
    }
    int left = tile - at;                        // which of the sequences with a block of rank hi
    for (int s0 = 0; s0 < N; s0 += 64) {
        const SeqRange x = s0 == 0 ? own : seq_range(cu, s0 + lane, N, total_T);
        const bool has = (x.len + rows - 1) / rows >= hi;
        const uint64_t which = __ballot(has);
        const int count = __popcll(which);
        if (left < count) {
            const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(which >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)which, 0));
            const int l = __builtin_ctzll(__ballot(has && before == left));
            return SeqTile{__builtin_amdgcn_readlane(x.start, l), __builtin_amdgcn_readlane(x.len, l), hi};
        }
        left -= count;
    }
    return SeqTile{0, 0, 0};
}

}  // namespace lfm2sc
