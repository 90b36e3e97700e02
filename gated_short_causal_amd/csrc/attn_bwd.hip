// attn_bwd.hip -- backward of the causal attention over packed prompts.
//
// With p = exp(scale s - lse) and delta[t] = sum_d dout[t][d] out[t][d]:
//   dv[j] = sum_t p[t][j] dout[t]        ds[t][j] = p[t][j] (dout[t].v[j] - delta[t])
//   dk[j] = scale sum_t ds[t][j] q[t]    dq[t] = scale sum_j ds[t][j] k[j]
// where the sums over t of dk and dv run over every query head of the group.
//
// Two passes over the score blocks, neither with atomics, so the gradients are
// the same bits every time: one by key blocks (dk, dv stay in registers while
// the group's heads and queries stream past), one by query blocks (dq stays,
// keys stream).  Both form p again from q, k and lse: 7 products for the 5 that the
// formulas need (8 where dk and dv go apart).  Per executed product the long case is
// near what a library product reaches (T = 8192, 32 / 8 heads of 64: 889-927 us = 1.04-1.08
// PFLOP/s executed, 0.74-0.77 of the formulas' five); D = 128 waits more (two waves per
// SIMD, 37% of the cycles in the matrix unit).  dq summed with atomics would save
// two products and the bits' order.
//
// Fewer bits: p and ds are operands of a second product and enter it rounded to
// bf16 once (2^-9 of each), and delta takes the output as the caller holds it, in
// bf16.  Gradients are off by 2.5e-3 (relative 2-norm) where their own rounding
// alone gives 1.7e-3; ds in two bf16 parts would need two more products.  p, dp,
// ds up to there, delta and all sums are fp32.
#include "attn_common.hpp"
#include "hybrid.hpp"

namespace lfm2sc {

// delta and lse in base 2, [Hq][total_T] each.  D / 8 lanes hold one head of a
// row; a wave does 8 consecutive rows, after which lane j of those lanes
// (j < 8) writes row j.
template <int D>
__global__ __launch_bounds__(256) void attn_delta_kernel(AttnGradArgs a) {
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 8;
    const int head = blockIdx.y * (64 / kLanes) + lane / kLanes, j = lane % kLanes;
    if (t0 >= a.f.total_T || head >= a.f.Hq) return;
    float mine = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        float s = 0.f;
        if (t0 + r < a.f.total_T) {
            float x[8], y[8];
            load_f32x8<uint16_t>(a.dout + (t0 + r) * a.dout_stride + head * D + 8 * j, x);
            load_f32x8<uint16_t>(a.f.out + (t0 + r) * a.f.out_stride + head * D + 8 * j, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x[i], y[i], s);
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) s += __shfl_xor(s, d, 64);
        if (j == r) mine = s;
    }
    const int64_t t = t0 + j;
    if (j < 8 && t < a.f.total_T) {
        const int64_t at = (int64_t)head * a.f.total_T + t;
        a.delta[at] = mine;
        a.lse2[at] = a.f.lse[at] * kLog2e;
    }
}

// dk (kK) and dv (kV), or one of them: a wave owns 32 keys, a workgroup 32 W
// consecutive ones, for G / splits query heads of the group.  S slots of R-row
// query tiles (q rows, dout rows) and of their lse and delta in LDS.
template <int D, int W, int R, int S, bool kV, bool kK, typename X, typename Y, typename Z>
__device__ __forceinline__ void kv_part(const AttnGradArgs& a, X qslot, Y dslot, Z zslot, int block, int wave, int lane) {
    using T = Tile<D>;
    constexpr int kBN = 32 * W;
    const int c = lane & 31, h = lane >> 5;
    const AttnArgs& f = a.f;
    const int G = f.Hq / f.Hkv / a.splits;       // heads of this workgroup
    const int kvh = block % f.Hkv, split = block / f.Hkv % a.splits;
    const int head0 = (kvh * a.splits + split) * G;
    const SeqTile st = find_seq_tile(f.cu, f.N, f.total_T, block / (f.Hkv * a.splits), kBN);
    if (st.len == 0) return;
    const int n0 = ((st.len + kBN - 1) / kBN - st.rank) * kBN;
    const int wkey = n0 + wave * 32;
    const int first = n0 / R, last = (st.len + R - 1) / R;    // query tiles [first, last) of R rows
    const int per_head = last - first, steps = per_head * G;

    const TileCopy<D, W, R> qcopy(wave, lane, f.q_stride), dcopy(wave, lane, a.dout_stride);
    auto issue = [&](uint8_t* qb, uint8_t* db, float* zb, int step) {
        step = min(step, steps - 1);
        const int head = head0 + step / per_head, t = first + step % per_head;
        const int rows = min(R, st.len - t * R);
        const int64_t row = st.start + (int64_t)t * R;
        qcopy(f.q + row * f.q_stride + (int64_t)head * D, f.q_stride, rows, qb, wave);
        dcopy(a.dout + row * a.dout_stride + (int64_t)head * D, a.dout_stride, rows, db, wave);
        // every wave brings its own copy of the rows' lse and delta (64 of each; those past the rows read as 0)
        const int64_t at = (int64_t)head * f.total_T + row;
        float* z = zb + wave * 128;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(row_rsrc(a.lse2 + at, rows * 4), (lds_ptr_t)z, 4, lane * 4, 0, 0, 0);
        if constexpr (kK)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(row_rsrc(a.delta + at, rows * 4), (lds_ptr_t)(z + 64), 4, lane * 4, 0, 0, 0);
    };
    constexpr int kPer = 2 * decltype(qcopy)::kDma + (kK ? 2 : 1);       // copies of a tile per wave
    issue(qslot(IC<0>{}), dslot(IC<0>{}), zslot(IC<0>{}), 0);
    if constexpr (S > 2) issue(qslot(IC<1>{}), dslot(IC<1>{}), zslot(IC<1>{}), 1);

    bf16x8 kf[D / 16], vf[D / 16];
    const bool exists = wkey + c < st.len;
    const int64_t krow = st.start + wkey + c;
    load_row_operand<D>(kf, f.k + krow * f.k_stride + (int64_t)kvh * D, h, exists);
    if constexpr (kK) load_row_operand<D>(vf, f.v + krow * f.v_stride + (int64_t)kvh * D, h, exists);
    const LaneOffsets<D> lo(lane);
    const float cs = f.scale * kLog2e;
    f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[b][i] = dv[b][i] = 0.f;

    // 32 query rows (n * 32 .. of the tile) against the wave's keys
    auto rows32 = [&](const uint8_t* qb, const uint8_t* db, const float* lb, const float* eb, int n, int r0) {
        f32x16 s, e;
        bf16x8 p[2], g[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = e[i] = 0.f;
#pragma unroll
        for (int ds = 0; ds < D / 16; ++ds) s = mfma32(lds_row(qb + n * 32 * T::kRowB, lo.row[ds]), kf[ds], s);
        if constexpr (kK) {
#pragma unroll
            for (int ds = 0; ds < D / 16; ++ds) e = mfma32(lds_row(db + n * 32 * T::kRowB, lo.row[ds]), vf[ds], e);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 x = *reinterpret_cast<const float4*>(lb + n * 32 + 8 * j + 4 * h);
            s[4 * j] = exp2_fast(__builtin_fmaf(s[4 * j], cs, -x.x));
            s[4 * j + 1] = exp2_fast(__builtin_fmaf(s[4 * j + 1], cs, -x.y));
            s[4 * j + 2] = exp2_fast(__builtin_fmaf(s[4 * j + 2], cs, -x.z));
            s[4 * j + 3] = exp2_fast(__builtin_fmaf(s[4 * j + 3], cs, -x.w));
        }
        if (r0 < wkey + 31) {                    // the first of the rows lies before the wave's last key
            const int key = wkey + c - r0 - 4 * h;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if ((i & 3) + 8 * (i >> 2) < key) s[i] = 0.f;
        }
        if constexpr (kV) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) p[ks] = to_operand(s, ks);
        }
        if constexpr (kK) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 y = *reinterpret_cast<const float4*>(eb + n * 32 + 8 * j + 4 * h);
                e[4 * j] = s[4 * j] * (e[4 * j] - y.x);
                e[4 * j + 1] = s[4 * j + 1] * (e[4 * j + 1] - y.y);
                e[4 * j + 2] = s[4 * j + 2] * (e[4 * j + 2] - y.z);
                e[4 * j + 3] = s[4 * j + 3] * (e[4 * j + 3] - y.w);
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) g[ks] = to_operand(e, ks);
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int at = (n * 32 + ks * 16) * T::kRowB;
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                if constexpr (kV) dv[b] = mfma32(lds_transposed(db + at, lo.tr[0][b], lo.tr[1][b]), p[ks], dv[b]);
                if constexpr (kK) dk[b] = mfma32(lds_transposed(qb + at, lo.tr[0][b], lo.tr[1][b]), g[ks], dk[b]);
            }
        }
    };
    for_stages<S>(steps, [&](auto u, int i) {
        constexpr int refill = (decltype(u)::value + S - 1) % S;
        wait_vm<(S - 2) * kPer>();
        stage_barrier();
        issue(qslot(IC<refill>{}), dslot(IC<refill>{}), zslot(IC<refill>{}), i + S - 1);
        const int t = first + i % per_head;
        const float* z = zslot(u) + wave * 128;
        if (wkey >= st.len) return;
#pragma unroll
        for (int n = 0; n < R / 32; ++n)
            if (t * R + n * 32 + 31 >= wkey) rows32(qslot(u), dslot(u), z, z + 64, n, t * R + n * 32);
    });
    wait_vm<0>();                                // no copy may outlive the workgroup
    if (a.splits == 1) {
        if constexpr (kK) store_transposed<D>(a.dk + krow * a.dk_stride + (int64_t)kvh * D, dk, f.scale, h, exists);
        if constexpr (kV) store_transposed<D>(a.dv + krow * a.dv_stride + (int64_t)kvh * D, dv, 1.f, h, exists);
    } else if (exists) {
        const int64_t one = f.total_T * f.Hkv * D;           // [split][dk, dv][total_T][Hkv * D] fp32
        float* p = a.part + 2 * split * one + (krow * f.Hkv + kvh) * D + 4 * h;
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                float* x = p + 32 * b + 2 * i;
                if constexpr (kK)
                    *reinterpret_cast<float4*>(x) = make_float4(dk[b][i], dk[b][i + 1], dk[b][i + 2], dk[b][i + 3]);
                if constexpr (kV)
                    *reinterpret_cast<float4*>(x + one) = make_float4(dv[b][i], dv[b][i + 1], dv[b][i + 2], dv[b][i + 3]);
            }
    }
}

// Adds up the splits of dk and dv: a workgroup takes 8 rows of a sequence.
template <int D>
__global__ __launch_bounds__(256) void attn_dkv_sum_kernel(AttnGradArgs a) {
    const AttnArgs& f = a.f;
    const SeqTile st = find_seq_tile(f.cu, f.N, f.total_T, blockIdx.x, 8);
    if (st.len == 0) return;
    const int row0 = (st.rank - 1) * 8, rows = min(8, st.len - row0);
    const int per_row = f.Hkv * D / 4;
    const int64_t one = f.total_T * f.Hkv * D;
    for (int i = threadIdx.x; i < rows * per_row; i += 256) {
        const int64_t row = st.start + row0 + i / per_row;
        const int col = i % per_row * 4;
        const float* p = a.part + row * f.Hkv * D + col;
        float4 k = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + one);
        for (int s = 1; s < a.splits; ++s) {
            const float4 x = *reinterpret_cast<const float4*>(p + 2 * s * one);
            const float4 y = *reinterpret_cast<const float4*>(p + (2 * s + 1) * one);
            k.x += x.x; k.y += x.y; k.z += x.z; k.w += x.w;
            v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
        }
        *reinterpret_cast<uint2*>(a.dk + row * a.dk_stride + col) =
            make_uint2(Elem<uint16_t>::pack2(k.x * f.scale, k.y * f.scale), Elem<uint16_t>::pack2(k.z * f.scale, k.w * f.scale));
        *reinterpret_cast<uint2*>(a.dv + row * a.dv_stride + col) =
            make_uint2(Elem<uint16_t>::pack2(v.x, v.y), Elem<uint16_t>::pack2(v.z, v.w));
    }
}

// dq: a wave owns 32 query rows of one head, a workgroup 32 W consecutive ones.
template <int D, int W, int R, int S, typename X, typename Y>
__device__ __forceinline__ void dq_part(const AttnGradArgs& a, X kslot, Y vslot, int block, int wave, int lane) {
    using T = Tile<D>;
    constexpr int kBM = 32 * W;
    const int c = lane & 31, h = lane >> 5;
    const AttnArgs& f = a.f;
    const int G = f.Hq / f.Hkv;
    const int kvh = block % f.Hkv, head = kvh * G + (block / f.Hkv) % G;
    const SeqTile st = find_seq_tile(f.cu, f.N, f.total_T, block / f.Hq, kBM);
    if (st.len == 0) return;
    const int q0 = (st.rank - 1) * kBM;
    const int wrow = q0 + wave * 32;
    const int tiles = (min(q0 + kBM, st.len) + R - 1) / R;

    const uint16_t* kp = f.k + st.start * f.k_stride + (int64_t)kvh * D;
    const uint16_t* vp = f.v + st.start * f.v_stride + (int64_t)kvh * D;
    const TileCopy<D, W, R> kcopy(wave, lane, f.k_stride), vcopy(wave, lane, f.v_stride);
    auto issue = [&](uint8_t* kb, uint8_t* vb, int t) {
        t = min(t, tiles - 1);
        const int rows = min(R, st.len - t * R);
        kcopy(kp + (int64_t)t * R * f.k_stride, f.k_stride, rows, kb, wave);
        vcopy(vp + (int64_t)t * R * f.v_stride, f.v_stride, rows, vb, wave);
    };
    issue(kslot(IC<0>{}), vslot(IC<0>{}), 0);
    if constexpr (S > 2) issue(kslot(IC<1>{}), vslot(IC<1>{}), 1);

    bf16x8 qf[D / 16], df[D / 16];
    const bool exists = wrow + c < st.len;
    const int64_t row = st.start + wrow + c;
    load_row_operand<D>(qf, f.q + row * f.q_stride + (int64_t)head * D, h, exists);
    load_row_operand<D>(df, a.dout + row * a.dout_stride + (int64_t)head * D, h, exists);
    float lse = 0.f, del = 0.f;
    if (exists) {
        lse = a.lse2[(int64_t)head * f.total_T + row];
        del = a.delta[(int64_t)head * f.total_T + row];
    }
    const LaneOffsets<D> lo(lane);
    const float cs = f.scale * kLog2e;
    f32x16 dq[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[x][i] = 0.f;

    auto tile = [&](const uint8_t* kb, const uint8_t* vb, int t) {
#pragma unroll
        for (int n = 0; n < R / 32; ++n) {
            const int k0 = t * R + n * 32;
            if (k0 > wrow + 31) continue;
            f32x16 s, e;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = e[i] = 0.f;
#pragma unroll
            for (int ds = 0; ds < D / 16; ++ds) {
                s = mfma32(lds_row(kb + n * 32 * T::kRowB, lo.row[ds]), qf[ds], s);
                e = mfma32(lds_row(vb + n * 32 * T::kRowB, lo.row[ds]), df[ds], e);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = exp2_fast(__builtin_fmaf(s[i], cs, -lse)) * (e[i] - del);
            if (k0 + 31 > wrow) {
                const int r = wrow + c - k0 - 4 * h;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if ((i & 3) + 8 * (i >> 2) > r) s[i] = 0.f;
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const bf16x8 g = to_operand(s, ks);
                const int at = (n * 32 + ks * 16) * T::kRowB;
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
                    dq[x] = mfma32(lds_transposed(kb + at, lo.tr[0][x], lo.tr[1][x]), g, dq[x]);
            }
        }
    };
    const int last = min(wrow + 32, st.len) - 1;
    for_stages<S>(tiles, [&](auto u, int t) {
        constexpr int refill = (decltype(u)::value + S - 1) % S;
        wait_vm<(S - 2) * 2 * decltype(kcopy)::kDma>();
        stage_barrier();
        issue(kslot(IC<refill>{}), vslot(IC<refill>{}), t + S - 1);
        if (t * R <= last && wrow < st.len) tile(kslot(u), vslot(u), t);
    });
    wait_vm<0>();
    store_transposed<D>(a.dq + row * a.dq_stride + (int64_t)head * D, dq, f.scale, h, exists);
}

// All kinds of workgroup in one launch, the key blocks first: they run longest,
// and the query blocks fill in behind them.  kApart: dk and dv in workgroups of
// their own: for D = 128 the accumulators of both leave one wave per SIMD (341
// registers), and forming p once more for dv costs less than losing the second
// wave (13 packed sequences of up to 1531 rows, 16 heads of 128: 216 -> 192 us;
// for D = 64 both fit, and apart they take 1030 instead of 907 us at T = 8192).
template <int D, int W, int R, int S, bool kApart>
__global__ __launch_bounds__(64 * W, 2) void attn_grad_kernel(AttnGradArgs a, int kv_blocks) {
    constexpr int kTileB = R * Tile<D>::kRowB, kZ = 128 * W;
    // a variable per slot: the compiler then knows which reads a copy in flight cannot touch
    __shared__ __attribute__((aligned(1024))) uint8_t x0[kTileB], x1[kTileB], y0[kTileB], y1[kTileB];
    __shared__ __attribute__((aligned(1024))) uint8_t x2[S > 2 ? kTileB : 16], y2[S > 2 ? kTileB : 16];
    __shared__ __attribute__((aligned(1024))) float z0[kZ], z1[kZ], z2[S > 2 ? kZ : 4];
    auto x = [&](auto u) -> uint8_t* { return pick_slot<decltype(u)::value>(x0, x1, x2); };
    auto y = [&](auto u) -> uint8_t* { return pick_slot<decltype(u)::value>(y0, y1, y2); };
    auto z = [&](auto u) -> float* { return pick_slot<decltype(u)::value>(z0, z1, z2); };
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int b = blockIdx.x;
    if (b < kv_blocks) {
        kv_part<D, W, R, S, !kApart, true>(a, x, y, z, b, wave, lane);
    } else if (kApart && b < 2 * kv_blocks) {
        kv_part<D, W, R, S, true, false>(a, x, y, z, b - kv_blocks, wave, lane);
    } else {
        dq_part<D, W, R, S>(a, x, y, b - (kApart ? 2 : 1) * kv_blocks, wave, lane);
    }
}

constexpr int kGW = 4;                           // waves per workgroup

// Workgroups that share the query heads of a key block.  A key block's
// workgroup walks its group's heads one after the other; with fewer than two of
// them per CU the first key blocks' walks outlast everything else, so the heads
// are dealt to several workgroups whose fp32 sums are added up afterwards
// (T = 4096, 32 / 8 heads of 64: 1 -> 363 us, 2 -> 253 + 10 us, 4 -> 257 + 19 us;
// T = 8192, 512 workgroups already: 1 -> 917 us, 2 -> 922 + 14 us).
int attn_backward_splits(int Hq, int Hkv, int64_t total_T, int N) {
    const int G = Hq / Hkv;
    const int64_t blocks = (total_T / (32 * kGW) + 1) * Hkv;
    // a walk of few tiles is shorter than the launch that adds the splits up
    const int64_t tiles = (total_T / N + 63) / 64;
    for (int s = 1; s < G; ++s)
        if (G % s == 0 && (blocks * s >= 512 || G / s * tiles <= 4)) return s;
    return G;
}

template <int D, int R, int S, bool kApart>
static hipError_t launch_bwd(const AttnGradArgs& a, hipStream_t s) {
    const AttnArgs& f = a.f;
    const int64_t rows = 32 * kGW, per_row = f.N == 1 ? (f.total_T + rows - 1) / rows : f.total_T / rows + f.N;
    const int64_t kv = per_row * f.Hkv * a.splits, all = kv * (kApart ? 2 : 1) + per_row * f.Hq;
    const int64_t deltas = (f.total_T + 31) / 32, sums = a.splits > 1 ? f.total_T / 8 + f.N : 0;
    if (too_many(all, 64 * kGW) || too_many(deltas, 256) || too_many(sums, 256)) return hipErrorInvalidConfiguration;
    const int heads = 64 / (D / 8);
    hipLaunchKernelGGL((attn_delta_kernel<D>), dim3((uint32_t)deltas, (f.Hq + heads - 1) / heads), dim3(256), 0, s, a);
    hipLaunchKernelGGL((attn_grad_kernel<D, kGW, R, S, kApart>), dim3((uint32_t)all), dim3(64 * kGW), 0, s, a, (int)kv);
    if (a.splits > 1) hipLaunchKernelGGL((attn_dkv_sum_kernel<D>), dim3((uint32_t)sums), dim3(256), 0, s, a);
    return hipGetLastError();
}

// R rows per staged tile and S slots.  D = 64: 64, 3 (gradients at T = 8192 889 us; 64, 2 1093; 32, 4 1150; 64, 4 as
// 64, 3).  D = 128: 64, 2 (a training step of 13 x 1531 rows 258.5 us; 32, 3 262.5; 32, 4 267).
hipError_t launch_attn_backward(const AttnGradArgs& a, int D, hipStream_t s) {
    return D == 64 ? launch_bwd<64, 64, 3, false>(a, s) : launch_bwd<128, 64, 2, true>(a, s);
}

}  // namespace lfm2sc
