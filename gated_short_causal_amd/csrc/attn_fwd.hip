// attn_fwd.hip -- causal attention over packed prompts, grouped heads.
//
// One pass over the keys with the running maximum m and sum l of each query
// row's softmax.  A wave owns 32 query rows of one head; a workgroup's W
// waves own consecutive rows and share the K and V tiles (kKT keys) that are
// copied to LDS ahead of use, S slots of them.  Scores are formed transposed, S^T = K Q^T, so
// that a lane holds 16 keys of one query per 32-key block: the row maximum and
// sum are in-lane up to one exchange between the wave's halves, and
// P^T = exp(S^T - m), rounded to bf16, is in place as the operand of
// O^T += V^T P^T.  P never leaves the registers.
//
// Fewer bits: the matrix unit takes bf16 operands, so p enters the product with v
// rounded once (half a step, 2^-9 of it; l sums the unrounded p).  The output is
// then off by 2.0e-3 (relative 2-norm, 64-bit softmax) where its own rounding
// alone gives 1.6e-3; p as the sum of two bf16 parts would cost a third product.
// Scores, m, l and o stay fp32.
//
// What bounds it: long prompts run at the clock that the matrix and vector units
// leave each other (1.9 GHz of 2.4): T = 8192, 32 / 8 heads of 64, 280-290 us = 950-980
// TFLOP/s with the vector unit busy 76% and the matrix unit 50% of the cycles;
// 16 / 2 heads of 128, 260-270 us = 1.03 PFLOP/s (a library product of 8192^3:
// 1.24).  One sequence of up to ~2000 tokens has fewer workgroups than CUs or not
// many more, and takes the time of its longest row block: about 0.9 us per 64 keys
// (T = 1024: 16.6 us; two wave groups that share its keys, joined in LDS: 15.9).
// Measured and not kept: 64 rows per wave (75 us at 8 x 2048
// against 67), 8 waves (70), 128-key tiles (68), separate code for tiles without
// a mask (116 -> 162 registers: 336 us at 8192 against 304).
#include "attn_common.hpp"
#include "hybrid.hpp"

namespace lfm2sc {

// A launch of one sequence whose workgroups are all resident at once: CU i gets
// blocks i, i + 256, .. in falling order, so the CUs with the first of each
// round would get all the heavy ones.  Every other round of `fold` row blocks
// runs the other way (T = 4096, 32 heads of 64: 87 -> 82 us).
__device__ __forceinline__ int folded(int t, int blocks, int fold) {
    if (fold < 2) return t;
    const int round = t / fold;
    return (round & 1) && (round + 1) * fold <= blocks ? round * fold + fold - 1 - t % fold : t;
}

template <int D, int W, int kKT, int S>
__global__ __launch_bounds__(64 * W, 2) void attn_fwd_kernel(AttnArgs a, int fold) {
    using T = Tile<D>;
    constexpr int kBM = 32 * W, NB = kKT / 32;
    constexpr int kTileB = kKT * T::kRowB;
    // a variable per slot: the compiler then knows which reads a copy in flight cannot touch
    __shared__ __attribute__((aligned(1024))) uint8_t k0[kTileB], k1[kTileB], v0[kTileB], v1[kTileB];
    __shared__ __attribute__((aligned(1024))) uint8_t k2[S > 2 ? kTileB : 16], v2[S > 2 ? kTileB : 16];
    auto kslot = [&](auto u) -> uint8_t* { return pick_slot<decltype(u)::value>(k0, k1, k2); };
    auto vslot = [&](auto u) -> uint8_t* { return pick_slot<decltype(u)::value>(v0, v1, v2); };

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
    // block -> (row block, head): all heads of a row block together, the key/value heads dealt to the XCDs in
    // turn, so the heads that share keys and values run on the same XCDs
    const int G = a.Hq / a.Hkv;
    const int b = blockIdx.x;
    const int kvh = b % a.Hkv, head = kvh * G + (b / a.Hkv) % G;
    const SeqTile st = find_seq_tile(a.cu, a.N, a.total_T, folded(b / a.Hq, gridDim.x / a.Hq, fold), kBM);
    if (st.len == 0) return;
    const int q0 = (st.rank - 1) * kBM;
    const int wrow = q0 + wave * 32;             // the wave's first row in the sequence
    const int tiles = (min(q0 + kBM, st.len) + kKT - 1) / kKT;

    const uint16_t* kp = a.k + st.start * a.k_stride + (int64_t)kvh * D;
    const uint16_t* vp = a.v + st.start * a.v_stride + (int64_t)kvh * D;
    const TileCopy<D, W, kKT> kcopy(wave, lane, a.k_stride), vcopy(wave, lane, a.v_stride);
    auto issue = [&](uint8_t* kb, uint8_t* vb, int t) {
        t = min(t, tiles - 1);
        const int rows = min(kKT, st.len - t * kKT);
        kcopy(kp + (int64_t)t * kKT * a.k_stride, a.k_stride, rows, kb, wave);
        vcopy(vp + (int64_t)t * kKT * a.v_stride, a.v_stride, rows, vb, wave);
    };

    issue(k0, v0, 0);
    if constexpr (S > 2) issue(k1, v1, 1);

    // the wave's queries as B operands: row c, values 16 s + 8 h ..
    bf16x8 qf[D / 16];
    const int row = wrow + c;
    load_row_operand<D>(qf, a.q + (st.start + row) * a.q_stride + (int64_t)head * D, h, row < st.len);
    const LaneOffsets<D> lo(lane);
    const float cs = a.scale * kLog2e;           // exp(scale s) = exp2(cs s)
    float m = kNegInf, l = 0.f;
    f32x16 o[D / 32];
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] = 0.f;

    auto tile = [&](const uint8_t* kb, const uint8_t* vb, int t) {
        f32x16 s[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[n][i] = 0.f;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int ds = 0; ds < D / 16; ++ds) s[n] = mfma32(lds_row(kb + n * 32 * T::kRowB, lo.row[ds]), qf[ds], s[n]);
        if (t * kKT + kKT - 1 > wrow) {          // the tile reaches past the wave's first row
            const int r = row - t * kKT - 4 * h;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n * 32 + (i & 3) + 8 * (i >> 2) > r) s[n][i] = kNegInf;
        }
        float mx = s[0][0];
#pragma unroll
        for (int i = 1; i < 16 * NB; ++i) mx = fmaxf(mx, s[i >> 4][i & 15]);
        const float mn = max_halves(mx) * cs;
        if (__any(mn > m + kLazy)) {
            const float ref = fmaxf(m, mn), alpha = exp2_fast(m - ref);
            l *= alpha;
#pragma unroll
            for (int db = 0; db < D / 32; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[db][i] *= alpha;
            m = ref;
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16 * NB; ++i) {
            const float p = exp2_fast(__builtin_fmaf(s[i >> 4][i & 15], cs, -m));
            s[i >> 4][i & 15] = p;
            sum += p;
        }
        l += sum;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const bf16x8 p = to_operand(s[n], ks);
#pragma unroll
                for (int db = 0; db < D / 32; ++db)
                    o[db] = mfma32(lds_transposed(vb + (n * 32 + ks * 16) * T::kRowB, lo.tr[0][db], lo.tr[1][db]), p, o[db]);
            }
    };

    const int last = min(wrow + 32, st.len) - 1;    // the wave's last row
    for_stages<S>(tiles, [&](auto u, int t) {
        constexpr int refill = (decltype(u)::value + S - 1) % S;
        wait_vm<(S - 2) * 2 * decltype(kcopy)::kDma>();
        stage_barrier();
        issue(kslot(IC<refill>{}), vslot(IC<refill>{}), t + S - 1);
        if (t * kKT <= last && wrow < st.len) tile(kslot(u), vslot(u), t);
    });
    wait_vm<0>();                                // no copy may outlive the workgroup

    const float sum = sum_halves(l);
    store_transposed<D>(a.out + (st.start + row) * a.out_stride + (int64_t)head * D, o, 1.f / sum, h, row < st.len);
    if (a.lse != nullptr && h == 0 && row < st.len)
        a.lse[(int64_t)head * a.total_T + st.start + row] = (m + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <int D, int W, int KT, int S>
static hipError_t launch_fwd(const AttnArgs& a, hipStream_t s) {
    // sum ceil(len / rows) over the sequences is at most this
    const int64_t rows = 32 * W, per_head = a.N == 1 ? (a.total_T + rows - 1) / rows : a.total_T / rows + a.N;
    const int64_t blocks = per_head * a.Hq;
    if (too_many(blocks, 64 * W)) return hipErrorInvalidConfiguration;
    constexpr int kResident = 256 * (D == 64 ? 4 : 3);           // workgroups
    const int fold = a.N == 1 && blocks <= kResident ? 256 / a.Hq : 0;
    hipLaunchKernelGGL((attn_fwd_kernel<D, W, KT, S>), dim3((uint32_t)blocks), dim3(64 * W), 0, s, a, fold);
    return hipGetLastError();
}

hipError_t launch_attn_prefill(const AttnArgs& a, int D, hipStream_t s) {
    // keys per tile and slots: D = 64 leaves four workgroups per CU with two slots of 64 keys (8 x 2048: 56.3 us; 32, 3
    // and 64, 3 60), D = 128 three with three slots of 32 (13 x 1531: 52.1 us; 32, 2 54.0; 32, 4 57.6; 64, 2 56.2)
    return D == 64 ? launch_fwd<64, 4, 64, 2>(a, s) : launch_fwd<128, 4, 32, 3>(a, s);
}

}  // namespace lfm2sc
