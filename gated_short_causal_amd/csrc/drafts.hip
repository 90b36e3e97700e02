// drafts.hip -- verification of drafted tokens against the target's
// probabilities (speculative sampling), from given random numbers.
//
// Draft s of a sequence, token x with probabilities p (target) and q (draft),
// is accepted while u q(x) < p(x); the product of two fp32 values is exact in
// fp64.  With a drafts accepted, the next token is drawn from
//   r = p_a                         every draft accepted
//   r = max(p_a - q_a, 0)           else (q_a: 1 at the draft's token when no
//                                   draft probabilities are given; in r, NaN and
//                                   negative entries of both rows count as 0)
//   r = p_a                         where that leaves nothing
// as the lowest index whose running sum of r exceeds u sum r.  Sums and
// differences are fp64 throughout: the differences are exact up to the last
// bit, and an index turns on where a sum passes a border.
//
// Only one row of p and one of q per sequence is read.  Two forms:
//   whole   a workgroup per sequence holds its row in flight at once and finds the
//           token in the same kernel;
//   split   for few sequences with long rows: the rows are cut into chunks, one
//           kernel sums every chunk, a second finds the chunk in which the
//           border lies, from the sums, and reads that chunk again.
#include "common.hpp"
#include "hybrid.hpp"

namespace lfm2sc {

constexpr int kDT = 256;                         // threads per workgroup
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// 8 consecutive probabilities from any element address (rows of an odd
// vocabulary are aligned to an element only).
template <typename E>
__device__ __forceinline__ Raw8<E> load_probs(const E* row, int i) {
    Raw8<E> r;
    // a 32-bit byte offset to a wave-uniform row: V < 2^30
    const u32x4_any* v = reinterpret_cast<const u32x4_any*>(reinterpret_cast<const char*>(row) + (uint32_t)i * (uint32_t)sizeof(E));
#pragma unroll
    for (int i = 0; i < Elem<E>::kChunks; ++i) {
        const u32x4 x = v[i];
        r.c[i] = make_uint4(x.x, x.y, x.z, x.w);
    }
    return r;
}
// The first `n` < 8 of them, then zeros.
template <typename E>
__device__ __forceinline__ Raw8<E> load_probs_few(const E* p, int n) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = 0.f;
        if (i < n) {
            if constexpr (sizeof(E) == 2) f[i] = __uint_as_float((uint32_t)p[i] << 16);
            else f[i] = p[i];
        }
    }
    return from_f32<E>(f);
}
template <typename E> __device__ __forceinline__ double prob(const E* p) {
    if constexpr (sizeof(E) == 2) return (double)__uint_as_float((uint32_t)*p << 16);
    else return (double)*p;
}

// What the acceptance leaves to draw from.
template <typename E>
struct Draw {
    int accepted;
    const E* p;        // target row
    const E* q;        // draft row, or nullptr
    int hole;          // token whose probability is taken out (without draft rows), or -1
};

// Wave-uniform: lane s looks at draft s.
template <typename E>
__device__ __forceinline__ Draw<E> accept(const DraftArgs<E>& a, int n, int lane) {
    const int drafts = a.num_drafts == nullptr ? a.L : min(max(a.num_drafts[n], 0), a.L);
    bool reject = false;
    int token = -1;
    if (lane < drafts) {
        token = a.tokens[(int64_t)n * a.L + lane];
        double p = 0., q = 1.;
        if (token >= 0 && token < a.V) {
            p = prob(a.target + ((int64_t)n * (a.L + 1) + lane) * a.target_stride + token);
            if (a.draft != nullptr) q = prob(a.draft + ((int64_t)n * a.L + lane) * a.draft_stride + token);
        }
        reject = !((double)a.u_accept[(int64_t)n * a.L + lane] * q < p);
    }
    const uint64_t no = __ballot(reject);
    Draw<E> d;
    d.accepted = no != 0 ? __builtin_ctzll(no) : drafts;
    d.p = a.target + ((int64_t)n * (a.L + 1) + d.accepted) * a.target_stride;
    d.q = nullptr;
    d.hole = -1;
    if (no != 0) {
        if (a.draft != nullptr) d.q = a.draft + ((int64_t)n * a.L + d.accepted) * a.draft_stride;
        else d.hole = __builtin_amdgcn_readlane(token, d.accepted);
    }
    return d;
}

// r of 8 consecutive tokens from index i, of which x and y (kRows: there are
// draft rows) are the target's and the draft's probabilities: max(x - y, 0),
// without draft rows x outside the hole; 0 for the first `skip` (kEnd).  A NaN or
// negative y is 0 from the start (a median drops a NaN); the difference is fp64,
// its sign is exact, and a NaN of it (x, or both infinite) counts as nothing.
template <bool kRows, bool kEnd, typename E>
__device__ __forceinline__ void weights(const Raw8<E>& xr, const Raw8<E>& yr, int i, int hole, int skip, double* r) {
    float x[8], y[8];
    to_f32(xr, x);
    if constexpr (kRows) to_f32(yr, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (kRows) {
            if constexpr (kEnd) x[j] = j >= skip ? x[j] : 0.f;
            r[j] = fmax((double)x[j] - (double)__builtin_amdgcn_fmed3f(y[j], 0.f, __builtin_inff()), 0.);
        } else {
            bool some = x[j] > 0.f && i + j != hole;
            if constexpr (kEnd) some = some && j >= skip;
            r[j] = (double)(some ? x[j] : 0.f);
        }
    }
}
__device__ __forceinline__ double sum8(const double* r) {
    return ((r[0] + r[1]) + (r[2] + r[3])) + ((r[4] + r[5]) + (r[6] + r[7]));
}

// The rows to draw from: as the rule leaves them, or (plain) the target's own.
template <typename E>
struct Source {
    const E* p;
    const E* q;        // nullptr: none
    int hole, V;
    __device__ Source(const Draw<E>& d, int V_, bool plain)
        : p(d.p), q(plain ? nullptr : d.q), hole(plain ? -1 : d.hole), V(V_) {}
    // Where 8 tokens from index i (at or beyond the end too) are read: the row's last 8 at most, of which those
    // before i are skipped.
    __device__ __forceinline__ int at(int i) const { return min(i, max(V - 8, 0)); }
    // r of tokens at(i) .. at(i) + 7, 0 before i
    __device__ __forceinline__ void operator()(int i, double* r) const {
        const int k = at(i);
        Raw8<E> x, y;
        if (V < 8) {
            x = load_probs_few(p, V);
            if (q != nullptr) y = load_probs_few(q, V);
        } else {
            x = load_probs(p, k);
            if (q != nullptr) y = load_probs(q, k);
        }
        if (q != nullptr) weights<true, true>(x, y, k, hole, i - k, r);
        else weights<false, true>(x, x, k, hole, i - k, r);
    }
    // Over N pieces of 8 tokens, 512 apart from index i, f(piece, r of at(..) .. at(..) + 7); V >= 8.  Every load is
    // issued before the first use.  kEnd: some lie at or beyond the row's end, or at or beyond `limit`, and count as
    // nothing.
    template <int N, bool kRows, bool kEnd, typename F>
    __device__ __forceinline__ void pieces(int i, int limit, F f) const {
        Raw8<E> x[N], y[N];
        auto where = [&](int n) { return !kEnd ? i + n * 512 : at(i + n * 512 < limit ? i + n * 512 : i); };
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = load_probs(p, where(n));
        if constexpr (kRows) {
#pragma unroll
            for (int n = 0; n < N; ++n) y[n] = load_probs(q, where(n));
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            double r[8];
            const int k = where(n), skip = i + n * 512 < limit ? i + n * 512 - k : 8;
            weights<kRows, kEnd>(x[n], kRows ? y[n] : x[n], k, hole, skip, r);
            f(n, r);
            __builtin_amdgcn_sched_barrier(0);   // one piece's fp64 values at a time
        }
    }
    template <int N, typename F>
    __device__ __forceinline__ void each(int i, int limit, bool end, F f) const {
        if (q != nullptr) {
            if (end) pieces<N, true, true>(i, limit, f);
            else pieces<N, true, false>(i, limit, f);
        } else {
            if (end) pieces<N, false, true>(i, limit, f);
            else pieces<N, false, false>(i, limit, f);
        }
    }
};

// Lane `lane` of x (uniform).
__device__ __forceinline__ double read_lane(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int kCtrl, int kRows>
__device__ __forceinline__ double dpp_add(double x) {            // lanes without a source add 0
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, kRows, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, kRows, 0xf, false);
    return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Running sums over the lanes (row_shr 1, 2, 4, 8, then row_bcast 15 and 31).
__device__ __forceinline__ double wave_scan(double x) {
    x = dpp_add<0x111, 0xf>(x);
    x = dpp_add<0x112, 0xf>(x);
    x = dpp_add<0x114, 0xf>(x);
    x = dpp_add<0x118, 0xf>(x);
    x = dpp_add<0x142, 0xa>(x);
    return dpp_add<0x143, 0xc>(x);
}
__device__ __forceinline__ double wave_sum(double x) { return read_lane(wave_scan(x), 63); }

// Of the sums that the lanes hold in order: the first whose running sum (from
// `before`) passes the border, and the running sum before it; without one
// (rounding, u not below 1, a NaN) the last positive one; index -1 if none is
// positive.  Wave-uniform.
struct Found {
    int index;
    double before;
    bool passed;
};
__device__ __forceinline__ Found find_sum(double v, double before, double border) {
    const double scan = before + wave_scan(v);
    const uint64_t some = __ballot(v > 0.), over = __ballot(v > 0. && scan > border);
    if (some == 0) return Found{-1, before, false};
    const int i = over != 0 ? __builtin_ctzll(over) : 63 - __builtin_clzll(some);
    return Found{i, i == 0 ? before : read_lane(scan, i - 1), over != 0};
}

// The token among 8 x 64, lane l holding r of tokens i .. i + 7 (i grows with the
// lane), by the same rule.
__device__ __forceinline__ int pick_token(const double* r, int i, double before, double border) {
    const Found lane = find_sum(sum8(r), before, border);
    if (lane.index < 0) return -1;
    double cum = lane.before;
    int hit = -1, pos = -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        cum += r[j];
        if (r[j] > 0.) {
            pos = i + j;
            if (cum > border && hit < 0) hit = i + j;
        }
    }
    return __builtin_amdgcn_readlane(hit >= 0 ? hit : pos, lane.index);
}

template <typename E>
__device__ __forceinline__ void write_drafts(const DraftArgs<E>& a, int n, int accepted, int token) {
    a.accept_len[n] = accepted;
    if (a.keep_len != nullptr) a.keep_len[n] = accepted + 1;
    a.next_token[n] = token;
}

// The token among N pieces of 512 (below `limit`), lane l at index first of the
// first piece.
template <int N, typename E>
__device__ __forceinline__ int find_token(const Source<E>& src, int first, int limit, double before, double border, int lane) {
    double r[8], sums = 0.;                      // lane i: piece i
    int piece = 0;
    if (N > 1 && src.V >= 8) {
        src.template each<N>(first, limit, true, [&](int i, const double* w) {
            const double s = wave_sum(sum8(w));
            if (lane == i) sums = s;
        });
        const Found f = find_sum(sums, before, border);
        piece = max(f.index, 0);
        before = f.before;
    }
    src(first + piece * 512, r);
    return pick_token(r, src.at(first + piece * 512), before, border);
}

// Whole form: wave w takes the w-th of 16 runs of ceil(V / 8192) pieces of 512
// tokens, N pieces (a group) at a time; every lane's sums of its groups stay in
// LDS.  The wave in whose run the border lies adds its groups' sums up over the
// lanes, finds the group, then the piece in it, which it reads again.  N: pieces
// whose loads are in flight at once (at most 64 registers of them: 256 KiB per
// workgroup; with draft rows in fp32, 21 of the sums' registers go to scratch).
constexpr int kWW = 16;
constexpr int kWholeGroups = 8;
template <typename E> constexpr int kWholeN = sizeof(E) == 2 ? 8 : 4;

template <typename E, int N>
__global__ __launch_bounds__(64 * kWW) void draft_whole_kernel(DraftArgs<E> a) {
    __shared__ double part[kWW];
    __shared__ double mine[kWholeGroups][64 * kWW];
    const int n = blockIdx.x, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Draw<E> d = accept(a, n, lane);
    const int pieces = (a.V + kWW * 512 - 1) / (kWW * 512), groups = (pieces + N - 1) / N;   // at most kWholeGroups
    const int run0 = wave * pieces * 512, limit = min(run0 + pieces * 512, a.V), start = run0 + lane * 8;
    double total = 0.;
    bool plain = false;
    for (;;) {
        const Source<E> src(d, a.V, plain);
        double own = 0.;
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
            double s = 0.;
            if (N == 1) {
                double r[8];
                src(start, r);
                s = sum8(r);
            } else {
                const int first = start + g * N * 512;
                src.template each<N>(first, limit, first - lane * 8 + N * 512 > limit,
                                     [&](int, const double* r) { s += sum8(r); });
            }
            mine[g][threadIdx.x] = s;
            own += s;
        }
        own = wave_sum(own);
        if (lane == 0) part[wave] = own;
        __syncthreads();
        total = wave_sum(lane < kWW ? part[lane & (kWW - 1)] : 0.);
        if (total > 0. || plain) break;
        plain = true;                            // nothing left: the target's own row
        __syncthreads();
    }
    const double border = (double)a.u_sample[n] * total;
    const Found run = find_sum(lane < kWW ? part[lane & (kWW - 1)] : 0., 0., border);
    if (run.index < 0) {
        if (threadIdx.x == 0) write_drafts(a, n, d.accepted, -1);
        return;
    }
    if (wave != run.index) return;
    double sums = 0.;                            // lane g: group g
#pragma unroll
    for (int g = 0; g < kWholeGroups; ++g) {
        const double s = wave_sum(g < groups ? mine[g][threadIdx.x] : 0.);
        if (lane == g) sums = s;
    }
    const Found group = find_sum(sums, run.before, border);
    const Source<E> src(d, a.V, plain);
    const int token = find_token<N>(src, start + group.index * N * 512, limit, group.before, border, lane);
    if (lane == 0) write_drafts(a, n, d.accepted, token);
}

template <typename E>
__global__ __launch_bounds__(kDT) void draft_sums_kernel(DraftArgs<E> a, int chunks) {
    __shared__ double part[2][kDT / 64];
    const int n = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Draw<E> d = accept(a, n, lane);
    const int start = chunk * kDraftChunk;
    const Source<E> rest(d, a.V, false), target(d, a.V, true);
    double sr = 0., sp = 0.;
    for (int i = start + threadIdx.x * 8; i < min(start + kDraftChunk, a.V); i += kDT * 8) {
        double r[8], p[8];
        rest(i, r);
        target(i, p);
        sr += sum8(r);
        sp += sum8(p);
    }
    sr = wave_sum(sr);
    sp = wave_sum(sp);
    if (lane == 0) {
        part[0][wave] = sr;
        part[1][wave] = sp;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double s = 0.;
#pragma unroll
        for (int w = 0; w < kDT / 64; ++w) s += part[threadIdx.x][w];
        a.sums[((int64_t)n * 2 + threadIdx.x) * chunks + chunk] = s;
    }
}

// A wave per sequence: the chunk from the sums, then the chunk 512 tokens at a time.
template <typename E>
__global__ __launch_bounds__(64) void draft_pick_kernel(DraftArgs<E> a, int chunks) {
    const int n = blockIdx.x, lane = threadIdx.x;
    const Draw<E> d = accept(a, n, lane);
    const double* sums = a.sums + (int64_t)n * 2 * chunks;
    auto sum_all = [&](const double* p) {
        double t = 0.;
        for (int c = lane; c < chunks; c += 64) t += p[c];
        return wave_sum(t);
    };
    double total = sum_all(sums);
    const bool plain = !(total > 0.);
    if (plain) {
        sums += chunks;
        total = sum_all(sums);
    }
    const double border = (double)a.u_sample[n] * total;
    Found chunk{-1, 0., false};
    double run = 0.;
    for (int c0 = 0; c0 < chunks && !chunk.passed; c0 += 64) {
        const double s = c0 + lane < chunks ? sums[c0 + lane] : 0.;
        const Found f = find_sum(s, run, border);
        if (f.index >= 0) chunk = Found{c0 + f.index, f.before, f.passed};
        run += wave_sum(s);
    }
    int token = -1;
    if (chunk.index >= 0)
        token = find_token<kDraftChunk / 512>(Source<E>(d, a.V, plain), chunk.index * kDraftChunk + lane * 8, a.V, chunk.before,
                                              border, lane);
    if (lane == 0) write_drafts(a, n, d.accepted, token);
}

int draft_chunks(int V) { return (V + kDraftChunk - 1) / kDraftChunk; }

template <typename E>
hipError_t launch_drafts(const DraftArgs<E>& a, hipStream_t s) {
    // split form: few sequences (CUs left idle by one workgroup each) of long rows.  us in a graph, whole / split, by
    // sequences and vocabulary; fp32 with draft rows: 1 x 100003 15.0 / 9.1, 32 x 128256 18.9 / 15.5, 64 x 128256 22-24 / 21,
    // 64 x 65536 13.2 / 15.5, 256 x 65536 27.7 / 33.8; bf16 with: 8 x 100003 22.4 / 10.2, 32 x 128256 17.2 / 13.6, 64 x 128256
    // 17.3 / 18.2; bf16 without: 1 x 128256 14.5 / 9.8, 32 x 128256 15.3 / 12.2, 64 x 128256 16.3 / 16.4, 256 x 128256 19.8 / 35;
    // fp32 without: 32 x 128256 15.3 / 13.2, 64 x 128256 15.8 / 17.6.  At 65536 they differ by little up to 32 sequences (1:
    // 9.6 / 9.1; bf16 11 / 9.3).  The whole form loses where 64 rows of an odd length above 65536 have draft rows in bf16
    // (64 x 100003: 23.9 / 16.1).
    constexpr int N = kWholeN<E>;
    const bool split = a.V > kWW * kWholeGroups * N * 512 || (a.N <= 32 && a.V > 65536);
    if (!split) {
        if (too_many(a.N, 64 * kWW)) return hipErrorInvalidConfiguration;
        const dim3 grid(a.N), block(64 * kWW);
        if (a.V <= kWW * 512) hipLaunchKernelGGL((draft_whole_kernel<E, 1>), grid, block, 0, s, a);
        else if (a.V <= kWW * 4 * 512) hipLaunchKernelGGL((draft_whole_kernel<E, 4>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((draft_whole_kernel<E, N>), grid, block, 0, s, a);
        return hipGetLastError();
    }
    const int chunks = draft_chunks(a.V);
    if (too_many((int64_t)chunks * a.N, kDT)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((draft_sums_kernel<E>), dim3((uint32_t)(chunks * a.N)), dim3(kDT), 0, s, a, chunks);
    hipLaunchKernelGGL((draft_pick_kernel<E>), dim3(a.N), dim3(64), 0, s, a, chunks);
    return hipGetLastError();
}
template hipError_t launch_drafts<uint16_t>(const DraftArgs<uint16_t>&, hipStream_t);
template hipError_t launch_drafts<float>(const DraftArgs<float>&, hipStream_t);

}  // namespace lfm2sc
