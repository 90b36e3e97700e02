// drafts.hip -- verification of drafted tokens against the target's
// probabilities (speculative sampling), from given random numbers.
//
// Draft s of a sequence, token x with probabilities p (target) and q (draft),
// is accepted while u q(x) < p(x); the product of two fp32 values is exact in
// fp64.  With a drafts accepted, the next token is drawn from
//   r = p_a                         every draft accepted
//   r = max(p_a - q_a, 0)           else (q_a: 1 at the draft's token when no
//                                   draft probabilities are given)
//   r = p_a                         where that leaves nothing
// as the lowest index whose running sum of r exceeds u sum r.  Sums and
// differences are fp64 throughout: the differences are exact up to the last
// bit, and an index turns on where a sum passes a border.
//
// Only one row of p and one of q per sequence is read.  The rows are cut into
// chunks: one kernel sums every chunk, a second finds the chunk in which the
// border lies, from the sums, and reads that chunk again.
#include "common.hpp"
#include "hybrid.hpp"

namespace lfm2sc {

constexpr int kDT = 256;                         // threads per workgroup
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// 8 consecutive probabilities from any element address (rows of an odd
// vocabulary are aligned to an element only); zeros at and beyond `left`.
template <typename E>
__device__ __forceinline__ void load_probs(const E* p, int64_t left, float* f) {
    if (left >= 8) {
        Raw8<E> r;
        const u32x4_any* v = reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
        for (int i = 0; i < Elem<E>::kChunks; ++i) {
            const u32x4 x = v[i];
            r.c[i] = make_uint4(x.x, x.y, x.z, x.w);
        }
        to_f32(r, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = 0.f;
            if (i < left) {
                if constexpr (sizeof(E) == 2) f[i] = __uint_as_float((uint32_t)p[i] << 16);
                else f[i] = p[i];
            }
        }
    }
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

// r of 8 consecutive tokens from index i, and the clean p.
template <typename E>
__device__ __forceinline__ void weights(const Draw<E>& d, int i, int V, double* r, double* p) {
    float x[8], y[8];
    load_probs<E>(d.p + i, V - i, x);
    if (d.q != nullptr) {
        load_probs<E>(d.q + i, V - i, y);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = i + j == d.hole ? x[j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const double diff = (double)x[j] - (double)y[j];
        r[j] = diff > 0. ? diff : 0.;            // NaN counts as nothing
        p[j] = x[j] > 0.f ? (double)x[j] : 0.;
    }
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
    return x;
}

template <typename E>
__global__ __launch_bounds__(kDT) void draft_sums_kernel(DraftArgs<E> a, int chunks) {
    __shared__ double part[2][kDT / 64];
    const int n = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Draw<E> d = accept(a, n, lane);
    const int start = chunk * a.chunk;
    double sr = 0., sp = 0.;
    for (int i = start + threadIdx.x * 8; i < min(start + a.chunk, a.V); i += kDT * 8) {
        double r[8], p[8];
        weights(d, i, a.V, r, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sr += r[j];
            sp += p[j];
        }
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

template <typename E>
__global__ __launch_bounds__(kDT) void draft_pick_kernel(DraftArgs<E> a, int chunks) {
    __shared__ double part[kDT / 64];
    __shared__ int found[kDT / 64], lastpos[kDT / 64];
    const int n = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Draw<E> d = accept(a, n, lane);
    // totals; every thread walks the same sums in order
    const double* sr = a.sums + (int64_t)n * 2 * chunks;
    const double* sp = sr + chunks;
    double total = 0.;
    for (int c = 0; c < chunks; ++c) total += sr[c];
    const bool residual = total > 0.;
    if (!residual) {
        total = 0.;
        for (int c = 0; c < chunks; ++c) total += sp[c];
    }
    const double* sums = residual ? sr : sp;
    const double border = (double)a.u_sample[n] * total;
    // the first chunk in which the running sum passes the border; without one (u not below 1, a NaN) the last that
    // adds anything
    double before = 0., run = 0.;
    int pick = -1;
    for (int c = 0; c < chunks; ++c) {
        const double s = sums[c];
        if (s > 0.) {
            pick = c;
            before = run;
        }
        run += s;
        if (run > border) break;
    }
    int token = -1;
    if (pick >= 0) {
        const int start = pick * a.chunk, end = min(start + a.chunk, a.V);
        // rounds of kDT x 8 tokens in order, so the running sum grows along the index
        int best = -1, last = -1;
        for (int i0 = start; i0 < end && best < 0; i0 += kDT * 8) {
            const int i = i0 + threadIdx.x * 8;
            double r[8], p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = p[j] = 0.;
            if (i < end) weights(d, i, a.V, r, p);
            double own = 0.;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!residual) r[j] = p[j];
                own += r[j];
            }
            double scan = own;
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) {
                const double up = __shfl_up(scan, s, 64);
                if (lane >= s) scan += up;
            }
            __syncthreads();
            if (lane == 63) part[wave] = scan;
            __syncthreads();
            double base = before, all = before;
#pragma unroll
            for (int w = 0; w < kDT / 64; ++w) {
                if (w < wave) base += part[w];
                all += part[w];
            }
            double cum = base + (scan - own);
            int hit = 0x7fffffff, pos = -1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                cum += r[j];
                if (r[j] > 0.) {
                    pos = i + j;
                    if (cum > border && hit == 0x7fffffff) hit = i + j;
                }
            }
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) {
                hit = min(hit, __shfl_xor(hit, s, 64));
                pos = max(pos, __shfl_xor(pos, s, 64));
            }
            if (lane == 0) {
                found[wave] = hit;
                lastpos[wave] = pos;
            }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kDT / 64; ++w) {
                if (found[w] != 0x7fffffff && (best < 0 || found[w] < best)) best = found[w];
                last = max(last, lastpos[w]);
            }
            before = all;
        }
        token = best >= 0 ? best : last;
    }
    if (threadIdx.x == 0) {
        a.accept_len[n] = d.accepted;
        if (a.keep_len != nullptr) a.keep_len[n] = d.accepted + 1;
        a.next_token[n] = token;
    }
}

int draft_chunks(int V) { return (V + kDraftChunk - 1) / kDraftChunk; }

template <typename E>
hipError_t launch_drafts(DraftArgs<E> a, hipStream_t s) {
    a.chunk = kDraftChunk;
    const int chunks = draft_chunks(a.V);
    if ((int64_t)chunks * a.N >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((draft_sums_kernel<E>), dim3((uint32_t)(chunks * a.N)), dim3(kDT), 0, s, a, chunks);
    hipLaunchKernelGGL((draft_pick_kernel<E>), dim3(a.N), dim3(kDT), 0, s, a, chunks);
    return hipGetLastError();
}
template hipError_t launch_drafts<uint16_t>(DraftArgs<uint16_t>, hipStream_t);
template hipError_t launch_drafts<float>(DraftArgs<float>, hipStream_t);

}  // namespace lfm2sc
