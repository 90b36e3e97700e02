// seq_find.hpp -- the sequence of a packed call that a wave's row or unit belongs
// to: row offsets are device data.
#pragma once

#include "common.hpp"

namespace lfm2sc {

struct SeqAt {
    int seq;
    int begin, end;          // cu[seq], cu[seq + 1], as they are
    int extra;               // of `also`
};

// The last sequence i in [0, N), N >= 1, with before(i, cu[i]), or 0: `before` holds for
// a leading part of the offsets where they do not fall, and any result is within
// bounds where they do.  also: an array [N] of which the sequence's entry is wanted
// too, or nullptr.  Wave-uniform.
//
// Up to 256 sequences every lane looks at four offsets, and their entries come out of
// the lanes: one memory round trip.  More take one for each factor of 64.
template <typename F>
__device__ __forceinline__ SeqAt find_seq(const int32_t* __restrict__ cu, const int32_t* __restrict__ also, int N, F before) {
    const int lane = threadIdx.x & 63;
    SeqAt r;
    r.extra = 0;
    if (N <= 256) {
        int v[4], x[4] = {0, 0, 0, 0};           // offset 4 lane + j + 1, entry 4 lane + j
        const int first = cu[0];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = cu[min(4 * lane + j + 1, N)];
            if (also != nullptr) x[j] = also[min(4 * lane + j, N - 1)];
        }
        r.seq = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) r.seq += __popcll(__ballot(4 * lane + j + 1 < N && before(4 * lane + j + 1, v[j])));
        auto pick = [](const int (&a)[4], int i) {
            const int j = i & 3, y = j == 0 ? a[0] : j == 1 ? a[1] : j == 2 ? a[2] : a[3];
            return __builtin_amdgcn_readlane(y, i >> 2);
        };
        r.seq = __builtin_amdgcn_readfirstlane(r.seq);
        r.begin = r.seq == 0 ? first : pick(v, r.seq - 1);
        r.end = pick(v, r.seq);
        if (also != nullptr) r.extra = pick(x, r.seq);
        return r;
    }
    int lo = 0, hi = N;                          // before(lo) or lo == 0; not before(hi), or hi == N
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64, at = lo + (lane + 1) * step;
        const int part = __popcll(__ballot(at < hi && before(at, cu[min(at, N)])));
        const int next = lo + part * step;
        hi = min(next + step, hi);
        lo = next;
    }
    r.seq = __builtin_amdgcn_readfirstlane(lo);
    r.begin = cu[r.seq];
    r.end = cu[r.seq + 1];
    if (also != nullptr) r.extra = also[r.seq];
    return r;
}

}  // namespace lfm2sc
