// attn_cached8.hip -- plan and dispatch of the attention over a paged cache of
// 8-bit codes (attn_cached8.hpp).
#include <algorithm>

#include "attn_cached8.hpp"

namespace lfm2sc {

Cached8Plan cached8_plan(int D, int Hq, int Hkv, int N, int L, int prefix_len, int max_suffix) {
    Cached8Plan p;
    const int G = Hq / Hkv, rows_unit = 16 * cached8_row_tiles(L, G);
    const int64_t rows = (int64_t)N * L * G;
    const int64_t base = (int64_t)N * (((int64_t)L * G + rows_unit - 1) / rows_unit) * Hkv;
    const int64_t ptiles = ((int64_t)prefix_len + kC8Tile - 1) / kC8Tile, otiles = ((int64_t)max_suffix + kC8Tile - 1) / kC8Tile;
    p.prefix_splits = 0;
    p.prefix_chunk = 0;
    p.prefix_blocks = 0;
    p.form = base <= 512 && ptiles + otiles <= (base >= 128 ? 32 : 16) ? kDirect8
             : prefix_len > 0 && rows > kSharedRows                              ? kShared8
                                                                        : kSplit8;
    if (p.form == kDirect8) {
        p.suffix_splits = 0;
        p.suffix_blocks = base;
        return p;
    }
    if (prefix_len > 0) {
        const int64_t rows_wg = p.form == kShared8 ? kSharedRows : rows_unit, row_blocks = (rows + rows_wg - 1) / rows_wg;
        // seconds at 8e14 flops/s and 5e12 bytes/s; a batch fills about half of its longest suffix
        const double product = 4. * rows * Hkv * D * prefix_len / 8e14, read = (double)N * max_suffix * Hkv * D / 5e12;
        const double share = product / (product + read);
        const double slots = p.form == kShared8 ? 256. * form_per_simd(D, 1, kShared8) * (share > 0.8 ? 1. : share) : 256.;
        const int64_t want = (int64_t)(slots / (double)(row_blocks * Hkv)), most = (ptiles + 3) / 4;
        const int64_t splits = want < 1 ? 1 : want < most ? want : most;
        const int64_t per = (ptiles + splits - 1) / splits;
        p.prefix_chunk = (int)per * kC8Tile;
        p.prefix_splits = (int)((ptiles + per - 1) / per);
        p.prefix_blocks = row_blocks * Hkv * p.prefix_splits;
    }
    const int64_t most = (otiles + 3) / 4, want = std::min<int64_t>((rows_unit == 16 ? 2048 : 1024) / base, 32);
    p.suffix_splits = (int)(want < 1 ? 1 : want < most ? want : most);
    if (p.suffix_splits < 1) p.suffix_splits = 1;
    const int per_wg = form_waves(p.form) / own_waves(p.form);
    p.suffix_blocks = (base * p.suffix_splits + per_wg - 1) / per_wg;
    return p;
}

hipError_t launch_attn_cached8(Cached8Args a, int D, bool int8, hipStream_t s) {
    CachedArgs& c = a.c;
    const Cached8Plan p = cached8_plan(D, c.Hq, c.Hkv, c.N, c.L, c.prefix_len, a.max_suffix);
    c.prefix_splits = p.prefix_splits;
    c.prefix_chunk = p.prefix_chunk;
    c.prefix_blocks = p.prefix_blocks;
    c.suffix_splits = p.suffix_splits;
    const int64_t blocks = p.prefix_blocks + p.suffix_blocks;
    const bool join = p.prefix_splits + p.suffix_splits > 1;
    if (too_many(blocks, 64 * form_waves(p.form)) || (join && too_many(((int64_t)c.N * c.L * c.Hq + 3) / 4, 256)))
        return hipErrorInvalidConfiguration;
    const hipError_t e = D == 64 ? (int8 ? launch_cached8<64, true>(a, p.form, blocks, s) : launch_cached8<64, false>(a, p.form, blocks, s))
                                 : (int8 ? launch_cached8<128, true>(a, p.form, blocks, s) : launch_cached8<128, false>(a, p.form, blocks, s));
    if (e != hipSuccess || !join) return e;
    return launch_attn_join(c, D, s);
}

}  // namespace lfm2sc
