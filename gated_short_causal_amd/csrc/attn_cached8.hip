// attn_cached8.hip -- plan and dispatch of the attention over a paged cache of
// 8-bit codes (attn_cached8.hpp).
#include <algorithm>

#include "attn_cached8.hpp"

namespace lfm2sc {

// What the plan's splits go by, and the workspace's bound with them.
constexpr int kFewTiles = 16, kFewBlocks = 512;          // direct at up to so many tiles and row blocks, whatever else
constexpr int kMostOwnSplits = 32;
constexpr int kUnits16 = 2048, kUnits16Shared = 4096, kUnits32 = 1024;      // units of suffixes, by rows of a unit
constexpr int kCUs = 256;

Cached8Plan cached8_plan(int D, int Hq, int Hkv, int N, int L, int prefix_len, int max_suffix) {
    Cached8Plan p;
    const int G = Hq / Hkv, rows_unit = 16 * cached8_row_tiles(L, G);
    const int64_t rows = (int64_t)N * L * G;
    const int64_t base = (int64_t)N * (((int64_t)L * G + rows_unit - 1) / rows_unit) * Hkv;
    const int64_t ptiles = ((int64_t)prefix_len + kC8Tile - 1) / kC8Tile, otiles = ((int64_t)max_suffix + kC8Tile - 1) / kC8Tile;
    p.prefix_splits = 0;
    p.prefix_chunk = 0;
    p.prefix_blocks = 0;
    // Direct: no workspace, no join, but every sequence reads the prefix itself and a workgroup walks all of its keys.  Direct
    // and split, 8 heads of 64, keys behind no prefix: 1 x 1000 6.3 and 6.9 us, 1 x 2000 8.5 and 7.1; 16 x 2000 9.7 and
    // 11.3; 32 x 4000 17.6 and 19.3; 64 x 4000 30.6 and 29.7; 128 x 2000 28.3 and 31.5; 256 x 2000 equal; 8 x 8000 23.9 and 16.7.
    // Rows in blocks of 32 (8 tokens of 5 heads of 128): 16 x 4000 34.6 and 41.7, 64 x 999 52 and 36.  Behind a prefix (32
    // sequences, 4096 + 600): 15.9 and 12.1.
    const int64_t few = base < 128 ? kFewTiles : base < 256 || base > 512 || ptiles > 0 ? 32 : 64;
    // Shared: 128 query rows a workgroup.  Shared and split, rows behind 4096 + 600 keys: 64 rows 12.2 and 9.5 us, 256 rows 17.7
    // and 17.3, 1024 rows 33 and 38; behind 16384 + 100: 128 rows 24.4 and 22.5, 160 rows 26.5 and 27.5, 256 rows 29 and 37.
    if (base <= (ptiles > 0 || rows_unit == 32 ? kFewBlocks : 1024) && ptiles + otiles <= few) p.form = kDirect8;
    else p.form = prefix_len > 0 && rows > kSharedRows ? kShared8 : kSplit8;
    if (p.form == kDirect8) {
        p.suffix_splits = 0;
        p.suffix_blocks = base;
        return p;
    }
    if (prefix_len > 0) {
        const int64_t rows_wg = p.form == kShared8 ? kSharedRows : rows_unit, row_blocks = (rows + rows_wg - 1) / rows_wg;
        // The prefix of the shared form gets one workgroup a CU, two or as many as the card holds, by the share that its products
        // take of the time (seconds at 8e14 flops/s and 5e12 bytes/s; a batch fills about half of its longest suffix): numbers
        // in between wait for the CUs that have one more.  256 and 512 workgroups, us: 32 x 4 rows of 5 heads of 128, 4096 + 999
        // (share .67) 32.6 and 40.2; 64 x 8, 2048 + 999 (.67) 69.7 and 76.3; 1024 rows of 64, 8192 + 600 (.58) 51.8 and 48.7;
        // 16384 + 600 (.73) 90.7 and 67.7.  2048 rows, 2048 + 600 (.25): 256 56 us, 128 65; 1024 rows, 4096 + 600 (.4): 256
        // 34, 192 39, 320 38.  The number of splits is rounded down, so a batch just past a divisor of the slots leaves many
        // empty and walks longer parts: 512 single tokens behind 8192 + 1000 keys 116 us, 520 of them 191 (102 and 103 x 8
        // behind 4096 + 999, 5 heads of 128: 146 and 145).  The points are of block scales, those of D = 64 of single tokens;
        // the forms of 32 rows and a scale a token go by the same rule.
        const double product = 4. * rows * Hkv * D * prefix_len / 8e14, read = (double)N * max_suffix * Hkv * D / 5e12;
        const double share = product / (product + read);
        const int per_cu = p.form == kSplit8 ? 1 : share > 0.8 ? form_per_simd(D, 1, kShared8) : share > (rows_unit == 32 ? 0.7 : 0.55) ? 2 : 1;
        const double slots = (double)kCUs * per_cu;
        const int64_t want = (int64_t)(slots / (double)(row_blocks * Hkv)), most = (ptiles + 3) / 4;
        const int64_t splits = want < 1 ? 1 : want < most ? want : most;
        const int64_t per = (ptiles + splits - 1) / splits;
        p.prefix_chunk = (int)per * kC8Tile;
        p.prefix_splits = (int)((ptiles + per - 1) / per);
        p.prefix_blocks = row_blocks * Hkv * p.prefix_splits;
    }
    // Suffixes are split, down to 4 tiles, up to 2048 units of a workgroup; of 32 rows up to 1024 (64 x 8 tokens, 999 keys, no
    // prefix: 36 us, with 2048 53), of the shared form, a wave each, up to 4096 (1024 rows behind 4096 + 2000: 75 us, with 2048 80).
    const int64_t units = rows_unit == 32 ? kUnits32 : p.form == kShared8 ? kUnits16Shared : kUnits16;
    const int64_t most = (otiles + 3) / 4, want = std::min<int64_t>(units / base, kMostOwnSplits);
    p.suffix_splits = (int)(want < 1 ? 1 : want < most ? want : most);
    if (p.suffix_splits < 1) p.suffix_splits = 1;
    const int per_wg = form_waves(p.form) / own_waves(p.form);
    p.suffix_blocks = (base * p.suffix_splits + per_wg - 1) / per_wg;
    return p;
}

// At least the rows times parts that any call of these heads with no larger N, L, prefix_len and max_suffix joins, 0 where
// none joins: the plan's own number falls where a larger batch gets fewer splits or a longer bound another form, and a
// workspace is taken once for the largest of a program's calls.  Splits of the prefix times query rows are at most
// the slots times the 128 rows of a workgroup (32 of the split form), splits of the suffixes times rows at most the units
// times their rows; either is at least 1 where anything is joined, and at most a part to 4 tiles.
int64_t cached8_part_rows(int D, int Hq, int Hkv, int N, int L, int prefix_len, int max_suffix) {
    const int G = Hq / Hkv, rows_unit = 16 * cached8_row_tiles(L, G);
    const int64_t rows = (int64_t)N * L * Hq;
    const int64_t base = (int64_t)N * (((int64_t)L * G + rows_unit - 1) / rows_unit) * Hkv;
    const int64_t ptiles = ((int64_t)prefix_len + kC8Tile - 1) / kC8Tile, otiles = ((int64_t)max_suffix + kC8Tile - 1) / kC8Tile;
    const int64_t own = std::min<int64_t>((otiles + 3) / 4, kMostOwnSplits);
    if (base <= kFewBlocks && ptiles + otiles <= kFewTiles) return 0;        // direct, as are all below it
    static_assert(16 * kUnits16 == 32 * kUnits32, "both row units");
    if (prefix_len == 0) return own <= 1 ? 0 : std::min<int64_t>(rows * own, 16 * kUnits16);
    const int64_t slots = (int64_t)kCUs * std::max(2, form_per_simd(D, 1, kShared8));
    return std::max(rows, std::min<int64_t>(rows * ((ptiles + 3) / 4), kSharedRows * slots)) +
           std::max(rows, std::min<int64_t>(rows * own, 16 * kUnits16Shared));
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
    if (too_many(blocks, 64 * form_waves(p.form)) || (join && too_many(join_blocks(c), 256)))
        return hipErrorInvalidConfiguration;
    const hipError_t e = D == 64 ? (int8 ? launch_cached8<64, true>(a, p.form, blocks, s) : launch_cached8<64, false>(a, p.form, blocks, s))
                                 : (int8 ? launch_cached8<128, true>(a, p.form, blocks, s) : launch_cached8<128, false>(a, p.form, blocks, s));
    if (e != hipSuccess || !join) return e;
    return launch_attn_join(c, D, s);
}

}  // namespace lfm2sc
