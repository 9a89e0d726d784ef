// How a 4-bit product is divided: arithmetic on sizes, without GPU code, so that it
// is checked on the host too.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace qlin {
namespace w4 {

constexpr int kStreamTokens = 8;         // of a workgroup of the streaming kernel
constexpr int kSlot = 256;               // codes its waves take at a time
constexpr int kStreamWaves = 8;

// Threads of a launch: a grid of 2^32 or more is taken modulo that, without an error.
constexpr int64_t kMostThreads = 0xffffffff;

// How K ends: with a whole stage (or slot); inside one, which then is the last one's
// number of codes before the end, those that were had already against zeros; or
// before one is full, where every load is held inside K by itself.  (K = 6304, 18
// tokens, N = 40875, groups of 32: 135 us with every load held, so 81 us; a kernel
// for the first two together costs whole stages 2%, and the streaming kernel with
// fp32 scales 18%.)
enum Ends { kWhole, kInside, kShort };

// Rows of an expert whose offsets are `from` and `to`, whatever they hold: both are
// held to 0..rows before the difference is taken, which then passes no 32 bits
// (0 and -2^31 are 2^31 apart).  `beg`: its first row; at most `most` rows.
__host__ __device__ inline int expert_rows(int from, int to, int rows, int most, int &beg)
{
    beg = from < 0 ? 0 : from > rows ? rows : from;
    const int end = to < 0 ? 0 : to > rows ? rows : to;
    return end <= beg ? 0 : end - beg < most ? end - beg : most;
}

// Tiles of `tile` rows that cover every expert's rows (or M): at most this many.
inline int64_t row_tiles(int64_t M, int64_t experts, int64_t rows, int tile)
{
    return experts ? rows / tile + experts : (M + tile - 1) / tile;
}

// Whether the streaming kernel takes the call: up to 8 tokens (8 on 51200 x 5120
// 35 us, where tiles take 38 for 9; 12 would have to be streamed twice); of
// experts, which differ in their rows, up to 4 on average, or 8 where a tile of 64
// weight rows each does not fill the CUs twice.  128 experts on 1536 x 2048
// with 4 rows each 50 us against 51 us with tiles, with 6 rows 55 and 50 us;
// 8 experts on 1536 x 4096 with 8 rows each 10 and 21 us.
inline bool streams(int64_t M, int64_t N, int64_t experts, int64_t rows)
{
    if (!experts)
        return M <= kStreamTokens;
    const int64_t few = experts * ((N + 63) / 64) <= 512 ? kStreamTokens : kStreamTokens / 2;
    return rows <= few * experts;
}

// The streaming kernel's workgroup: 8 u weight rows, and its waves (no more than K
// has slots).
struct StreamPick {
    int u, waves;
};

// More rows a workgroup share one read of the tokens and one start, fewer
// give the 256 CUs more workgroups: 8 rows up to two workgroups a CU, 32
// from 16 times that (experts: of the tiles in the grid).  Measured, us
// with 8 / 16 / 32 rows, one token: 3.6 / 3.8 / 4.5 (2048 x 2048),
// 12.1 / 9.8 / 10.1 (10240 x 5120), 48 / 34.8 / 29.8 (51200 x 5120).  Where K
// is long, reading the tokens again is what costs, and 32 rows share it: 8
// tokens on 5120 x 25600 24.5 against 32.2 us with 16 rows, one token 23.6 and
// 22.8; on 5120 x 8192 10.8 and 12.3, 10.3 and 10.1.
// Waves: as many as K has slots while workgroups are few, one or two when
// they fill the GPU by themselves (32 tokens through 128 experts of 2048 x
// 768: 22.4 with one, 25.1 with two, 26.7 with three); experts' workgroups
// without rows count half (one token: 8 of 129 tiles have any; 12.1 with two
// waves, 16.3 with one on 1536 x 2048).
inline StreamPick pick_stream(int64_t N, int64_t K, int64_t experts, int64_t rows)
{
    const int64_t tiles = experts ? row_tiles(0, experts, rows, kStreamTokens) : 1, units = (N + 7) / 8 * tiles;
    const int u = units >= 4096 || (K >= 8192 && units > 512) ? 4 : units > 512 ? 2 : 1;
    const int64_t busy = experts ? (units + (N + 7) / 8 * std::min(rows, tiles) + 1) / 2 : units;
    const int waves = (int)std::min(std::max((6144 * u + busy - 1) / busy, (int64_t)1), (int64_t)kStreamWaves);
    return StreamPick{u, waves};
}

// (a dword of zero points needs four groups)
inline Ends stream_end(int64_t K, int64_t G)
{
    return K < kSlot || G < 4 ? kShort : K % kSlot == 0 ? kWhole : kInside;
}

// The tile kernel's tile, 16 tb tokens x 64 rb weight rows with ks codes of K
// at a time, and the parts of K: for M tokens, or with experts for `rows` rows
// of them (one part).
struct TilePick {
    int tb, rb, ks, splits;
};
constexpr TilePick kShortTile{4, 2, 128, 1};                // for K below a stage of any tile

// The tile and the parts of K with the least estimated time.  A CU runs `at_once`
// workgroups of a tile; with so many on every CU a stage takes `us` (`more` where
// they come in several rounds), with fewer down to 0.4 of that, and starting and
// ending a workgroup costs four stages.  Parts of K cost the traffic of their sums
// and another launch: 1 us of the GPU's time, but 4 of a caller's who does not
// replay graphs (59 tokens on 65 x 1280: 5.8 us in five parts, 6.7 in one, and 14.0
// against 9.5 us a call).  When it was fitted, of all these tiles with 1 to 20 parts
// this choice took 3% longer on the GPU than the best on average, 13% at most, on
// eight shapes from 2048 x 2048 to 51200 x 5120 and 5120 x 25600 with 12 to 1000
// tokens and groups of 64 and 128.  12 tokens on 51200 x 5120: 40 us with rb = 2,
// 43 us with rb = 1; 32 on 5120 x 25600 with groups of 64 and zero points: 35 us in
// the twelve parts it picks (nine stages each, the last a single one), 37 in ten,
// 41 in twenty, 168 in one; 512 on 10240 x 5120: 75 us with tb, rb = 4, 2, 85 us
// with 4, 4; 2048: 263 and 234 us.
// With experts, whose rows differ, no tile is higher than 1.5 times their mean
// (25 rows each of 128 experts on 1536 x 2048: 68 us as picked, 1, 2; 75 us with
// 2, 2; 86 us with tb = 4); this choice was then 1% off the best on average, 8 to
// 128 experts with 2 to 150 rows each.
inline TilePick pick_tile(int64_t M, int64_t N, int64_t K, int64_t experts, int64_t rows)
{
    static const struct {
        int tb, rb, ks, at_once;
        double us, more;
    } kTiles[] = {{1, 1, 256, 3, 1.3, 1.3}, {1, 2, 256, 2, 1.55, 1.55}, {2, 1, 256, 3, 1.7, 1.7},
                  {2, 2, 256, 2, 2.0, 2.0}, {4, 2, 128, 3, 2.0, 2.1}, {4, 4, 128, 2, 2.9, 2.5}};
    constexpr int kMostParts = 20;
    TilePick best = kShortTile;
    double least = 1e30;
    for (const auto &t : kTiles) {
        const int64_t high = 16 * t.tb, stages = (K + t.ks - 1) / t.ks;
        // each expert that has rows has a tile, and its last one is half full on average
        const double mean = experts ? (double)rows / experts : 0;
        if ((t.tb > 1 && experts && high > 1.5 * mean && K >= 256) || t.ks > K)
            continue;
        const double tall = experts ? experts * std::max(std::min(1.0, mean), mean / high + 0.5) : (double)((M + high - 1) / high);
        const double each_cu = tall * ((N + 64 * t.rb - 1) / (64 * t.rb)) / 256;
        // (outputs that are too many for one launch of the sum of the parts are not split)
        const int most = experts || M * N > kMostThreads / 2 ? 1 : (int)std::min<int64_t>(kMostParts, stages);
        for (int splits = 1; splits <= most; ++splits) {
            const int64_t each = (stages + splits - 1) / splits;
            if ((stages + each - 1) / each != splits)
                continue;                                    // a part would be empty
            const double whole = std::floor(each_cu * splits / t.at_once);
            const double rest = std::ceil(each_cu * splits - whole * t.at_once - 1e-9);
            double us = (whole + (rest > 0 ? 0.4 + 0.6 * rest / t.at_once : 0)) * (each + 4) * (whole > 0 ? t.more : t.us);
            if (splits > 1)
                us += 4.0 + splits * (double)M * N * 8 / 5e6;
            if (us < least) {
                least = us;
                best = TilePick{t.tb, t.rb, t.ks, splits};
            }
        }
    }
    return best;
}

// How K ends in a tile's stages of ks codes.
inline Ends tile_end(int64_t K, int ks) { return K < ks ? kShort : K % ks == 0 ? kWhole : kInside; }

}  // namespace w4
}  // namespace qlin
