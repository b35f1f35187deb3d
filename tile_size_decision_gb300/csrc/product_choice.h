// The choice of a product's kernel, tile and split (host code, free of CUDA).
#pragma once

#include <algorithm>
#include <cstdint>

namespace tiles {

// How a product runs: on CTA pairs, or with the few-rows kernel; the rows and
// columns of a tile, and the CTAs along K.
struct Choice { bool pair; int rows, cols, split; };

// The cheapest by a model in nanoseconds: a start, then the larger of
//   - the rounds over the resident blocks x (a round's own start and end + its
//     K blocks x the time of one), and
//   - the bytes at the measured copy rate, times how far a kernel stays from it.
// Few rows (two blocks an SM): a second resident block and the addition over a
// cluster cost extra.  8-bit pairs: a K block's time depends on the kernel
// (tiles up to 128 or 256 wide), not on the tile's width.  The constants are fitted
// to the times of 150 products on a GB300 with every kernel (m 1 to 25,000, n
// and k 128 to 4096, up to 32 groups): within 5 to 9% of them on average, and
// the choice within 1% of the best.  Both sides, in 8 bits: 16 rows of 4096 x
// 4096 5.4 us against 20.3 on pairs, 1000 x 4096 x 128 10.0 against 6.4; 32
// groups of 53 rows, 128 x 2816 in 16 bits, 16.6 against 11.8, 8 of 62 rows,
// 128 x 1024, 3.9 against 5.5.  Tiles of 128 rows never won: 8-bit sums of 128
// rows leave room for one block an SM.
inline Choice choose(bool fp8, int64_t m, int64_t n, int64_t k, int64_t groups, int sms, int pairs) {
    const int64_t kb = (k + (fp8 ? 127 : 63)) / (fp8 ? 128 : 64);
    // Groups that can have rows, each with a weight of its own (0: dense).
    // (With half a tile for every group counted, 1 row in 64 groups by 1024 x
    // 4096 in 16 bits took 16.0 us on unsplit blocks, 5.8 now.)
    const int64_t some = std::min(groups, m);
    // Row tiles: grouped, half a tile a group more than the rows fill, at
    // least one for every group that can have rows.
    auto row_tiles = [&](int64_t rows) {
        if (groups == 0) return (m + rows - 1) / rows;
        return std::max(some, m / rows + some / 2);
    };
    const int64_t eb = fp8 ? 1 : 2;
    const int64_t weights = groups == 0 ? 1 : some;
    const double dram_ns = static_cast<double>((weights * n * k + m * k) * eb + 2 * m * n) / 6786.0;
    Choice best{};
    double best_ns = 0;
    auto offer = [&](const Choice& c, double ns) {
        if (best_ns == 0 || ns < best_ns) { best = c; best_ns = ns; }
    };
    struct Few { int rows; double start, round, block, second, cluster, far; };
    static constexpr Few few16[] = {{16, 1150, 2260, 250, 640, 35, 1.08},
                                    {32, 1000, 2720, 265, 900, 16, 1.10},
                                    {64, 570, 3710, 340, 1490, 5, 1.15}};
    static constexpr Few few8[] = {{16, 820, 2230, 310, 610, 35, 1.00},
                                   {32, 720, 2780, 360, 870, 8, 1.10},
                                   {64, 120, 4010, 465, 1760, 4, 1.20}};
    for (const Few& f : fp8 ? few8 : few16) {
        const int64_t units = row_tiles(f.rows) * ((n + 127) / 128);
        // CTAs along K: while the units leave SMs without a block, at least
        // two K blocks a CTA.
        int split = 1;
        while (split < 8 && units * split < sms && kb >= split * 4) split *= 2;
        const double rounds = static_cast<double>((units * split + 2 * sms - 1) / (2 * sms));
        const double work = rounds * (f.round + static_cast<double>((kb + split - 1) / split) * f.block) +
                            (units * split > sms ? f.second : 0);
        offer(Choice{false, f.rows, 128, split},
              f.start + std::max(work, dram_ns * f.far) + (split > 1 ? f.cluster * f.rows : 0));
    }
    // Pairs: 8-bit tiles as narrow as the rounds allow, in either kernel.
    struct Pair { int most, least; double start, round, block; };
    static constexpr Pair pair16[] = {{256, 256, 4400, 1350, 250}};
    static constexpr Pair pair8[] = {{256, 160, 3970, 1620, 460}, {128, 64, 3500, 1100, 300}};
    for (int i = 0; i < (fp8 ? 2 : 1); ++i) {
        const Pair& p = fp8 ? pair8[i] : pair16[i];
        int64_t fewest = INT64_MAX;
        int cols = p.most;
        for (int c = p.most; c >= p.least; c -= 32) {
            const int64_t rounds = (row_tiles(256) * ((n + c - 1) / c) + pairs - 1) / pairs;
            if (rounds <= fewest) { fewest = rounds; cols = c; }
        }
        offer(Choice{true, 256, cols, 1},
              p.start + std::max(static_cast<double>(fewest) * (p.round + kb * p.block),
                                 dram_ns * 1.05));
    }
    return best;
}

}  // namespace tiles
