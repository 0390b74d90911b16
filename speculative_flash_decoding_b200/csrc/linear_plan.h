// Choices of alspec_linear that depend on how many clusters the device holds
// (host arithmetic, no CUDA).
#pragma once

#include <algorithm>
#include <cstdint>

namespace alspec {

constexpr int kLinM = 128;        // features per tile
constexpr int kLinPair = 128;     // batch rows of a tile up to which a CTA works alone
constexpr int kLinMaxSplit = 8;   // CTAs of a cluster

// Clusters of c CTAs that a device holds at once, [c]; 0: none fits (a part
// of a device may have no eight SMs, or two, beside each other).  Single CTAs
// always do.
struct LinClusters {
    int n[kLinMaxSplit + 1];
};

// Large batches: pairs of CTAs, so that each brings half of x.  From 250
// rows on x is more bytes than W: 250 x 8192 x 8192 took 43.6 us without.
inline bool lin_pairs(const LinClusters& fit, int nt, int features) {
    return nt > kLinPair && features > kLinM && fit.n[2] > 0;
}

// CTAs that share the K of a tile: the number that makes (waves of clusters)
// x (blocks of a CTA, plus 16 for a wave's beginning and end and four for the
// exchange where there is one) smallest.  Clusters leave SMs idle (148 SMs
// hold 74 pairs, but 45 clusters of 3, 33 of 4, 26 of 5, 15 of 8), and a
// second wave costs more than idle SMs: 33 x 4096 x 6144 (48 tiles) takes 24
// us with 3, 19.6 with 5 and 15 with 2.
// `ctas`: CTAs that work on a tile's block of K together.
inline int lin_split(const LinClusters& fit, int64_t tiles, int kblocks, int ctas) {
    int best = 1;
    int64_t least = INT64_MAX;
    for (int c = 1; c * ctas <= kLinMaxSplit && c <= std::max(1, kblocks / 4); ++c) {
        const int held = c * ctas == 1 ? std::max(1, fit.n[1]) : fit.n[c * ctas];
        if (held < 1) continue;
        const int64_t waves = (tiles + held - 1) / held;
        const int64_t cost = waves * ((kblocks + c - 1) / c + (c > 1 ? 20 : 16));
        if (cost < least) least = cost, best = c;
    }
    return best;
}

}  // namespace alspec
