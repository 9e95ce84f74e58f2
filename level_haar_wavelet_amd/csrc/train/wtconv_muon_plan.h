// wtconv_muon_plan.h -- how the products of a Newton-Schulz step are cut into
// tiles and dealt to workgroups, and what workspace that takes.  Host arithmetic
// alone, so that it can be compiled and checked without a GPU.
#ifndef WTCONV_MUON_PLAN_H
#define WTCONV_MUON_PLAN_H

#include <cstddef>
#include <cstdint>

#include "../../../include/wtconv.h"
#include "wtconv_check.h"

namespace wtc_muon {

// The whole iteration of a matrix n x m, n <= m, in one workgroup of eight waves,
// where one can hold it.  One 32-row block: four tiles of 32 columns a wave;
// two: two tiles (registers).
constexpr int kOneWaves = 8;
inline bool one_fits(int n, int m)
{
    return n <= 32 ? m <= 4 * kOneWaves * 32 : n <= 64 && m <= 2 * kOneWaves * 32;
}

constexpr int kTiledThreads = 256;  // of a workgroup of the tiled path

// A tile of TILE x TILE: how the four waves share it, and a stage's 32-blocks of
// k (twice as many in a deep one).
template <int TILE>
struct Shape {
    static constexpr int kWavesK = TILE == 32 ? 4 : 1;          // waves along k
    static constexpr int kBlocks = TILE == 128 ? 1 : TILE == 64 ? 2 : 4;  // KB
    static constexpr int kSide = TILE == 32 ? 32 : TILE / 2;    // of a wave's part
};

// How the tiles of a product are dealt to workgroups.  kSlots workgroups run at
// once (two a compute unit).  A last round of few tiles, or an only round, may
// be cut along k so that it fills them: 528 tiles of 4096^3 took 1.42 rounds
// of 512 uncut (268 us a product, 222 cut).
struct Deal {
    int tile, tiles, full, slices, cut;
    size_t bytes;  // of the slices' sums
    double us;     // what it should take
};

constexpr int kSlots = 512;

// Whether stages of twice the k pay: so few workgroups that each has a compute
// unit, and its LDS, for itself, and more than three stages of the other kind
// (1x96x384, of one or three: 71.5 us against 67.6).
inline bool is_deep(int64_t groups, int blocks, int tile)
{
    return groups <= kSlots / 2 && tile < 128 && blocks > 3 * (tile == 32 ? Shape<32>::kBlocks : Shape<64>::kBlocks);
}

// Of a tile of 32, 64, 128: us of 32 of k, alone on a compute unit (in stages of
// twice the k, and without) and with a second workgroup there; us of a
// workgroup's start and end; us for adding a slice of a tile.  Measured on
// products of 96 to 4096.
constexpr double kDeep[] = {0.125, 0.29, 1.1}, kAlone[] = {0.15, 0.33, 1.1}, kShared[] = {0.20, 0.46, 1.45}, kEnds[] = {2.0, 2.5, 6.0},
                 kSlice[] = {0.25, 0.25, 2.5}, kLaunch = 4.0;

inline double round_us(int64_t groups, int blocks, int t, bool deep)
{
    const int64_t rounds = groups / kSlots, rest = groups % kSlots;
    double us = (double)rounds * (blocks * kShared[t] + kEnds[t]);
    if (rest) us += blocks * (deep ? kDeep[t] : rest > kSlots / 2 ? kShared[t] : kAlone[t]) + kEnds[t];
    return us;
}

// The tile and the cut that should take the least time, for matrices of
// rows x k by k x cols before padding.
inline Deal make_deal(int rows, int cols, int k, bool sym, int64_t batch)
{
    Deal best = {};
    const int blocks = (k + 31) / 32;
    for (int t = 0; t < 3; ++t) {
        const int tile = 32 << t;
        const int64_t ni = (rows + tile - 1) / tile, nj = (cols + tile - 1) / tile;
        const int64_t all = (sym ? ni * (ni + 1) / 2 : ni * nj) * batch, rest = all % kSlots;
        for (int want = 1; want <= 8; ++want) {
            if (want > 1 && (!rest || rest * want > kSlots || blocks / want < 4)) break;
            Deal d = {};
            d.tile = tile;
            d.full = (int)(want > 1 ? all - rest : all);
            d.cut = (blocks + want - 1) / want;
            d.slices = (blocks + d.cut - 1) / d.cut;
            const bool deep = is_deep(want > 1 ? d.full + rest * d.slices : all, d.cut, tile);
            d.us = kLaunch + round_us(d.full, blocks, t, deep);
            if (want > 1) {
                d.us += round_us(rest * d.slices, d.cut, t, deep) + kLaunch + d.slices * kSlice[t];
                d.bytes = align256((size_t)rest * d.slices * tile * tile * 4 * (tile == 32 ? 4 : 1));
            }
            if (!best.tile || d.us < best.us) best = d;
        }
    }
    return best;
}

inline int pad(int v, int t) { return (v + t - 1) / t * t; }

// The same deal on the padded sides (a multiple of its tile).
inline void fit_deal(Deal &d, int lp, int rp, int kp, bool sym, int64_t batch)
{
    const int64_t ni = lp / d.tile, nj = rp / d.tile;
    d.tiles = (int)(sym ? ni * (ni + 1) / 2 : ni * nj);
    const int64_t all = d.tiles * batch;
    if (d.slices < 2) {
        d.full = (int)all;
        return;
    }
    const int blocks = kp / 32, rest = (int)(all % kSlots);
    d.full = (int)(all - rest);
    d.cut = (blocks + d.slices - 1) / d.slices;
    d.slices = (blocks + d.cut - 1) / d.cut;
    d.bytes = align256((size_t)rest * d.slices * d.tile * d.tile * 4 * (d.tile == 32 ? 4 : 1));
}

// Sides and buffers of the tiled path.
struct Plan {
    bool one;  // a workgroup a matrix, no workspace
    int n, m, tall, np, mp, parts;
    Deal gram, poly, apply;   // the three products of a step
    size_t xbytes, abytes, part;  // planes of X and of A, slices' sums
};

inline Plan make_plan(const wtconv_ortho_desc_t &d)
{
    Plan p = {};
    p.tall = d.rows > d.cols;
    p.n = (int)(p.tall ? d.cols : d.rows);
    p.m = (int)(p.tall ? d.rows : d.cols);
    p.one = one_fits(p.n, p.m);
    if (p.one) return p;
    p.gram = make_deal(p.n, p.n, p.m, true, d.batch);
    p.poly = make_deal(p.n, p.n, p.n, true, d.batch);
    p.apply = make_deal(p.n, p.m, p.n, false, d.batch);
    // sides are padded to the largest tile in use, and to the 64 of ortho_split
    const int big = p.gram.tile == 128 || p.poly.tile == 128 || p.apply.tile == 128 ? 128 : 64;
    p.np = pad(p.n, big);
    p.mp = pad(p.m, big);
    fit_deal(p.gram, p.np, p.np, p.mp, true, d.batch);
    fit_deal(p.poly, p.np, p.np, p.np, true, d.batch);
    fit_deal(p.apply, p.np, p.mp, p.np, false, d.batch);
    p.part = p.gram.bytes > p.poly.bytes ? p.gram.bytes : p.poly.bytes;
    if (p.part < p.apply.bytes) p.part = p.apply.bytes;
    p.xbytes = align256((size_t)p.np * p.mp * 4 * d.batch);
    p.abytes = align256((size_t)p.np * p.np * 4 * d.batch);
    const int64_t want = ((int64_t)p.n * p.m + 16 * kTiledThreads - 1) / (16 * kTiledThreads);
    p.parts = (int)(want < 1024 ? want : 1024);
    return p;
}

// X and X^T twice, A, P, the norm's parts, the slices' sums.
inline size_t workspace_bytes(const Plan &p, int64_t batch)
{
    if (p.one) return 0;
    return 4 * p.xbytes + 2 * p.abytes + align256(sizeof(double) * p.parts * batch) + p.part;
}

}  // namespace wtc_muon

#endif  // WTCONV_MUON_PLAN_H
