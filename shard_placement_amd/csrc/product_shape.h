// product_shape.h -- which tile, split and launch a layer product takes
// (linear.hip).  Rules on sizes alone; host code without HIP.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace tide {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

constexpr int64_t kSplitUnit = 256;  // contraction elements

enum Kind { kForward, kGradInput, kGradWeight };

// Tile and split for a product of I x J outputs.
struct Shape {
    int bi, bj, bk;
    int halves;  // of the contraction inside a workgroup
    int32_t tiles_i, tiles_j, splits;
    int64_t split_depth;
};

inline void set_split(Shape* s, int64_t I, int64_t J, int64_t depth, int64_t splits) {
    const int64_t units = ceil_div(depth, kSplitUnit);
    const int64_t each = std::max<int64_t>(1, ceil_div(units, std::max<int64_t>(1, splits)));
    s->tiles_i = (int32_t)ceil_div(I, s->bi);
    s->tiles_j = (int32_t)ceil_div(J, s->bj);
    s->split_depth = each * kSplitUnit;
    s->splits = (int32_t)std::max<int64_t>(1, ceil_div(units, each));
}

// The steps of 64 contraction elements that a tile runs: the split's, or the
// contraction's where that ends first.
inline int64_t steps_of(const Shape& s, int64_t depth) {
    return ceil_div(std::min(depth, s.split_depth), 64);
}

// What a tile costs, in microseconds: a step when a quarter of the compute units
// have one (`step`) and what it takes longer when all have (`power`: the clock
// falls), measured at K = 8192; and the rest of a tile's life (first loads,
// epilogue; of the 128-wide ones as 2 to 16 steps show it in all three layouts:
// 300 x 1024 x 1024 forward, dx and dW 12.3, 12.3 and 8.9 us with two sets of
// waves, 14.8, 13.9 and 9.3 with one).  Of the last tile, two sets of waves take
// a step each in that time.
struct TileCost {
    int bi, bj, halves;
    double step, power, rest;
};
constexpr TileCost kTiles[] = {{256, 256, 1, 1.25, 0.30, 7.0},
                               {256, 192, 1, 0.95, 0.36, 6.0},
                               {256, 128, 1, 0.72, 0.33, 5.0},
                               {128, 128, 1, 0.60, 0.00, 4.6},
                               {128, 128, 2, 1.10, 0.00, 4.2}};
// Two 128 x 128 tiles on a compute unit take a step each in this time.
constexpr double kPairStep = 0.95;
constexpr int kCus = 256;

// A tile of 256 rows, with `used` of the compute units at work.
inline double wide_tile_us(const TileCost& c, double steps, double used) {
    return steps * (c.step + c.power * used * used) + c.rest;
}

// 256-wide tiles of dW read x widened to bf16, which is a launch of its own
// before them: 3 bytes an element at 5.5 MB/us.
inline double widen_us(int64_t T, int64_t K) { return 4.0 + 3.0 * (double)T * (double)K / 5.5e6; }

inline double product_us(Kind kind, const TileCost& c, const Shape& s, int64_t I, int64_t J,
                         int64_t depth) {
    const int64_t groups = (int64_t)s.tiles_i * s.tiles_j * s.splits;
    const double rounds = (double)ceil_div(groups, kCus);
    const double steps = (double)steps_of(s, depth);
    double us;
    if (c.halves == 2) {
        us = rounds * (std::ceil(steps / 2) * c.step + c.rest);
    } else if (c.bi == 128) {
        const double pairs = (double)(int64_t)(rounds / 2), single = rounds - 2 * pairs;
        us = pairs * (steps * kPairStep + c.rest) + single * (steps * c.step + c.rest);
    } else {
        us = rounds * wide_tile_us(c, steps, (double)groups / (rounds * kCus));
        if (kind == kGradWeight) us += widen_us(depth, I);
    }
    // partial sums: a compute unit writes 40 KB/us, the join is a launch of its
    // own and reads 5.5 MB/us (dx of 128 x 1024 x 5120 takes 15.4 us in four
    // splits, 13.1 whole)
    if (s.splits > 1)
        us += rounds * 4.0 * c.bi * c.bj / 40e3 +
              4.0 + 4.0 * (double)s.splits * (double)I * (double)J / 5.5e6;
    return us;
}

// Up to 64 rows of outputs the A operand's bytes bound the product: narrow
// tiles, and the contraction split until about two workgroups a compute unit
// keep loads in flight (5120 x 5120 and 16 rows: 13.8 us, with one 15.6, with
// four 16.8).  A forward weight of more bytes than the 256 MB cache holds is
// read 512 bytes of a row at a time and past the cache, in tiles that fill
// LDS: 80 us for 28672 x 8192 and 16 rows, 115 otherwise.  Smaller weights are
// faster from the cache (5120 x 5120 and 24 rows: 30 us that way).
// Otherwise the tile and split of the least estimated time.  2048 x 5120
// outputs of depth 13824: 264 us with the 256 x 192 tiles this takes, 290 with
// 256 x 256, 313 with 128 x 128.  A 128 x 128 tile that has a compute unit to
// itself is worked on by two sets of waves, half the contraction each, which
// keeps twice the loads in flight: forward of 1024 x 1024 x 1024 12.5 us, with
// one set 15.2; 2048 x 2048 x 5120 50, 60; 1500 x 1500 x 3000 takes one set and
// three splits, two workgroups a compute unit, 32 (with two sets 39).  Every
// number of splits up to 16 is looked at: 77 x 768 x 8192 forward takes 16, 13.8
// us, with 8 15.2; 493 x 81 x 3904 16, 11.5, with 4 14.2.  Over 60 products with
// every tile and split the estimates of the better forms are 1.02 (forward), 0.92
// (dx) and 0.91 (dW) of what they take in the median, and the choice is 2% off
// the best, 20% at worst.  Operand bytes are not among the costs: a weight of
// hundreds of MB with 65 to 256 tokens takes up to half as long again.
inline Shape choose(Kind kind, int64_t I, int64_t J, int64_t depth, double* estimate = nullptr) {
    Shape s = {};
    s.bk = 64;
    s.halves = 1;
    if (J <= 64) {
        s.bi = 128;
        s.bj = J <= 16 ? 16 : J <= 32 ? 32 : 64;
        if (kind == kForward && s.bj <= 32 && I * depth > ((int64_t)128 << 20)) s.bk = 256;
        const int64_t want = s.bk == 256 ? kCus : 2 * kCus;
        int64_t splits = want / std::max<int64_t>(1, ceil_div(I, s.bi));
        // a contraction of up to 1024 is over before a join would be, and up to
        // 2048 two sets of waves do what two splits would, without one (us with two
        // sets / in two splits for forward, dx and dW of 28672 outputs a row, 40
        // rows: depth 1032 17.8 / 22.9, 15.8 / 20.4, 13.3 / 20.1; depth 2048 31.0 /
        // 30.4, 29.7 / 29.4, 20.2 / 23.2; depth 4096 65.5 / 62.9, 52.9 / 50.5, 49.0 / 42.7)
        const bool sets = s.bj > 16 && s.bk == 64;
        if (depth <= 1024 || (sets && depth <= 2048 && splits == 2)) splits = 1;
        set_split(&s, I, J, depth, splits);
        // one set of waves where more of the smaller workgroups fit (65536 x 1024
        // and 40 rows: 23.8 us, with two sets 29.5); up to 16 rows or 512 elements
        // there is nothing to gain from two.  40 rows, depth 1024, 768 and 5120
        // outputs a row: forward 9.1 and 9.2 (one set 10.5 and 10.6), dx 9.0 and
        // 9.4 (9.9 and 11.2), dW 10.6 and 10.8 (12.9 and 13.0)
        if (sets && s.splits == 1 && depth > 512 && s.tiles_i <= kCus) s.halves = 2;
        return s;
    }
    const int64_t most = std::min<int64_t>(16, std::max<int64_t>(1, ceil_div(depth, kSplitUnit)));
    double best = 0.0;
    for (const TileCost& c : kTiles) {
        for (int64_t splits = 1; splits <= most; ++splits) {
            Shape t = s;
            t.bi = c.bi;
            t.bj = c.bj;
            t.halves = c.halves;
            set_split(&t, I, J, depth, splits);
            // a split takes whole units, so fewer splits may do, which had their turn
            if (t.splits < splits) continue;
            const double us = product_us(kind, c, t, I, J, depth);
            if (best == 0.0 || us < best) {
                best = us;
                s = t;
            }
            if ((int64_t)t.tiles_i * t.tiles_j >= 4 * kCus) break;  // enough without
        }
    }
    if (estimate) *estimate = best;
    return s;
}

// dx [T, K] and dW [N, K] in one launch of 256-wide tiles, the longer ones
// first: the pair of tiles of the least estimated time, or none if that is not
// 3% less than `best`, that of the two products one after the other.
// (Measured, both gradients with dz, against two launches: 2048 x 13824 x 5120
// 496 us, 600; 8192 x 8192 x 1024 272, 331; 3000 x 1280 x 8192 129, 141; and 748
// against 729 for 700 x 28672 x 8192, whose estimates were 0.7% apart.)
inline bool choose_pair(int64_t T, int64_t N, int64_t K, double best, Shape* in, Shape* weight,
                        bool* in_first) {
    constexpr int kWide = 2;  // 256 x 256 and 256 x 192
    bool found = false;
    best *= 0.97;
    for (int a = 0; a < kWide; ++a) {
        for (int b = 0; b < kWide; ++b) {
            const TileCost &cx = kTiles[a], &cw = kTiles[b];
            Shape x = {cx.bi, cx.bj, 64, 1, 0, 0, 1, 0}, w = {cw.bi, cw.bj, 64, 1, 0, 0, 1, 0};
            set_split(&x, K, T, N, 1);
            set_split(&w, K, N, T, 1);
            const int64_t nx = (int64_t)x.tiles_i * x.tiles_j, nw = (int64_t)w.tiles_i * w.tiles_j;
            const double tx = wide_tile_us(cx, (double)steps_of(x, N), 1.0),
                         tw = wide_tile_us(cw, (double)steps_of(w, T), 1.0);
            const double longer = std::max(tx, tw), shorter = std::min(tx, tw);
            const int64_t n_long = tx >= tw ? nx : nw;
            int64_t n_short = nx + nw - n_long;
            // whole rounds of the longer; then the shorter beside the rest of
            // them, and on the whole chip behind them
            double us = widen_us(T, K) + (double)(n_long / kCus) * longer;
            const int64_t rest = n_long % kCus;
            if (rest) {
                us += longer;
                n_short -= (kCus - rest) * (int64_t)(longer / shorter);
            }
            if (n_short > 0) us += (double)ceil_div(n_short, kCus) * shorter;
            if (us < best) {
                best = us;
                *in = x;
                *weight = w;
                *in_first = tx >= tw;
                found = true;
            }
        }
    }
    return found;
}

inline int64_t grid_of(const Shape& s) { return (int64_t)s.tiles_i * s.tiles_j * s.splits; }

// Whether a forward product goes by the weight's rows (gemv_kernel) instead of
// tiles: up to 4 tokens, z not kept (whole checkpoint blocks need the tiles'
// epilogue).  direct: x and W can be read where they lie; otherwise tiles need a
// copy of W (4 x 4096 x 1001: 11.7 us by rows, 21.2).  Read in place, with
// weights that come from memory (us by rows / in tiles, N x K):
//   1 token   512 x 512 4.1 / 4.8, 1024 x 8192 8.0 / 10.5, 28672 x 8192 73.9 / 78.3
//   2         256 x 512 5.9 / 4.8, 256 x 1024 6.0 / 7.0, 256 x 8192 9.2 / 8.6,
//             1024 x 8192 9.9 / 11.4, 4096 x 4096 11.0 / 12.0
//   4         256 x 8192 13.3 / 9.2, 1024 x 8192 14.0 / 12.0, 4096 x 4096 14.5 / 12.3,
//             28672 x 4096 52.9 / 61.5, 28672 x 28672 258 / 278
// (rows: 32 multiply-adds for 16 bytes of W at 4 tokens, which only the largest
// weights' bytes hide; tiles: a second launch where the contraction is split).
inline bool forward_by_rows(int64_t T, int64_t N, int64_t K, bool keep, bool direct) {
    if (T > 4 || K < 8 || keep) return false;
    if (T == 1 || !direct) return true;
    if (T == 2) return K > 512 && (K <= 1024 || N >= 512);
    return N * K > ((int64_t)96 << 20);
}

// The gradients' products: dx [T, K] with N (rounded up to 8) terms, dW [N, K]
// with T, and whether they share a launch.  dx, dw: it is wanted and no size is 0.
struct Gradients {
    Shape in, weight;
    bool pair;
    bool in_first;  // of 256-wide tiles in one launch: dx's are the longer ones
};

inline Gradients choose_gradients(int64_t T, int64_t N, int64_t K, bool dx, bool dw) {
    const int64_t width = round_up(N, 8);
    Gradients g = {};
    double in_us = 0.0, w_us = 0.0;
    g.weight = choose(kGradWeight, K, N, T, &w_us);
    g.in = choose(kGradInput, K, T, width, &in_us);
    // Both in one launch where together they are at most two workgroups a
    // compute unit, dx with half as many splits if need be (94 x 2560 x 2248: 20.5
    // us, in two launches 29.0); then a short contraction is cheaper whole than
    // split and joined (a join is 5 us, a step of 64 0.6), and half as many splits
    // that leave each workgroup a compute unit to itself are better than all of
    // them (212 x 2560 x 912: 18.8 us, 21.4).
    if (dx && dw && g.in.bi == 128 && g.weight.bi == 128 && g.weight.bj == 128 && g.weight.splits == 1) {
        Shape in = g.in;
        auto fit = [&](int64_t groups) {
            const int64_t most = (groups - grid_of(g.weight)) / ((int64_t)in.tiles_i * in.tiles_j);
            if (most < in.splits && 2 * most >= in.splits) set_split(&in, K, T, width, most);
        };
        fit(2 * kCus);
        g.pair = grid_of(in) + grid_of(g.weight) <= 2 * kCus;
        if (width <= 1024) set_split(&in, K, T, width, 1);
        fit(kCus);
        if (g.pair) g.in = in;
    }
    if (dx && dw && !g.pair && in_us > 0.0 && w_us > 0.0)
        g.pair = choose_pair(T, width, K, in_us + w_us, &g.in, &g.weight, &g.in_first);
    return g;
}

}  // namespace tide
