// How the kernels of the grouped and dropout layers are cut: tiles, splits of the
// contraction, parts of a group's rows.  Functions of the shape alone, which the
// workspace sizes, the launches and the tests share; plain C++, no device code.
#pragma once

#include <algorithm>
#include <cstdint>

namespace nf4lora {

inline int64_t ceil_to(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles that any division of M rows into E groups can need.
inline int64_t most_tiles(bool grouped, int E, int64_t M, int rows) {
    if (!grouped) return div_up(M, rows);
    return (M + (rows - 1) * std::min<int64_t>(E, M)) / rows;
}

// Row tiles to expect (for split sizes): half a tile lost per group.
inline int64_t likely_tiles(int E, int64_t M, int rows) {
    return std::max<int64_t>(1, (M + rows / 2 * std::min<int64_t>(E, M)) / rows);
}

struct GroupSplit {
    int splits;
    int per;
};

// `steps` split into parts of at least four steps so that tiles x parts is
// about `ctas`; no part is empty.
inline GroupSplit split_steps(int64_t tiles, int64_t steps, int ctas) {
    // a few steps are over before a second kernel could add their parts
    if (steps <= 8) return {1, static_cast<int>(steps)};
    int64_t s = std::max<int64_t>(1, (ctas + tiles / 2) / std::max<int64_t>(1, tiles));
    s = std::min(s, std::max<int64_t>(1, steps / 4));
    const int64_t per = div_up(steps, s);
    return {static_cast<int>(div_up(steps, per)), static_cast<int>(per)};
}

inline int rank_width(int r) { return static_cast<int>(ceil_to(r, 16)); }
inline int rank64(int r) { return static_cast<int>(ceil_to(r, 64)); }

// Sets of accumulators that a CTA of T or V can hold beside another CTA's, and
// the steps that one of them takes at most.
inline int rank_sets(int r) { return 256 / rank_width(r); }
constexpr int kRunSteps = 16;

// Contraction splits of T (steps over K) and V (over N): two CTAs per SM.  A tile
// for every SM is enough, though: halves would only add their sum (16000 tokens
// over 64 experts of 2048 x 1408, step: 454 us with two parts, 438 with one).
inline GroupSplit rows_split(int E, int64_t M, int64_t contraction, int r, int num_sms) {
    const int64_t tiles = likely_tiles(E, M, 128), steps = div_up(contraction, 64), most = kRunSteps * rank_sets(r);
    GroupSplit s{1, static_cast<int>(steps)};
    if (tiles < num_sms) s = split_steps(tiles, steps, 2 * num_sms);
    if (s.per > most) {
        const int64_t per = div_up(steps, div_up(steps, most));
        s = {static_cast<int>(div_up(steps, per)), static_cast<int>(per)};
    }
    return s;
}

// Steps of a part of a group's rows for dB (out rows N) and dA (out rows K): so
// many that the parts of an even batch are about one per SM, at least eight and at
// most kGradSteps, a part having one accumulator of additions that truncate (sums
// of one sign over 262144 rows of 11008 columns come out 6.2e-4 too small on
// average in three parts, 3.2e-5 in 32; half a unit of the 16-bit result is 2e-3 to
// 4e-3).  The number of parts stays one that a grid can have.
constexpr int64_t kGradSteps = 128, kMostParts = 1 << 14;
inline int grad_part_steps(int E, int64_t M, int64_t out_rows, int num_sms) {
    const int64_t groups = std::min<int64_t>(E, M), steps = div_up(div_up(M, groups), 64);
    const int64_t parts = std::max<int64_t>(1, num_sms / (div_up(out_rows, 256) * groups));
    const int64_t per = std::min(std::max<int64_t>(8, div_up(steps, parts)), kGradSteps);
    return static_cast<int>(std::max(per, div_up(div_up(M, 64), kMostParts)));
}
// Parts of the longest group there can be, and partials in all: a group of n > p
// steps has at most 2 n / p parts.
inline int64_t most_parts(int64_t M, int part_steps) { return std::max<int64_t>(1, div_up(div_up(M, 64), part_steps)); }
inline int64_t most_partials(int E, int64_t M, int part_steps) {
    const int64_t one = most_parts(M, part_steps);
    return one == 1 ? 0 : (E == 1 ? one : 2 * one);
}

// How the fused product is cut: by a model of its time in clocks, from the
// measured parts (per step of a tile the decode's and the issue's share and a term
// for its tokens; per tile its start, its end and, where the next tile's MMAs wait
// for them, the stores of its results; for a split contraction the partials' way
// through memory and one more kernel).  Measured at the choice between the two
// kernels for many tokens: 125 tokens in each of 64 experts of 2048 x 1408, a
// training step: 328 us with 256-token tiles, 345 with 512; 1024 in each of eight
// of 4096 x 11008: 1570 against 1295.
// The groups are taken as equal, which the host has to.
struct FusedPlan {
    int tile;       // the kernel: tiles of up to 32 or 64 (two CTAs per SM), 256 or 512 tokens
    int tile_rows;
    int splits;
    int k_main, k_ext;  // steps
};

inline FusedPlan plan_fused(bool dx, int E, int64_t M, int64_t cols, int64_t contraction, int r, int num_sms) {
    const int64_t groups = std::min<int64_t>(E, M), mean = div_up(M, groups), col_tiles = div_up(cols, 256);
    FusedPlan best{};
    const bool few = mean <= (dx ? 24 : 64);
    double best_cost = 1e30;
    const int64_t pairs = num_sms / 2 * (few ? 2 : 1);
    for (int rows = !few ? 512 : dx ? 32 : 64; rows >= 32; rows -= 32) {
        const int64_t per_group = div_up(mean, rows), size = ceil_to(div_up(mean, per_group), 32);
        const int64_t tiles = groups * per_group * col_tiles;
        const int tile = few ? (dx ? 32 : 64) : rows <= 256 ? 256 : 512, wide = tile == 512 ? 64 : 128;
        const int k_main = static_cast<int>(div_up(contraction, wide)), k_ext = 2 * rank64(r) / wide;
        const double step = few           ? 1500.0
                            : tile == 256 ? (dx ? 1520.0 : 1400.0) + 1.2 * size
                                         : std::max(700.0 + 0.8 * size, 930.0);
        const double ends = few || tile == 256 ? 4000.0 : 3000.0 + 16.0 * size;
        // many tokens: only to put work on every SM at all
        const int most = few ? 8 : static_cast<int>(std::min<int64_t>(8, pairs / tiles));
        for (int splits = 1; splits <= std::max(1, most) && (splits == 1 || splits * 4 <= k_main); ++splits) {
            const double rounds = static_cast<double>(div_up(tiles * splits, pairs));
            double cost = rounds * (step * static_cast<double>(div_up(k_main, splits) + k_ext) + ends);
            if (splits > 1) cost += 6000.0 + static_cast<double>(splits) * M * cols * 8 / 2000.0;
            if (cost < 0.97 * best_cost) {
                best_cost = cost;
                best = {tile, rows, splits, k_main, k_ext};
            }
        }
    }
    return best;
}

}  // namespace nf4lora
