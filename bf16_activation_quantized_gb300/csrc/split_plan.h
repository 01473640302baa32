// split_plan.h -- how the 8-bit products and the weights' gradients are cut into CTAs: host
// code without CUDA, so that a test can ask for the form that a size takes.
#pragma once

namespace w4a16 {

constexpr int kFp8Block = 128;       // elements of a row per scale; weights: 128 x 128
constexpr int kMaxSplit = 8;         // CTAs that share a tile's sum at most

inline int ceil_div(long long x, long long y) { return int((x + y - 1) / y); }

// How a product is cut.  size 16 to 128: the kernel for few rows, of that template size,
// with bt rows of x per tile; 0: the kernel for many rows, with pairs of CTAs or without.
// split: CTAs of a cluster, which share a tile's sum or are a pair.  ctas: launched.
struct Fp8Plan {
    int size, bt, split, ctas, occupancy;
    bool pair;
};

// The forms compared by their time in microseconds, as they measured on 152 SMs with the
// weights in L2 (2560 x 9728, 8192 x 8192, 19456 x 2560, 4096 x 2048 and 1024 x 4096, 144 to
// 4096 rows), beside what all have in common: a block of 128 that is summed over 0.20 (32
// rows and fewer; with two CTAs on an SM 0.28), 0.29 (64 rows; 0.46), 0.36 (128 rows), 0.46
// (128 rows, 256 columns), 0.41 (a pair's 256 and 256); from a tile to the next 1.8 (few
// rows) or 1.0 (many); sums that CTAs share 1 and 0.3 for each (few rows) or 2 and 1.6
// (many).  Groups fill half of their last tile.
inline Fp8Plan fp8_plan(int M, int out, int blocks, int groups, bool grouped, int sms) {
    const int used = !grouped ? 1 : groups < M ? groups : M;                // groups with rows at most
    const int rows = ceil_div(M, used);                                     // a group's, if they are even
    Fp8Plan best = {};
    double best_time = 0;
    auto consider = [&](int size, int tile_rows, bool pair, int split) {
        Fp8Plan p = {};
        p.size = size, p.pair = pair, p.occupancy = size && size <= 64 ? 2 : 1;
        p.bt = size == 0 ? 128 : grouped ? size : (ceil_div(rows, ceil_div(rows, size)) + 15) & ~15;
        const int per = pair ? 2 : split, slots = p.occupancy * sms / per;
        const long long cols = ceil_div(out, size ? kFp8Block : 2 * kFp8Block);
        const long long most = cols * (grouped ? M / tile_rows + used : ceil_div(M, tile_rows));
        if (split > 1 && (most > slots || blocks < 2 * split)) return;
        const long long tiles = grouped ? cols * (2LL * M / tile_rows + used + 1) / 2 : most;
        const double block = pair ? 0.41 : size == 0 ? 0.46 : size == 128 ? 0.36
                             : tiles * split <= sms ? (size == 64 ? 0.29 : 0.20) : size == 64 ? 0.46 : 0.28;
        const int waves = ceil_div(tiles, slots);
        const double time = waves * (ceil_div(blocks, split) * block + (size ? 1.8 : 1.0)) +
                            (split == 1 ? 0.0 : size ? 1.0 + 0.3 * split : 2.0 + 1.6 * split);
        p.split = per;
        p.ctas = per * int(most < slots ? most : slots);
        if (best_time == 0 || time < best_time) best = p, best_time = time;
    };
    const int size = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    for (int split = 1; split <= kMaxSplit; split *= 2) consider(size, size, false, split);
    if (rows <= 64) return best;
    for (int split = 1; split <= kMaxSplit; split *= 2) {
        consider(128, 128, false, split);
        consider(0, 128, false, split);
    }
    consider(0, 256, true, 1);
    return best;
}

// Pairs of CTAs that share a tile's rows in the weights' gradients: as long as all find a place
// and a part holds a few stages (row_step rows each) of a group's rows, if the groups are even.
inline int wgrad_split(long long tiles, int pairs, int rows, int groups, int row_step) {
    int split = 1;
    while (split < 4 && tiles * split * 2 <= pairs && rows / groups >= 8 * row_step * split) split *= 2;
    return split;
}

}  // namespace w4a16
