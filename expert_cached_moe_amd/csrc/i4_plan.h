// Which kernel a product with 4-bit weights takes: rules on sizes and the number of compute units.  Host code
// without HIP.
#pragma once

#include <cmath>
#include <cstdint>

namespace moe {
namespace i4 {

// Up to 8 rows of x, and by expert up to 8 tokens: the few-row kernel (8 tokens: 4096 x 4096 7.5 us against 8.3 on tiles of 32
// rows, 12288 x 4096 13.2 against 25, 32768 x 4096 27 against 26, 100003 x 4096 71 against 65; 4 tokens there 48 against 65; 4096 x
// 4096 at 16 tokens, in two blocks of 8, 12.2 against 8.3).  By expert too: 128 of 2048 x 768, top 8, at 8 tokens 42 us against 46
// on tiles, at 16 tokens 68 against 61; 256 of 4096 x 1536 and the shared one, top 6, 113-118 against 132 and 173 against 168.
constexpr int kFewTokens = 8;
// Dense products of more rows too, where blocks of 8 rows by 16 of the weights leave a CU one workgroup at most and rows
// are long: the tiles' waves split K no further than the few-row kernel's, and wait for each slice (16 x 2048 x 12288 13.4 us
// against 17.0, in fp32 parts 32 x 1024 x 12288 29 and 46, 128 x 256 x 8192 10.5 and 12.5; 32 x 1024 x 1024 4.3 both; two
// workgroups a CU, 64 x 1024 x 8192: 17.7 against 12.7).
inline bool few_dense(int64_t T, int64_t N, int64_t K, int n_cu) {
    return T <= kFewTokens || (K > 1024 && (N + 15) / 16 * ((T + kFewTokens - 1) / kFewTokens) <= n_cu);
}

// The kernels for more rows: tiles of `rows` of x by `cols` of the weights, K split over `split` groups of waves,
// up to `slots` workgroups a CU.  A slice of 64 k takes `one` us with one workgroup on each CU and `more` for each further
// one; 256 x 256 tiles take `one` and, with more of them than CUs, `more` on top: a chip at its power limit.  `tile` us are
// for the start and the results.
// Measured on bf16 x (replays of a graph over weights used in turn): 4096 x 4096 at 32 rows 8.4 us on 32 x 32 tiles (17 on 128 x
// 32 and 64 x 64), at 128 11.2 on 64 x 32 (17.3 on 128 x 32), at 512 27 on 128 x 64 (34 on 128 x 32, 102 on 256 x 256); 4096 x
// 12288 at 256 rows 50 on 128 x 32 (86 on 128 x 64); 16384 x 4096 at 1024 rows 118 on 256 x 256 (151 on 128 x 128); 100003 x 4096
// at 32 rows 71 on 32 x 128 (88 on 64 x 128, 108 on 32 x 32), at 64 92 on 64 x 128 (112 on 32 x 128), at 128 147 on 128 x 128 (153
// on 64 x 128), at 256 224 on 256 x 256 (259 on 128 x 128).  By expert (as above): at 64 tokens 86 on 32 x 128 (114 on 64 x 128), at
// 1,024 180 on 64 x 128 (201 on 32 x 128, 253 on 256 x 256), at 2,048 291 on 64 x 128 (339 on 32 x 128, but 275 on 256 x 256), at 4,096
// 446 on 256 x 256 (499 on 128 x 128, 1008 on 64 x 64).
struct Kind {
    int rows, cols, split, slots;
    double one, more, tile;
};
enum { kMid32x32, kMid64x32, kMid128x32, kMid64x64, kMid128x64, kMid32x128, kMid64x128, kMid128x128, kTurns, kKinds };
constexpr Kind kKind[kKinds] = {
    {32, 32, 8, 1, 0.87, 0.0, 1.5},   {64, 32, 8, 1, 1.12, 0.0, 1.5},   {128, 32, 4, 1, 0.95, 0.0, 1.5},
    {64, 64, 4, 1, 1.00, 0.0, 1.5},   {128, 64, 4, 1, 1.45, 0.0, 1.5},  {32, 128, 1, 6, 0.38, 0.34, 1.5},
    {64, 128, 1, 3, 0.48, 0.36, 1.5}, {128, 128, 1, 2, 0.95, 0.32, 5.0}, {256, 256, 1, 1, 1.60, 0.20, 10.0},
};
// Time of `tiles` row tiles over N weight rows of K, `slices` walks of 64 k each.
inline double kind_time(int kind, double tiles, int64_t N, int64_t slices, int n_cu) {
    const Kind& k = kKind[kind];
    const double blocks = tiles * double((N + k.cols - 1) / k.cols), steps = double((slices + k.split - 1) / k.split);
    const double whole = std::floor(blocks / (n_cu * k.slots)), rest = std::ceil((blocks - whole * n_cu * k.slots) / n_cu);
    const double full = (k.one + (kind == kTurns ? 1 : k.slots - 1) * k.more) * steps + k.tile;
    return whole * full + (rest > 0 ? (k.one + (rest - 1) * k.more) * steps + k.tile : 0.0);
}
// Workgroups of a launch (the threads of one fit 31 bits; 256 x 256 tiles are few enough for every product that memory
// holds).
constexpr int64_t kMostBlocks = 0x7FFFFFFF / 512;
inline bool fits(int kind, int64_t tiles, int64_t N) {
    return kind == kTurns || tiles <= kMostBlocks / ((N + kKind[kind].cols - 1) / kKind[kind].cols);
}
// Dense: T rows, `planes` walks over K.
inline int plan_dense(int64_t T, int64_t N, int64_t K, int planes, int n_cu) {
    int best = 0;
    double least = 1e30;
    for (int k = 0; k < kKinds; ++k) {
        const int64_t tiles = (T + kKind[k].rows - 1) / kKind[k].rows;
        const double t = kind_time(k, double(tiles), N, (K + 63) / 64 * planes, n_cu);
        if (t < least && fits(k, tiles, N)) least = t, best = k;
    }
    return best;
}
// The most row tiles that n entries of `rows` rows in all can have.
inline int64_t map_tiles(int64_t n, int64_t rows, int tile) { return rows / tile + n; }
// Experts: `pairs` rows over n entries (their numbers of rows are known on the device only: as if each pair chose
// at random), N and K of one product.
inline double entry_tiles(int n, int64_t pairs, int rows) {
    const double busy = n * (1.0 - std::exp(-double(pairs) / n)), each = pairs / busy;
    return busy * (each <= rows / 2 ? 1.0 : each / rows + 0.5);
}
inline int plan_experts(int n, int64_t pairs, int64_t N, int64_t K, int n_cu) {
    int best = 0;
    double least = 1e30;
    for (int k = 0; k < kKinds; ++k) {
        const double t = kind_time(k, entry_tiles(n, pairs, kKind[k].rows), N, (K + 63) / 64, n_cu);
        if (t < least && fits(k, map_tiles(n, pairs, kKind[k].rows), N)) least = t, best = k;
    }
    return best;
}
}  // namespace i4
}  // namespace moe
