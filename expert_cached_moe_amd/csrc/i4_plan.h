// Which kernel a product with 4-bit weights takes: rules on sizes and the number of compute units.  Host code
// without HIP.
#pragma once

#include <cmath>
#include <cstdint>

namespace moe {
namespace i4 {

// Up to 8 rows of x: the few-row kernel (100003 x 4096 at 8 tokens 77-82 us against 93 on tiles of 32 rows, 4096 x 4096
// 7.8 against 8.8; at 16 tokens, in two blocks of 8, 12.8 against 8.9).
constexpr int kFewTokens = 8;

// The kernels for more rows: tiles of `rows` of x by `cols` of the weights, K split over `split` groups of waves,
// `slots` workgroups a CU.  A slice of 64 k takes `one` us with one workgroup on each CU and `full` with all.
// Measured on bf16 x (dense, whole kernel): 4096 x 4096 at 32 rows 9.3 us on 32 x 32 tiles (the next best 17), at 64 11.7
// on 64 x 32 (17.9 on 64 x 64), at 128 19 on 128 x 32 (26 on 128 x 64), at 512 39 on 128 x 64 (51 on 64 x 64, 103 on 256 x
// 256); 4096 x 12288 at 128 rows 50 on 128 x 32 against 82; 100003 x 4096 at 32 rows 93 on 32 x 128 (135 on 32 x 32), at 64
// 106 on 64 x 128, at 256 243 on 256 x 256 (302 on 128 x 256).  `full` of the largest is that of a chip at its power limit.
struct Kind {
    int rows, cols, split, slots;
    double one, full;
};
enum { kMid32x32, kMid64x32, kMid128x32, kMid64x64, kMid128x64, kMid32x128, kMid64x128, kMid128x256, kTurns, kKinds };
constexpr Kind kKind[kKinds] = {
    {32, 32, 8, 1, 1.08, 1.08},  {64, 32, 8, 1, 1.55, 1.55},   {128, 32, 4, 1, 0.97, 0.97},
    {64, 64, 4, 1, 1.15, 1.15},  {128, 64, 4, 1, 1.75, 1.75},  {32, 128, 2, 2, 0.83, 1.45},
    {64, 128, 2, 2, 0.98, 1.65}, {128, 256, 1, 2, 1.07, 2.30}, {256, 256, 1, 1, 1.50, 1.90},
};
// Time of `tiles` row tiles over N weight rows of K, `slices` walks of 64 k each.
inline double kind_time(int kind, double tiles, int64_t N, int64_t slices, int n_cu) {
    const Kind& k = kKind[kind];
    const double blocks = tiles * double((N + k.cols - 1) / k.cols), steps = double((slices + k.split - 1) / k.split);
    const double whole = std::floor(blocks / (n_cu * k.slots)), rest = blocks - whole * n_cu * k.slots;
    const double last = rest <= 0 ? 0 : rest <= n_cu ? k.one * steps + 1.5 : k.full * steps + 1.5;
    return whole * (k.full * steps + 1.5) + last;
}
// Dense: T rows, `planes` walks over K.
inline int plan_dense(int64_t T, int64_t N, int64_t K, int planes, int n_cu) {
    int best = 0;
    double least = 1e30;
    for (int k = 0; k < kKinds; ++k) {
        const double t = kind_time(k, double((T + kKind[k].rows - 1) / kKind[k].rows), N, (K + 63) / 64 * planes, n_cu);
        if (t < least) least = t, best = k;
    }
    return best;
}
// Experts: `pairs` rows over n entries (their numbers of rows are known on the device only: as if each pair chose
// at random), N and K of one product.
inline double busy_entries(int n, int64_t pairs) { return n * (1.0 - std::exp(-double(pairs) / n)); }
inline double entry_tiles(int n, int64_t pairs, int rows) {
    const double busy = busy_entries(n, pairs), each = pairs / busy;
    return busy * (each <= rows / 2 ? 1.0 : each / rows + 0.5);
}
inline int plan_experts(int n, int64_t pairs, int64_t N, int64_t K, int n_cu) {
    int best = 0;
    double least = 1e30;
    for (int k = 0; k < kKinds; ++k) {
        const double t = kind_time(k, entry_tiles(n, pairs, kKind[k].rows), N, (K + 63) / 64, n_cu);
        if (t < least) least = t, best = k;
    }
    return best;
}
// The few-row kernel walks entries of more rows in blocks of 8: it takes the call where that is rare.
constexpr int kFewBlocks = 1024;
inline bool few_experts(int n, int64_t T, int64_t pairs, bool shared) {
    if (T <= kFewTokens) return true;
    return n > 0 && n + (pairs + (shared ? T : 0)) / 8 + 1 <= kFewBlocks && T <= 64 && pairs <= 4 * busy_entries(n, pairs);
}

}  // namespace i4
}  // namespace moe
