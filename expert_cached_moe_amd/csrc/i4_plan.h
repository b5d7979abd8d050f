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
// Measured on bf16 x (dense, whole kernel): 4096 x 4096 at 32 rows 8.6 us on 32 x 32 tiles (17 on 128 x 32 and 64 x 64),
// at 128 11.1 on 64 x 32 (17.3 on 128 x 32), at 512 28 on 128 x 64 (34 on 128 x 32, 102 on 256 x 256); 4096 x 12288 at 256
// rows 48 on 128 x 32 (77 on 128 x 64); 16384 x 4096 at 1024 rows 121 on 256 x 256 (180 on 128 x 128); 100003 x 4096 at 32
// rows 77 on 32 x 128 (98 on 64 x 128, 111 on 32 x 32), at 64 105 on 64 x 128 (140), at 128 161 on 128 x 128 (190), at 256
// 249 on 256 x 256 (309).  `full` of the largest is that of a chip at its power limit.
struct Kind {
    int rows, cols, split, slots;
    double one, full;
};
enum { kMid32x32, kMid64x32, kMid128x32, kMid64x64, kMid128x64, kMid32x128, kMid64x128, kMid128x128, kTurns, kKinds };
constexpr Kind kKind[kKinds] = {
    {32, 32, 8, 1, 0.87, 0.87},  {64, 32, 8, 1, 1.10, 1.15},  {128, 32, 4, 1, 0.95, 0.95},
    {64, 64, 4, 1, 1.00, 1.00},  {128, 64, 4, 1, 1.45, 1.45}, {32, 128, 2, 3, 0.57, 1.80},
    {64, 128, 1, 3, 0.48, 1.20}, {128, 128, 1, 2, 0.95, 1.27}, {256, 256, 1, 1, 1.48, 1.93},
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
