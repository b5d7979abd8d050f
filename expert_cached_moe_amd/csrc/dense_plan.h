// Which kernel a product of the dense operators takes: rules on sizes, types and the number of
// compute units.  Host code without HIP, so that a program without a GPU can list what they choose.
#pragma once

#include <cstdint>

namespace moe {
namespace dense {

constexpr int kMaxKI8 = 131056;       // 128 * 128 * K stays below 2^31

// Element type of the operands of a product.
enum { kF32 = 0, kBF16 = 1, kI8 = 2 };

// Which operands of C[m][n] = sum_k A(m, k) B(n, k) have k as their contiguous dimension: NT
// both (A [M][K], B [N][K]); NN only A (B [K][N]); TN neither (A [K][M], B [K][N]).
enum { kNT = 0, kNN = 1, kTN = 2 };

// What becomes of the sums.
enum {
    kStore = 0,   // out[m][n] = acc, rounded to the operands' type
    kScale = 1,   // out[m][n] = acc * row_scale[m] * col_scale[n] (integer products), rounded to bf16
    kGate = 2,    // columns are interleaved gate / up: out[m][i] = silu(g) * u; gu[m][n] = acc if kept
    kGate8 = 3,   // the same from integer sums and scales, out in fp32
    kScale32 = 5, // as kScale, out in fp32
    kDGate = 4,   // acc = dh[m][i]: out[m][..] = dg, du interleaved, from gu (pre-activations)
};

// Epilogues that pair two runs of 16 columns.
constexpr bool paired(int epi) { return epi == kGate || epi == kGate8; }
inline int elem_bytes(int type) { return type == kI8 ? 1 : type == kBF16 ? 2 : 4; }

struct Sizes {
    int64_t M;
    int32_t N, K;
};

// Scratch for partial sums: products with few tiles are split along K to fill the chip.
constexpr int64_t kPartBytes = int64_t(32) << 20;
// Elements between the rows of a partial sum: a multiple of 8 from N up.
constexpr int64_t part_ld(int32_t N) { return (int64_t(N) + 7) / 8 * 8; }
// Scratch of moe_i8_matmul for partial sums.  More than kSplitTokens tokens are never split: wide
// outputs fill the chip unsplit; narrow ones would gain (2048 x 256 x 8192, by the model of plan_tiles,
// 24.5 us against 15.3 split), at the price of 32 MiB more for every workspace.
constexpr int64_t kSplitTokens = 1024;
inline int64_t i8_part_bytes(int64_t T) { return T > kSplitTokens ? 0 : kPartBytes; }

// ---------------------------------------------------------------- row quantisation

// Threads a row, and vectors of 8 numbers that each holds in registers between the maximum and the
// codes: the least that hold the row, and 1024 threads for rows too few to fill the chip.
constexpr int kQuantizeVec = 8;
struct RowThreads {
    int threads, hold;
};
inline RowThreads plan_rows(int64_t rows, int32_t cols) {
    const int64_t some = 256 * kQuantizeVec, many = 1024 * kQuantizeVec;
    if (rows <= 512 && cols > some) return RowThreads{1024, cols <= many ? 1 : cols <= 2 * many ? 2 : 4};
    if (cols <= 4 * some) return RowThreads{256, cols <= some ? 1 : cols <= 2 * some ? 2 : 4};
    return RowThreads{1024, 2};
}

// ---------------------------------------------------------------- few tokens

// Whether a product kNT goes to the few-token kernel, the weight stream.  It takes up to 16 tokens,
// and up to 32 while the weights are 32 MiB at most: 100003 x 4096 codes take it 71 us at 16 tokens
// and 101 at 24, the tiles 106 and 93-108; a 4096 x 12288 bf16 block 66 and 110 us against 87 and
// 88; 8192 x 4096 codes 8.6 and 13.7 us against 14.6; 2048 x 2048 codes 5.2 and 6.0 against 7.3.
constexpr int kFewTokens = 32;
inline bool few_tokens(const Sizes& p, int es) {
    return p.M <= 16 || (p.M <= kFewTokens && int64_t(p.N) * p.K * es <= (int64_t(32) << 20));
}
// Whether the few-token kernel quantises x itself: few enough numbers; rows (ld elements apart) that
// can be read 16 bytes at a time (whole_rows), offsets below its range; and few enough outputs, since
// every 16 of them convert all numbers again (4096 columns, one token: 8192 outputs 8.5 us against
// 10.8 in two launches, 100003 77 against 67; 4 tokens: 4096 9.3 against 9.7, 6144 12.8 against 11.4,
// 100003 107 against 68; 1024 columns, 8 tokens, 4096 outputs 6.3 against 8.2).  Between the two
// borders a little is given up: 24576 outputs at one token take 21.0 in two launches, 20.3 inside.
constexpr int kFewQuant = 16384;
inline bool quantise_inside(int64_t ld, bool whole_rows, int32_t T, int32_t K, int32_t N) {
    const int64_t results = int64_t(T) * N;
    return whole_rows && T <= 8 && int64_t(T) * K <= kFewQuant && (T == 1 || ld < (int64_t(1) << 25)) &&
           (results <= 16384 || (N <= 16384 && results * K <= int64_t(1) << 25));
}

// The few-token kernel: mt 8-token tiles, r 8-row weight tiles a workgroup; walk over groups of rows;
// one: K is one pass (kFewPass bytes of each row).
constexpr int kFewPass = 4096;
struct Few {
    int mt, r;
    bool walk, one;
};
inline Few plan_few(const Sizes& p, int es, bool gated, bool quant, int n_cu) {
    const int tiles = int((p.M + 7) / 8), mt = tiles > 2 ? 4 : tiles;
    const bool one = int64_t(p.K) * es <= kFewPass;
    if (quant) return Few{1, 2, false, one};
    // 16 rows a workgroup leave CUs idle below N = 4096: 8 then
    if (!gated && p.N < 4096 && mt == 1) return Few{1, 1, false, one};
    // A walk of 32 rows at a time, one workgroup a CU, keeps the stream going from group to group and
    // halves the reading of x: it wins where the rows fill the chip, in one pass of K (100003 x 4096
    // codes 64 us at one token, 66 at 8 and 71 at 16, against 66, 70 and 86 with 16 rows) and, with
    // three groups or more for every CU, in several (100003 x 8192 136 and 169 at 8 and 16 tokens
    // against 177 and 222; 16384 x 16384 63 at 12 tokens against 61; at 2 tokens 139 against 118).
    const bool wide = mt <= 2 && p.N >= 8192 && (one || (p.M > 2 && p.N >= 96 * n_cu));
    return Few{mt, wide ? 4 : 2, mt > 1 || wide, one};
}

// ---------------------------------------------------------------- tiles on the matrix cores

constexpr int kSliceBytes = 128;      // of K in a slice

// Tile and split of K: the least of the times that a model fitted to measurements gives, in us.
// A slice takes `slice` and `more` for each further workgroup on its CU (up to `slots`), a tile
// `tile` to start and finish; a split costs a second kernel and its partial sums both ways.
// Measured (8-bit codes, whole call): 300 x 4096 x 4096: 256-tiles 40 us, 128 20, 64 13, 128
// split in two 23; 2000 x 4096 x 4096: 44, 34, 50; 1024 x 8192 x 8192: 74, 63, 94; 100 x 8192 x
// 4096: 64-tiles 19, split in two 16.6, in eight 21.  fp32: eight times the matrix time.  Four
// stages instead of two on the smaller tiles, and 256 x 128 tiles in turns, gained nothing.  It ranks
// tiles; as a time it can be far off (777 x 2051 x 1552 codes: 7.9 by the model, 11.7 measured).
struct Tiling {
    int tile, splits;            // tile: kTile256, kTile128, kTile64
};
enum { kTile256 = 0, kTile128 = 1, kTile64 = 2 };
inline Tiling plan_tiles(const Sizes& p, const Sizes* q, int es, int64_t part_bytes, int64_t n_cu) {
    struct Kind { int bm, bn, slots; double slice, more, tile; };
    static const Kind half[] = {{256, 256, 1, 1.3, 0.0, 6.0}, {128, 128, 2, 0.68, 0.28, 3.0}, {64, 64, 4, 0.36, 0.13, 1.5}};
    static const Kind fp32[] = {{256, 256, 1, 8.6, 0.0, 6.0}, {128, 128, 2, 2.3, 2.1, 3.0}, {64, 64, 4, 0.65, 0.55, 1.5}};
    const Kind* kinds = es == 4 ? fp32 : half;
    const int64_t nk = (int64_t(p.K) * es + kSliceBytes - 1) / kSliceBytes;
    static const int splits[] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, 24, 28, 32};
    const int64_t one = p.M * part_ld(p.N) + (q ? q->M * part_ld(q->N) + 64 : 0);       // numbers of one split's sums
    Tiling best{kTile256, 1};
    double best_t = 1e30;
    for (int c = 0; c < 3; ++c) {
        const Kind& k = kinds[c];
        auto count = [&](const Sizes& r) { return (r.M + k.bm - 1) / k.bm * ((r.N + k.bn - 1) / k.bn); };
        const int64_t tiles = count(p) + (q ? count(*q) : 0);
        for (int sp : splits) {
            if (sp > 1 && sp * 4 > nk) break;
            const int64_t sums = one * sp, share = (nk + sp - 1) / sp;
            // (256-tiles that could be split and still fill the chip would need more scratch)
            if (sp > 1 && (sums * 4 > part_bytes || c == kTile256)) break;
            if (share * (sp - 1) >= nk) continue;            // every split has slices
            const int64_t groups = tiles * sp, rounds = (groups + n_cu * k.slots - 1) / (n_cu * k.slots);
            const int64_t on_cu = (groups + n_cu - 1) / n_cu < k.slots ? (groups + n_cu - 1) / n_cu : k.slots;
            const double t = rounds * (share * (k.slice + k.more * (on_cu - 1)) + k.tile) + (sp > 1 ? 3.0 + sums * 1.4e-6 : 0.0);
            if (t < best_t) best_t = t, best = Tiling{c, sp};
        }
    }
    return best;
}

}  // namespace dense
}  // namespace moe
