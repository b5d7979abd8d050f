// Prints the kernels that calls of the dense operators launch on a GPU of 256 compute units, one line
// a call, from the rules that the library itself uses (" split": with K split over workgroups).
// Calls, one a line, on the standard input:
//   m X LD WHOLE T N K Y   moe_i8_matmul: x and y types (MOE_A_*), elements between x's rows, whether
//                          those start on 16 bytes
//   8 T H I                moe_i8_ffn
//   f TYPE T H I           moe_dense_ffn (MOE_W_F32 or MOE_W_BF16)
//   b TYPE T H I           moe_dense_ffn_backward
//   q X WHOLE ROWS COLS    moe_i8_quantize
#include <cstdio>

#include "../expert_cached_moe_amd/csrc/dense_plan.h"

using namespace moe::dense;

static const int kCus = 256;
static const char* const kTile[] = {"Turns", "Tile<128, 128, 2, 2> ", "Tile<64, 64, 2, 2> "};
static const char* yes(bool v) { return v ? "true" : "false"; }

static void rows(int x, bool whole, long rows, int cols) {
    const RowThreads c = plan_rows(rows, cols);
    printf("k_quantize_rows<%s, %s, %d, %d>;", yes(x == kBF16), yes(whole), c.threads, c.hold);
}
// quant: 0, or the type of the numbers (1 bf16, 2 fp32)
static void few(int type, int epi, const Sizes& p, int quant) {
    const Few f = plan_few(p, elem_bytes(type), paired(epi), quant != 0, kCus);
    printf("k_few<%d, %d, %d, %d, %d, %s, %s, %s>;", type, epi, f.mt, f.r, quant, yes(f.walk), yes(f.walk && f.one),
           yes(!f.walk && !f.one));
}
static void tiles(const char* form, int type, int layout, int epi, const Tiling& c) {
    if (c.tile == kTile256) printf("k_mma_turns%s<%d, %d, %d>;", form, type, layout, epi);
    else printf("k_mma%s<%d, %d, %d, %s>%s;", form, type, layout, epi, kTile[c.tile], c.splits > 1 ? " split" : "");
    if (c.splits > 1) printf("k_join<%d, %d>;", type, epi);
}
static void product(int type, int layout, int epi, const Sizes& p, int64_t part) {
    if (layout == kNT && few_tokens(p, elem_bytes(type))) return few(type, epi, p, 0);
    tiles("", type, layout, epi, plan_tiles(p, nullptr, elem_bytes(type), part, kCus));
}

int main() {
    char line[256];
    while (fgets(line, sizeof line, stdin)) {
        int x, y, whole, T, N, K, H, I;
        long ld;
        if (sscanf(line, "m %d %ld %d %d %d %d %d", &x, &ld, &whole, &T, &N, &K, &y) == 7) {
            const int epi = y == kF32 ? kScale32 : kScale;
            const Sizes p{T, N, K};
            if (x != kI8 && quantise_inside(ld, whole, T, K, N)) few(kI8, epi, p, x == kBF16 ? 1 : 2);
            else {
                if (x != kI8) rows(x, whole, T, K);
                product(kI8, kNT, epi, p, i8_part_bytes(T));
            }
        } else if (sscanf(line, "8 %d %d %d", &T, &H, &I) == 3) {
            const Sizes g{T, 2 * I, H}, d{T, H, I};
            if (quantise_inside(H, true, T, H, 2 * I)) few(kI8, kGate8, g, 1);
            else rows(kBF16, true, T, H), product(kI8, kNT, kGate8, g, kPartBytes);
            if (quantise_inside(I, true, T, I, H)) few(kI8, kScale, d, 2);
            else rows(kF32, true, T, I), product(kI8, kNT, kScale, d, kPartBytes);
        } else if (sscanf(line, "f %d %d %d %d", &x, &T, &H, &I) == 4) {
            product(x, kNT, kGate, Sizes{T, 2 * I, H}, kPartBytes);
            product(x, kNT, kStore, Sizes{T, H, I}, kPartBytes);
        } else if (sscanf(line, "b %d %d %d %d", &x, &T, &H, &I) == 4) {
            product(x, kNN, kDGate, Sizes{T, I, H}, kPartBytes);
            const Sizes p{2 * I, H, T}, q{H, I, T};
            const Tiling c = plan_tiles(p, &q, elem_bytes(x), kPartBytes, kCus);
            tiles("_pair", x, kTN, kStore, c);
            product(x, kNN, kStore, Sizes{T, H, 2 * I}, kPartBytes);
        } else if (sscanf(line, "q %d %d %d %d", &x, &whole, &T, &K) == 4) {
            rows(x, whole, T, K);
        } else {
            fprintf(stderr, "unknown call: %s", line);
            return 1;
        }
        printf("\n");
    }
}
