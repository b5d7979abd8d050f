// Products with 4-bit weights (moe_i4_*): the argument block of their kernels and the launchers.
//
// A row of K weights: weight k = 2^(exp - 127) * s * (code - z), with the codes two a byte (element
// 2 i in the low half of byte i), and for each group of 32, 64 or 128 along K one word: the low
// byte an e4m3 number s, the high byte the zero point z.  s has four significant bits and code - z
// four, so every weight is exact in bf16: a product on the matrix cores is one with these weights.
#pragma once

#include <hip/hip_runtime.h>

#include "i4_plan.h"
#include "internal.h"

namespace moe {
namespace i4 {

constexpr int kMaxK = 1 << 20;        // offsets inside a tile of rows stay below 2 GiB
constexpr int kMaxCount = 1 << 23;    // rows: the threads of a launch fit 32 bits

// Rows of 4-bit weights: those of entry e begin `offset(e)` bytes on in all three arrays.
struct Rows {
    const uint8_t* codes;    // [N][K / 2]
    const uint16_t* words;   // by 16 rows: see word_at
    const uint8_t* exps;     // [N]
    int32_t groups;          // of a row
    int32_t shift;           // log2 of a group's length
};

// What a product computes and where its rows come from and go to.  (h is rounded to bf16 once, as moe_expert_ffn's: what
// the down product's matrix instructions take; with all its bits it would enter as three parts, three times the work.)
enum {
    kOut16 = 0,   // dense: row r of x to row r of out, bf16
    kOut32 = 1,   // the same in fp32
    kGateUp = 2,  // an expert's rows: x of the pair's token to h of its place in expert order
    kDown = 3,    // h of a place to the pair's own row
};

// Where the word of row n, group g lies among N rows: runs of 16 rows lie one behind the other, in each the
// words of a group side by side (the last run has what rows are left).  So the words of a matrix instruction's rows are one
// piece of a line, not one of each row: as [N][groups] their loads took 15% of the time of the products of few rows.
struct WordAt {
    int64_t first;           // of group 0
    int32_t step;            // from group to group
};
#ifdef __HIP__
__host__ __device__
#endif
inline WordAt word_at(int64_t n, int64_t N, int32_t groups) {
    const int64_t run = n & ~int64_t(15), left = N - run;
    return WordAt{run * groups + (n - run), left < 16 ? int32_t(left) : 16};
}

struct Product {
    const uint16_t* x;       // bf16 rows, 16-byte aligned, ldx elements apart
    int64_t ldx;
    int64_t plane;           // fp32 activations: three bf16 parts, `plane` elements apart
    int32_t planes;          // 1 or 3
    int32_t N, K;
    Rows w;
    void* out;
    int64_t ldo;
    int64_t T;
    // experts: entry i of the list, its places offsets[e] .. offsets[e + 1] - 1 in expert order
    const int32_t *offsets, *perm;
    int32_t top_k;
    int64_t stride, shared;  // bytes from slot to slot; of the shared blob from slot 0
};

hipError_t launch_i4_quantize(const void* x, int x_type, int64_t ld_x, int64_t rows, int32_t cols, int group, int zero,
                              uint8_t* q, uint16_t* words, uint8_t* exps, hipStream_t s);
// Rows of numbers to bf16 rows of K back to back (fp32: three parts, T K elements apart).
hipError_t launch_i4_activations(const void* x, int x_type, int64_t ld_x, int64_t T, int32_t K, uint16_t* out, hipStream_t s);
// Records of all row tiles of the list's entries (map_tiles at most), behind a count: int32 count, 3 of padding, records of
// entry, its tile of rows, its first place, its rows.
hipError_t launch_i4_map(const ExpertList& list, const int32_t* offsets, int64_t T, int top_k, int rows, void* map,
                         hipStream_t s);
// What the product computes (kOut16 ...) on tiles of a kind of i4_plan.h; experts: with the map for its rows.
hipError_t launch_i4_mid(int what, int kind, const Product& p, const ExpertList* list, const void* map, int64_t max_tiles,
                         hipStream_t s);
hipError_t launch_i4_turns(int what, const Product& p, const ExpertList* list, const void* map, int64_t max_tiles,
                           hipStream_t s);
// Few rows of x (few_dense); experts: up to 8 tokens.
hipError_t launch_i4_few(int what, const Product& p, const ExpertList* list, hipStream_t s);

}  // namespace i4
}  // namespace moe
