// Launchers of the dense operators (moe_i8_*, moe_dense_*), and the argument block of their
// product kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "internal.h"

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

struct Product {
    const void* a;
    const void* b;
    int64_t lda, ldb;           // elements between rows of A and B
    int64_t M;
    int32_t N, K;
    void* out;
    int64_t ldo;                // elements between rows of out
    int32_t vec_out;            // kScale, kScale32: every even column lies on 4 bytes
    const float* row_scale;     // integer products
    const float* col_scale;
    void* part;                 // scratch for partial sums of part_bytes (0: none)
    int64_t part_bytes;
    void* gu;                   // kGate: written when not null; kDGate: read; rows of 2 I elements
    uint8_t* gu_low;            // bf16: their lower 8 of 24 bits
};

// Scratch for partial sums: products with few tiles are split along K to fill the chip.
constexpr int64_t kPartBytes = int64_t(32) << 20;
// Compute units of the current device.
int compute_units();

// One product on stream s: type kF32 / kBF16 / kI8, layout kNT / kNN, epilogue as above.
hipError_t launch_product(int type, int layout, int epi, const Product& p, hipStream_t s);
// Two products kTN, kStore of the same K > 0 in one launch; they share p's scratch.
hipError_t launch_gradients(int type, const Product& p, const Product& q, hipStream_t s);
// few tokens, NT: the weight stream.  It takes up to 16 tokens, and up to 32 while the weights
// are 32 MiB at most: 100003 x 4096 codes take it 71 us at 16 tokens and 101 at 24, the tiles 106
// and 93-108; a 4096 x 12288 bf16 block 66 and 110 us against 87 and 88; 8192 x 4096 codes 8.6
// and 13.7 us against 14.6; 2048 x 2048 codes 5.2 and 6.0 against 7.3.
constexpr int kFewTokens = 32;
inline bool few_tokens(const Product& p, int es) {
    return p.M <= 16 || (p.M <= kFewTokens && int64_t(p.N) * p.K * es <= (int64_t(32) << 20));
}
// With quant, a holds numbers of x_type (16-byte aligned rows) that the kernel quantises for
// itself: integer products of M <= 8 tokens with M * K <= kFewQuant.
constexpr int kFewQuant = 16384;
hipError_t launch_few(int type, int epi, const Product& p, hipStream_t s, int x_type = 0, bool quant = false);
// rows of cols numbers to codes and scales; x_type MOE_A_F32 / MOE_A_BF16
hipError_t launch_quantize(const void* x, int x_type, int64_t ld_x, int64_t rows, int32_t cols, int8_t* q,
                           float* scale, hipStream_t s);
// n16 16-byte units of zeros
hipError_t launch_zero(void* p, int64_t n16, hipStream_t s);

}  // namespace dense
}  // namespace moe
