// Launchers of the dense operators (moe_i8_*, moe_dense_*), and the argument block of their
// product kernels.  Types, layouts, epilogues and the rules that choose a kernel: dense_plan.h.
#pragma once

#include <hip/hip_runtime.h>

#include "dense_plan.h"
#include "internal.h"

namespace moe {
namespace dense {

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
    Sizes sizes() const { return Sizes{M, N, K}; }
};

// Compute units of the current device.
int compute_units();

// One product on stream s: type kF32 / kBF16 / kI8, layout kNT / kNN, epilogue as above.
hipError_t launch_product(int type, int layout, int epi, const Product& p, hipStream_t s);
// Two products kTN, kStore of the same K > 0 in one launch; they share p's scratch.
hipError_t launch_gradients(int type, const Product& p, const Product& q, hipStream_t s);
// Few tokens, NT.  With quant, a holds numbers of x_type (16-byte aligned rows) that the kernel
// quantises for itself.
hipError_t launch_few(int type, int epi, const Product& p, hipStream_t s, int x_type = 0, bool quant = false);
// rows of cols numbers to codes and scales; x_type MOE_A_F32 / MOE_A_BF16
hipError_t launch_quantize(const void* x, int x_type, int64_t ld_x, int64_t rows, int32_t cols, int8_t* q,
                           float* scale, hipStream_t s);
// n16 16-byte units of zeros
hipError_t launch_zero(void* p, int64_t n16, hipStream_t s);

}  // namespace dense
}  // namespace moe
