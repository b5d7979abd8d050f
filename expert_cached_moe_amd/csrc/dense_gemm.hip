// Products of the dense operators: C[m][n] = sum_k A(m, k) B(n, k) with the operator's last
// steps applied to the sums in registers.
//
// k_product: 64 x 64 tiles, 256 threads of 4 x 4 sums, operands staged 16 k at a time in LDS as
// 32-bit values; any type, layout and size.  A thread's columns are 16 apart, so the gate and
// up columns of one inner index (interleaved in blocks of 16) belong to one thread.
#include <hip/hip_runtime.h>

#include "dense_common.h"

namespace moe {
namespace dense {
namespace {

constexpr int kT = 64, kTK = 16;

template <int TYPE, int LAYOUT, int EPI>
__global__ void __launch_bounds__(256) k_product(const Product p) {
    typedef typename Elem<TYPE>::T E;
    typedef typename Elem<TYPE>::Acc Acc;
    __shared__ __attribute__((aligned(16))) Acc as_[kTK][kT + 4];
    __shared__ __attribute__((aligned(16))) Acc bs_[kTK][kT + 4];
    const int tid = threadIdx.x;
    const int n_tiles = (p.N + kT - 1) / kT;
    const int64_t m0 = int64_t(blockIdx.x / n_tiles) * kT;
    const int n0 = int(blockIdx.x % n_tiles) * kT;
    const E* a = static_cast<const E*>(p.a);
    const E* b = static_cast<const E*>(p.b);
    const int tr = tid / 16, tc = tid % 16;
    Acc acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
    for (int k0 = 0; k0 < p.K; k0 += kTK) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // A: 64 rows x 16 k; consecutive threads along the contiguous dimension
            const int idx = q * 256 + tid;
            const int ar = LAYOUT == kTN ? idx % kT : idx / kTK, ak = LAYOUT == kTN ? idx / kT : idx % kTK;
            const bool aok = m0 + ar < p.M && k0 + ak < p.K;
            const int64_t ao = LAYOUT == kTN ? int64_t(k0 + ak) * p.lda + m0 + ar : (m0 + ar) * p.lda + k0 + ak;
            as_[ak][ar] = aok ? value(a[aok ? ao : 0]) : Acc(0);
            const int br = LAYOUT == kNT ? idx / kTK : idx % kT, bk = LAYOUT == kNT ? idx % kTK : idx / kT;
            const bool bok = n0 + br < p.N && k0 + bk < p.K;
            const int64_t bo = LAYOUT == kNT ? int64_t(n0 + br) * p.ldb + k0 + bk : int64_t(k0 + bk) * p.ldb + n0 + br;
            bs_[bk][br] = bok ? value(b[bok ? bo : 0]) : Acc(0);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTK; ++k) {
            Acc av[4], bv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                av[i] = as_[k][4 * tr + i];
                bv[i] = bs_[k][tc + 16 * i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (TYPE == kI8) acc[i][j] += av[i] * bv[j];
                    else acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
                }
        }
        __syncthreads();
    }
    E* out = static_cast<E*>(p.out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 4 * tr + i;
        if (m >= p.M) continue;
        if constexpr (EPI == kStore || EPI == kScale || EPI == kDGate) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tc + 16 * j;
                if (n >= p.N) continue;
                if constexpr (EPI == kStore) {
                    put(out + m * p.ldo + n, float(acc[i][j]));
                } else if constexpr (EPI == kScale) {
                    const float v = float(acc[i][j]) * p.row_scale[m] * p.col_scale[n];
                    if (p.out_f32) put(static_cast<float*>(p.out) + m * p.ldo + n, v);
                    else put(static_cast<uint16_t*>(p.out) + m * p.ldo + n, v);
                } else {
                    // n is an inner index: its gate column is (n / 16) * 32 + n % 16
                    const int64_t g = m * 2 * p.N + (n / 16) * 32 + n % 16;
                    const E* gu = static_cast<const E*>(p.gu);
                    const float gate = value(gu[g]), up = value(gu[g + 16]), s = sigmoid(gate);
                    put(out + g, float(acc[i][j]) * up * silu_grad(gate, s));
                    put(out + g + 16, float(acc[i][j]) * gate * s);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const int n = n0 + tc + 16 * j;             // gate column; up is n + 16
                if (n >= p.N) continue;                     // (N is a multiple of 32)
                const int inner = n / 32 * 16 + n % 16;
                float g = float(acc[i][j]), u = float(acc[i][j + 1]);
                if constexpr (EPI == kGate8) {
                    g = g * p.row_scale[m] * p.col_scale[n];
                    u = u * p.row_scale[m] * p.col_scale[n + 16];
                    put(static_cast<float*>(p.out) + m * p.ldo + inner, silu(g) * u);
                } else {
                    if (p.gu) {
                        put(static_cast<E*>(p.gu) + m * p.N + n, g);
                        put(static_cast<E*>(p.gu) + m * p.N + n + 16, u);
                    }
                    put(out + m * p.ldo + inner, silu(g) * u);
                }
            }
        }
    }
}

template <int TYPE, int LAYOUT, int EPI>
hipError_t launch_simple(const Product& p, hipStream_t s) {
    const int64_t tiles = (p.M + kT - 1) / kT * ((p.N + kT - 1) / kT);
    if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_product<TYPE, LAYOUT, EPI>), dim3(unsigned(tiles)), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product(int type, int layout, int epi, const Product& p, hipStream_t s) {
    if (p.M <= 0 || p.N <= 0) return hipSuccess;
    if (type != kF32)
        return layout == kNT && few_tokens(p, type == kI8 ? 1 : 2) ? launch_few(type, epi, p, s)
                                                                   : launch_mma(type, layout, epi, p, s);
    if (layout == kNT && epi == kStore) return launch_simple<kF32, kNT, kStore>(p, s);
    if (layout == kNT && epi == kGate) return launch_simple<kF32, kNT, kGate>(p, s);
    if (layout == kNN && epi == kStore) return launch_simple<kF32, kNN, kStore>(p, s);
    if (layout == kNN && epi == kDGate) return launch_simple<kF32, kNN, kDGate>(p, s);
    if (layout == kTN && epi == kStore) return launch_simple<kF32, kTN, kStore>(p, s);
    return hipErrorInvalidValue;
}

}  // namespace dense
}  // namespace moe
