// Row quantisation to 8-bit integers: scale = max|row| / 127, code = row / scale to the nearest
// integer (ties to even, decided on the exact quotient).
//
// One workgroup a row.  The row is read once: up to HOLD vectors of 8 numbers a thread stay in
// registers between the maximum and the codes; longer rows read what is beyond again.  HOLD is
// the least that holds the row (its registers decide how many rows are in flight); rows too few
// to fill the chip take 1024 threads each.  Bound by memory: it reads the numbers and writes one
// byte for each: 8,192 x 12288 fp32 (503 MB) in 92-97 us, 5.3 TB/s, as a copy; 8,192 x 4096 bf16
// (101 MB) in 24-32 us; 8 x 4096 4.5 us, latency.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "dense_common.h"

namespace moe {
namespace dense {
namespace {

constexpr int kVec = kQuantizeVec;

// 8 numbers of a row from index i (in bounds, since cols is a multiple of 16)
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* row, int i, float (&v)[kVec]) {
    if constexpr (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(row) + i;
        if constexpr (VEC) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = dev::bf16_lo(w[j]);
                v[2 * j + 1] = dev::bf16_hi(w[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = bf16_f32(p[j]);
        }
    } else {
        const float* p = static_cast<const float*>(row) + i;
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 u = reinterpret_cast<const float4*>(p)[j];
                v[4 * j] = u.x, v[4 * j + 1] = u.y, v[4 * j + 2] = u.z, v[4 * j + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = p[j];
        }
    }
}

__device__ __forceinline__ void store8(int8_t* q, const float (&v)[kVec], float s, float inv) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j / 4] |= uint32_t(quantize_one(v[j], s, inv) & 255) << (8 * (j % 4));
    *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
}

template <bool BF16, bool VEC, int kThreads, int kHold>
__global__ void __launch_bounds__(kThreads) k_quantize_rows(const void* __restrict__ x, int64_t ld, int64_t rows,
                                                            int cols, int8_t* __restrict__ q,
                                                            float* __restrict__ scale) {
    __shared__ uint32_t s_top[kThreads / dev::kWave];
    const int tid = threadIdx.x;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const void* row = static_cast<const uint8_t*>(x) + r * ld * (BF16 ? 2 : 4);
        float v[kHold][kVec];
        uint32_t top = 0;
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            const int i = (h * kThreads + tid) * kVec;
            if (i < cols) {
                load8<BF16, VEC>(row, i, v[h]);
#pragma unroll
                for (int j = 0; j < kVec; ++j) top = max(top, __float_as_uint(v[h][j]) & 0x7FFFFFFFu);
            }
        }
        for (int i = (kHold * kThreads + tid) * kVec; i < cols; i += kThreads * kVec) {
            float t[kVec];
            load8<BF16, VEC>(row, i, t);
#pragma unroll
            for (int j = 0; j < kVec; ++j) top = max(top, __float_as_uint(t[j]) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int d = dev::kWave / 2; d >= 1; d >>= 1) top = max(top, uint32_t(__shfl_xor(int(top), d, dev::kWave)));
        if (tid % dev::kWave == 0) s_top[tid / dev::kWave] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / dev::kWave; ++w) top = max(top, s_top[w]);
        __syncthreads();
        const float s = row_scale(top), inv = inverse_scale(s);
        if (tid == 0) scale[r] = s;
        int8_t* qr = q + r * cols;
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            const int i = (h * kThreads + tid) * kVec;
            if (i < cols) store8(qr + i, v[h], s, inv);
        }
        for (int i = (kHold * kThreads + tid) * kVec; i < cols; i += kThreads * kVec) {
            float t[kVec];
            load8<BF16, VEC>(row, i, t);
            store8(qr + i, t, s, inv);
        }
    }
}

__global__ void __launch_bounds__(256) k_zero(uint4* p, int64_t n) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256)
        p[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace

namespace {
template <bool BF16, bool VEC>
void launch_rows(const void* x, int64_t ld, int64_t rows, int cols, int8_t* q, float* scale, hipStream_t s) {
    const dim3 grid(unsigned(rows < (1 << 20) ? rows : (1 << 20)));
    auto go = [&](auto threads_, auto hold_) {
        constexpr int THREADS = decltype(threads_)::value, HOLD = decltype(hold_)::value;
        hipLaunchKernelGGL((k_quantize_rows<BF16, VEC, THREADS, HOLD>), grid, dim3(THREADS), 0, s, x, ld, rows, cols, q,
                           scale);
    };
    typedef std::integral_constant<int, 256> Some;
    typedef std::integral_constant<int, 1024> Many;
    typedef std::integral_constant<int, 1> H1;
    typedef std::integral_constant<int, 2> H2;
    typedef std::integral_constant<int, 4> H4;
    const RowThreads c = plan_rows(rows, cols);
    if (c.threads == 256) {
        if (c.hold == 1) go(Some{}, H1{});
        else if (c.hold == 2) go(Some{}, H2{});
        else go(Some{}, H4{});
    } else {
        if (c.hold == 1) go(Many{}, H1{});
        else if (c.hold == 2) go(Many{}, H2{});
        else go(Many{}, H4{});
    }
}
}  // namespace

hipError_t launch_quantize(const void* x, int x_type, int64_t ld_x, int64_t rows, int32_t cols, int8_t* q,
                           float* scale, hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const bool bf16 = x_type == MOE_A_BF16;
    const int es = bf16 ? 2 : 4;
    // 16-byte loads when every row starts on 16 bytes
    const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld_x * es % 16 == 0;
    if (bf16 && vec) launch_rows<true, true>(x, ld_x, rows, cols, q, scale, s);
    else if (bf16) launch_rows<true, false>(x, ld_x, rows, cols, q, scale, s);
    else if (vec) launch_rows<false, true>(x, ld_x, rows, cols, q, scale, s);
    else launch_rows<false, false>(x, ld_x, rows, cols, q, scale, s);
    return hipGetLastError();
}

hipError_t launch_zero(void* p, int64_t n16, hipStream_t s) {
    if (n16 <= 0) return hipSuccess;
    const int64_t blocks = (n16 + 255) / 256;
    hipLaunchKernelGGL(k_zero, dim3(unsigned(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, static_cast<uint4*>(p),
                       n16);
    return hipGetLastError();
}

}  // namespace dense
}  // namespace moe
