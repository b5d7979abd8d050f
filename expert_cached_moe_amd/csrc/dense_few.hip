// Products of few tokens (up to 64) with weights contiguous along K: the weight stream.
//
// With few tokens the time is that of reading the weights once.  A workgroup owns 16 R rows of
// the weights and all tokens; its waves split K among them by 128-byte slices (wave w takes
// slices w, w + W, ...: together they read whole runs of each row).  A wave loads weights and
// activations straight into the registers of the 16x16 matrix instructions (16 rows of 64
// bytes a load, two loads make the lines whole), with kDepth slices in flight; nothing is
// staged, and the waves meet once, to add their sums in LDS in a fixed order.  The matrix
// instruction costs the same for 1 token as for 16.
//
// QUANT: x comes as numbers and is quantised on the way, by every workgroup for itself: the
// codes (at most kMaxCodes bytes) are kept in LDS.  That repeats T K conversions in every
// workgroup but saves a launch and a pass through memory.
#include <hip/hip_runtime.h>

#include "dense_common.h"
#include "dense_epilogue.h"

namespace moe {
namespace dense {
namespace {

using dev::kWave;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
constexpr uint32_t kOutside = 0xFFFFFFF0u, kRange = 0x80000000u;
constexpr int kSlice = 128, kDepth = 4;

__device__ __forceinline__ dev::f32x4 mma(const dev::u32x4& a, const dev::u32x4& b, const dev::f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mma(const dev::u32x4& a, const dev::u32x4& b, const i32x4& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}
template <int TYPE> struct FewAcc { typedef dev::f32x4 T; };
template <> struct FewAcc<kI8> { typedef i32x4 T; };

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, kRange, 0x00027000);
}
__device__ __forceinline__ dev::u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(dev::u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// MT: 16-token tiles; R: 16-row weight tiles of a workgroup (2 for the gated epilogues: a
// block of 16 gate rows and its 16 up rows)
template <int TYPE, int EPI, int MT, int R>
__global__ void __launch_bounds__(512) k_few(const Product p) {
    typedef typename FewAcc<TYPE>::T Acc;
    constexpr int ES = TYPE == kI8 ? 1 : 2;
    constexpr bool GATE = EPI == kGate || EPI == kGate8;
    static_assert(!GATE || R == 2, "gate and up tiles");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, waves = blockDim.x / kWave;
    const int n0 = blockIdx.x * 16 * R, T = int(p.M);
    const uint32_t kb = uint32_t(p.K) * ES;
    const __amdgpu_buffer_rsrc_t rw = rsrc(static_cast<const uint8_t*>(p.b) + int64_t(n0) * p.ldb * ES);
    const __amdgpu_buffer_rsrc_t rx = rsrc(static_cast<const uint8_t*>(p.a));
    uint32_t wo[R], xo[MT];
#pragma unroll
    for (int r = 0; r < R; ++r) wo[r] = uint32_t(min(r * 16 + lane % 16, p.N - 1 - n0)) * uint32_t(p.ldb * ES);
#pragma unroll
    for (int m = 0; m < MT; ++m) xo[m] = uint32_t(min(m * 16 + lane % 16, T - 1)) * uint32_t(p.lda * ES);
    Acc acc[MT][R];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[m][r] = Acc{0, 0, 0, 0};
    const uint32_t stride = uint32_t(waves) * kSlice;
    for (uint32_t s = wave * kSlice; s < kb; s += stride * kDepth) {
        dev::u32x4 w[kDepth][2][R], x[kDepth][2][MT];
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t k = s + d * stride + h * 64 + (lane / 16) * 16;
                const bool in = k < kb;            // past K: both operands read zeros
#pragma unroll
                for (int r = 0; r < R; ++r) w[d][h][r] = load16(rw, in ? wo[r] + k : kOutside);
#pragma unroll
                for (int m = 0; m < MT; ++m) x[d][h][m] = load16(rx, in ? xo[m] + k : kOutside);
            }
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[m][r] = mma(w[d][h][r], x[d][h][m], acc[m][r]);
    }
    Acc* red = reinterpret_cast<Acc*>(lds);        // [wave][m][r][lane]
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) red[((wave * MT + m) * R + r) * kWave + lane] = acc[m][r];
    __syncthreads();
    constexpr int PER = GATE ? 2 : 1, ITEMS = MT * R / PER;    // results of a wave at a time
    for (int it = wave; it < ITEMS; it += waves) {
        Acc sum[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            sum[q] = red[(it * PER + q) * kWave + lane];
            for (int v = 1; v < waves; ++v) sum[q] += red[(v * MT * R + it * PER + q) * kWave + lane];
        }
        const int m = it * PER / R, r = it * PER % R;
        const int t = m * 16 + lane % 16, n = n0 + r * 16 + 4 * (lane / 16);
        if (t >= T || n >= p.N) continue;
        if constexpr (EPI == kGate) finish_gate(p, t, n, sum[0], sum[PER - 1]);
        else if constexpr (EPI == kGate8) finish_gate8(p, t, n, sum[0], sum[PER - 1]);
        else if constexpr (EPI == kStore) finish_store(p, t, n, sum[0]);
        else finish_scale(p, t, n, sum[0]);
    }
}

template <int TYPE, int EPI, int MT, int R>
hipError_t launch_few_as(const Product& p, hipStream_t s) {
    const int64_t groups = (int64_t(p.N) + 16 * R - 1) / (16 * R);
    const int waves = 8;
    hipLaunchKernelGGL((k_few<TYPE, EPI, MT, R>), dim3(unsigned(groups)), dim3(waves * kWave),
                       waves * MT * R * kWave * 16, s, p);
    return hipGetLastError();
}

template <int TYPE, int EPI>
hipError_t choose_few(const Product& p, hipStream_t s) {
    constexpr bool GATE = EPI == kGate || EPI == kGate8;
    const int mt = int((p.M + 15) / 16);
    if constexpr (!GATE) {
        // one row tile a workgroup while that is what fills the chip
        if (p.N < 16 * 1024 && mt == 1) return launch_few_as<TYPE, EPI, 1, 1>(p, s);
    }
    if (mt == 1) return launch_few_as<TYPE, EPI, 1, 2>(p, s);
    if (mt == 2) return launch_few_as<TYPE, EPI, 2, 2>(p, s);
    return launch_few_as<TYPE, EPI, 4, 2>(p, s);
}

}  // namespace

hipError_t launch_few(int type, int epi, const Product& p, hipStream_t s) {
    if (p.M > kFewTokens) return hipErrorInvalidValue;
    if (type == kI8) {
        if (epi == kScale) return choose_few<kI8, kScale>(p, s);
        if (epi == kGate8) return choose_few<kI8, kGate8>(p, s);
    } else if (type == kBF16) {
        if (epi == kStore) return choose_few<kBF16, kStore>(p, s);
        if (epi == kGate) return choose_few<kBF16, kGate>(p, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace dense
}  // namespace moe
