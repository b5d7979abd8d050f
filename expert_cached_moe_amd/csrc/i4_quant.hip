// Rows of numbers to 4-bit codes with group scales, and activations to the rows that the products read.
//
// A thread takes 32 numbers of a row at a time; a group is 1, 2 or 4 neighbouring threads.  The row is
// read twice, first for its groups' spans t = (largest - smallest) / 15, or largest magnitude / 7, whose
// largest decides the row's power of two S (the least with t <= 448 S), then for the codes.  The group's
// scale s is t / S as an e4m3 number, rounded to nearest even, or up where there are zero points: then
// the span is at most 15 steps (to nearest it could be 15.9 and lose a whole step); without them the
// largest magnitude lies below 7.5 steps either way (e4m3 numbers are at most 1/17 off).  Quotients are
// formed in 64 bits and rounded half to even.  Done once for a model's weights: 8192 x 4096 bf16 weights 86 us,
// 100003 x 4096 950-1090 (0.8 TB/s read in effect; 17 and 200 at a copy's rate).  Bound by its loads: the numbers of a piece are
// read under branches of their own, two at most by one load, each waited for before the next, and rows shorter than 8192 leave
// threads idle.  The 64-bit divisions are some 17 us of the 86 (20 operations each).  Activations of 77 x 1568 fp32 numbers 3.
#include <hip/hip_runtime.h>

#include "i4_common.h"

namespace moe {
namespace i4 {
namespace {

using dev::kWave;

constexpr int kThreads = 256;

__device__ __forceinline__ float number(const float* p) { return *p; }
__device__ __forceinline__ float number(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }

// t / S as e4m3 (bits), 0 <= t / S <= 448 (1 + 2^-52)
__device__ __forceinline__ uint32_t e4m3_of(double u, bool up) {
    if (!(u > 0.0)) return 0;
    int e;
    frexp(u, &e);                                    // 2^(e - 1) <= u < 2^e
    if (e < -5) e = -5;                              // below 2^-6: subnormal, steps of 2^-9
    const double unit = ldexp(1.0, e - 4), n = up ? ceil(u / unit) : rint(u / unit);
    // n steps of 2^(e - 4): 8..16, or 0..8 for subnormal numbers; 16 carries into the exponent by itself
    const uint32_t bits = uint32_t((e + 5) * 8 + int(n));
    return bits < 0x7Eu ? bits : 0x7Eu;
}

// The numbers of 32 weights' group: largest and smallest with 0.
struct Span {
    double lo, hi;
};

template <class E>
__global__ __launch_bounds__(kThreads) void k_i4_quantize(const E* __restrict__ x, int64_t ld, int cols, int group, int zero,
                                                          uint8_t* __restrict__ q, uint16_t* __restrict__ words,
                                                          uint8_t* __restrict__ exps) {
    __shared__ double s_top[kThreads / kWave];
    __shared__ int s_bad;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, pieces = cols / 32, per = group / 32, groups = (pieces + per - 1) / per;
    const E* xr = x + row * ld;
    const double steps = zero ? 15.0 : 7.0;
    const WordAt at = word_at(row, gridDim.x, groups);
    bool bad = false;
    auto read = [&](int p, float (&v)[32]) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = p < pieces ? number(xr + p * 32 + i) : 0.0f;
    };
    auto span = [&](const float (&v)[32]) {
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            bad |= !(fabsf(v[i]) < 1.329227995784916e36f);        // 2^120
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
        }
        for (int d = 1; d < per; d <<= 1) {
            lo = fminf(lo, __shfl_xor(lo, d, kWave));
            hi = fmaxf(hi, __shfl_xor(hi, d, kWave));
        }
        return Span{double(lo), double(hi)};
    };
    auto width = [&](const Span& g) { return (zero ? g.hi - g.lo : fmax(g.hi, -g.lo)) / steps; };
    if (tid == 0) s_bad = 0;
    double top = 0.0;
    float v[32];
    for (int p0 = 0; p0 < pieces; p0 += kThreads) {
        read(p0 + tid, v);
        top = fmax(top, width(span(v)));
    }
#pragma unroll
    for (int d = kWave / 2; d >= 1; d >>= 1) top = fmax(top, __shfl_xor(top, d, kWave));
    if (tid % kWave == 0) s_top[tid / kWave] = top;
    __syncthreads();
    if (bad) s_bad = 1;
    __syncthreads();
    for (int w = 0; w < kThreads / kWave; ++w) top = fmax(top, s_top[w]);
    int e = 0;
    const double m = frexp(top / 448.0, &e);
    if (m == 0.5) --e;
    const bool nothing = s_bad || !(top > 0.0) || e < -100;
    const double S = nothing ? 0.0 : ldexp(1.0, e);
    if (tid == 0) exps[row] = s_bad ? 255 : nothing ? 0 : uint8_t(e + 127);
    for (int p0 = 0; p0 < pieces; p0 += kThreads) {
        const int p = p0 + tid;
        if (pieces > kThreads) read(p, v);
        const Span g = span(v);
        const uint32_t s = nothing ? 0u : e4m3_of(width(g) / S, zero);
        const double d = S * double(__builtin_amdgcn_cvt_f32_fp8(int(s), 0));
        const bool live = d > 0.0;
        int z = 8;
        if (zero && live) z = int(fmin(rint(-g.lo / d), 15.0));
        uint32_t c[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
        if (live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int n = int(fmin(fmax(rint(double(v[i]) / d) + double(z), 0.0), 15.0));
                c[i / 8] = (i % 8 ? c[i / 8] : 0u) | uint32_t(n) << (4 * (i % 8));
            }
        }
        if (p < pieces) {
            *reinterpret_cast<uint4*>(q + row * (cols / 2) + p * 16) = make_uint4(c[0], c[1], c[2], c[3]);
            if (p % per == 0) words[at.first + int64_t(p / per) * at.step] = uint16_t(s | uint32_t(z) << 8);
        }
    }
}

// 8 numbers a thread.  fp32: x = hi + mid + lo, each the upper 8 significant bits of what is left (cut, not
// rounded, so nothing overflows); an infinity or a NaN stays in the first part.
template <class E>
__global__ __launch_bounds__(kThreads) void k_i4_activations(const E* __restrict__ x, int64_t ld, int64_t T, int K,
                                                             uint16_t* __restrict__ out) {
    const int64_t per = K / 8;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < T * per; i += int64_t(gridDim.x) * kThreads) {
        const int64_t t = i / per;
        const int k = int(i % per) * 8;
        const E* xr = x + t * ld + k;
        uint32_t part[sizeof(E) == 4 ? 3 : 1][4];
    #pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = number(xr + j);
    #pragma unroll
            for (int a = 0; a < (sizeof(E) == 4 ? 3 : 1); ++a) {
                const uint32_t b = __float_as_uint(v) >> 16;
                part[a][j / 2] = j % 2 ? part[a][j / 2] | b << 16 : b;
                const bool whole = fabsf(v) < INFINITY;
                v = whole ? v - __uint_as_float(b << 16) : 0.0f;
                // (a NaN whose payload lies in the lower bits would be cut to an infinity)
                if (!whole && a == 0 && (__float_as_uint(number(xr + j)) & 0x7FFFFFFFu) > 0x7F800000u)
                    part[a][j / 2] |= j % 2 ? 0x400000u : 0x40u;
            }
        }
    #pragma unroll
        for (int a = 0; a < (sizeof(E) == 4 ? 3 : 1); ++a)
            *reinterpret_cast<uint4*>(out + a * T * K + t * K + k) = make_uint4(part[a][0], part[a][1], part[a][2], part[a][3]);
    }
}

}  // namespace

hipError_t launch_i4_quantize(const void* x, int x_type, int64_t ld_x, int64_t rows, int32_t cols, int group, int zero,
                              uint8_t* q, uint16_t* words, uint8_t* exps, hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const dim3 grid{unsigned(rows)}, block{kThreads};
    if (x_type == MOE_A_F32)
        hipLaunchKernelGGL((k_i4_quantize<float>), grid, block, 0, s, static_cast<const float*>(x), ld_x, cols, group, zero, q,
                           words, exps);
    else
        hipLaunchKernelGGL((k_i4_quantize<uint16_t>), grid, block, 0, s, static_cast<const uint16_t*>(x), ld_x, cols, group,
                           zero, q, words, exps);
    return hipGetLastError();
}

hipError_t launch_i4_activations(const void* x, int x_type, int64_t ld_x, int64_t T, int32_t K, uint16_t* out, hipStream_t s) {
    const int64_t items = T * (K / 8), blocks = (items + kThreads - 1) / kThreads;
    if (items == 0) return hipSuccess;
    const dim3 grid{unsigned(blocks < (1 << 20) ? blocks : 1 << 20)}, block{kThreads};
    if (x_type == MOE_A_F32)
        hipLaunchKernelGGL((k_i4_activations<float>), grid, block, 0, s, static_cast<const float*>(x), ld_x, T, K, out);
    else
        hipLaunchKernelGGL((k_i4_activations<uint16_t>), grid, block, 0, s, static_cast<const uint16_t*>(x), ld_x, T, K, out);
    return hipGetLastError();
}

}  // namespace i4
}  // namespace moe
