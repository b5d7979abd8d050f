// Device helpers of the dense operators' kernels: the gated activation with its derivative,
// 8-bit quantisation of one value, and typed loads and stores.
#pragma once

#include <hip/hip_runtime.h>

#include "dense.h"
#include "device_common.h"

namespace moe {
namespace dense {

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

template <int TYPE> struct Elem;
template <> struct Elem<kF32> { typedef float T; typedef float Acc; };
template <> struct Elem<kBF16> { typedef uint16_t T; typedef float Acc; };
template <> struct Elem<kI8> { typedef int8_t T; typedef int Acc; };

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = dev::f32_to_bf16_bits(v); }

// 1 / (1 + e^-z): e^-z overflows to infinity for z < -88.7, which gives the limit 0.
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }
// z / (1 + e^-z) within four steps of fp32 for z >= -87, from the hardware's exp2 and reciprocal (a step
// each): the rounding of z log2(e), which grows with z, and log2(e)'s own are carried into the result.
// From about -87.3 down, where e^z leaves the normal numbers, the result is -0 (the value's size is
// below 1.1e-36).  The exponent's argument is held to 128 on both sides: past that the result is z
// or -0 in any case, and z log2(e) itself overflows from 2.4e38 on.  (With expf and a division gate and
// up of the 4096 x 12288 8-bit block take 745 us instead of 711 for 8,192 tokens: nothing else runs
// meanwhile.)
__device__ __forceinline__ float silu(float z) {
    constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596303e-8f, kLn2 = 0.693147181f;
    const float n = -__builtin_amdgcn_fmed3f(z, -128.0f, 128.0f), p = n * kLog2e;
    const float rest = fmaf(n, kLog2eRest, fmaf(n, kLog2e, -p));
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(p) * fmaf(rest, kLn2, 1.0f));
}
// d silu / dz = s + z s (1 - s)
__device__ __forceinline__ float silu_grad(float z, float s) { return s * (1.0f + z * (1.0f - s)); }

// Scale of a row from the bit pattern of its largest magnitude (infinities and NaNs compare
// above every number as unsigned integers).
__device__ __forceinline__ float row_scale(uint32_t top) {
    if (top >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    const float s = float(double(__uint_as_float(top)) / 127.0);
    return s >= 1.17549435e-38f ? s : 0.0f;
}

// x / s rounded to the nearest integer, ties to even, decided on the exact quotient: the
// reciprocal gives a candidate that is off by one at most, and the remainder x - q s is exact
// in one fma (x has 24 bits, |remainder| is about s / 2 at most, and both are multiples of
// s's last place or half of it).  inv is 1 / s, or 0 for a row of scale 0 or NaN.
__device__ __forceinline__ int quantize_one(float x, float s, float inv) {
    if (inv == 0.0f) return 0;
    float q = rintf(x * inv);
    const float r = fmaf(-q, s, x), r2 = 2.0f * fabsf(r);
    if (r2 > s || (r2 == s && (int(q) & 1))) q += r > 0.0f ? 1.0f : -1.0f;
    return int(q);
}
__device__ __forceinline__ float inverse_scale(float s) { return s > 0.0f ? 1.0f / s : 0.0f; }

}  // namespace dense
}  // namespace moe
