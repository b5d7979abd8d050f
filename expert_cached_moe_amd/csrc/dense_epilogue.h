// The last steps of a product on four sums of consecutive columns of one row, shared by the
// matrix-core kernels.  (kGate, kGate8: four gate sums and the four up sums 16 columns on.)
#pragma once

#include "dense_common.h"

namespace moe {
namespace dense {

typedef __attribute__((ext_vector_type(4))) int i32x4;

// 4 values to p[0..3] in bf16 or fp32; VEC: p is 8 (16) bytes aligned
__device__ __forceinline__ void store4(uint16_t* p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(p) = make_uint2(dev::pack_bf16x2(a, b), dev::pack_bf16x2(c, d));
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

__device__ __forceinline__ void load4(float (&v)[4], const uint16_t* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = dev::bf16_lo(u.x), v[1] = dev::bf16_hi(u.x), v[2] = dev::bf16_lo(u.y), v[3] = dev::bf16_hi(u.y);
}
__device__ __forceinline__ void load4(float (&v)[4], const float* p) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
}

// The sigmoid of the block's kernels.  fp32: expf and a division.  bf16: hardware exp2 and
// reciprocal (about one fp32 step each; the results are rounded to bf16, 2^16 times coarser).
// Either way e^-z overflows to infinity for very negative z, whose reciprocal is 0.
template <int TYPE>
__device__ __forceinline__ float sigmoid_of(float z) {
    if constexpr (TYPE == kF32) return sigmoid(z);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// kStore: out[m][n .. n + 3]
template <int TYPE>
__device__ __forceinline__ void finish_store(const Product& p, int64_t m, int n, const dev::f32x4& v) {
    store4(static_cast<typename Elem<TYPE>::T*>(p.out) + m * p.ldo + n, v[0], v[1], v[2], v[3]);
}

// kScale: out[m][n .. n + 3] = sums * row scale * column scales; any N, any alignment
__device__ __forceinline__ void finish_scale(const Product& p, int64_t m, int n, const i32x4& v) {
    const float rs = p.row_scale[m];
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = float(v[j]) * rs * p.col_scale[n + j < p.N ? n + j : p.N - 1];
    const int64_t o = m * p.ldo + n;
    if (p.vec_out && n + 4 <= p.N) {
        if (p.out_f32) store4(static_cast<float*>(p.out) + o, f[0], f[1], f[2], f[3]);
        else store4(static_cast<uint16_t*>(p.out) + o, f[0], f[1], f[2], f[3]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (n + j < p.N) {
            if (p.out_f32) put(static_cast<float*>(p.out) + o + j, f[j]);
            else put(static_cast<uint16_t*>(p.out) + o + j, f[j]);
        }
}

// kGate: n is the gate column (n % 32 < 16), inner index n / 32 * 16 + n % 16
template <int TYPE>
__device__ __forceinline__ void finish_gate(const Product& p, int64_t m, int n, const dev::f32x4& g, const dev::f32x4& u) {
    typedef typename Elem<TYPE>::T E;
    if (p.gu) {
        E* s = static_cast<E*>(p.gu) + m * p.N + n;
        store4(s, g[0], g[1], g[2], g[3]);
        store4(s + 16, u[0], u[1], u[2], u[3]);
    }
    float h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = g[j] * sigmoid_of<TYPE>(g[j]) * u[j];
    store4(static_cast<E*>(p.out) + m * p.ldo + n / 32 * 16 + n % 16, h[0], h[1], h[2], h[3]);
}

// kGate8: the same from integer sums, in fp32 with the full-precision silu (h's codes are
// decided on it)
__device__ __forceinline__ void finish_gate8(const Product& p, int64_t m, int n, const i32x4& g, const i32x4& u) {
    const float rs = p.row_scale[m];
    const float4 gs = *reinterpret_cast<const float4*>(p.col_scale + n);
    const float4 us = *reinterpret_cast<const float4*>(p.col_scale + n + 16);
    const float gw[4] = {gs.x, gs.y, gs.z, gs.w}, uw[4] = {us.x, us.y, us.z, us.w};
    float h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = silu(float(g[j]) * rs * gw[j]) * (float(u[j]) * rs * uw[j]);
    store4(static_cast<float*>(p.out) + m * p.ldo + n / 32 * 16 + n % 16, h[0], h[1], h[2], h[3]);
}

// kDGate: v = dh[m][n .. n + 3], n an inner index
template <int TYPE>
__device__ __forceinline__ void finish_dgate(const Product& p, int64_t m, int n, const dev::f32x4& v) {
    typedef typename Elem<TYPE>::T E;
    const int64_t o = m * 2 * p.N + n / 16 * 32 + n % 16;
    float g[4], u[4], dg[4], du[4];
    load4(g, static_cast<const E*>(p.gu) + o);
    load4(u, static_cast<const E*>(p.gu) + o + 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float s = sigmoid_of<TYPE>(g[j]);
        dg[j] = v[j] * u[j] * silu_grad(g[j], s);
        du[j] = v[j] * g[j] * s;
    }
    E* d = static_cast<E*>(p.out) + o;
    store4(d, dg[0], dg[1], dg[2], dg[3]);
    store4(d + 16, du[0], du[1], du[2], du[3]);
}

}  // namespace dense
}  // namespace moe
