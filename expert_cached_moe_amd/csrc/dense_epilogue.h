// The last steps of a product on W (4 or 8) sums of consecutive columns of one row, shared by the
// product kernels.  For the gated epilogues those are W gate sums, and W up sums 16 columns on.
#pragma once

#include <type_traits>

#include "dense_common.h"

namespace moe {
namespace dense {

typedef __attribute__((ext_vector_type(4))) int i32x4;

// Four 32-bit words that lie on a 4-byte boundary: enough for a 16-byte store to memory.
typedef uint32_t __attribute__((ext_vector_type(4), aligned(4))) words4;
typedef uint32_t __attribute__((ext_vector_type(2), aligned(4))) words2;

// W values to p[0 .. W-1], 4 (fp32) or W (bf16, on a 4-byte boundary) at a time.  STREAM: past the caches, for results
// that leave as whole lines and are not read by the next kernel.
template <int W, bool STREAM = false>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[W]) {
    if constexpr (W == 8) {
        const dev::u32x4 u{dev::pack_bf16x2(v[0], v[1]), dev::pack_bf16x2(v[2], v[3]), dev::pack_bf16x2(v[4], v[5]),
                           dev::pack_bf16x2(v[6], v[7])};
        if (STREAM) __builtin_nontemporal_store(words4(u), reinterpret_cast<words4*>(p));
        else *reinterpret_cast<words4*>(p) = u;
    } else
        *reinterpret_cast<words2*>(p) = words2{dev::pack_bf16x2(v[0], v[1]), dev::pack_bf16x2(v[2], v[3])};
}
template <int W, bool STREAM = false>
__device__ __forceinline__ void store_row(float* p, const float (&v)[W]) {
#pragma unroll
    for (int q = 0; q < W; q += 4) {
        const words4 u = __builtin_bit_cast(dev::u32x4, dev::f32x4{v[q], v[q + 1], v[q + 2], v[q + 3]});
        if (STREAM) __builtin_nontemporal_store(u, reinterpret_cast<words4*>(p + q));
        else *reinterpret_cast<words4*>(p + q) = u;
    }
}
template <int W>
__device__ __forceinline__ void load_row(float (&v)[W], const uint16_t* p) {
    uint32_t u[W / 2];
    if constexpr (W == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        u[0] = q.x, u[1] = q.y, u[2] = q.z, u[3] = q.w;
    } else {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        u[0] = q.x, u[1] = q.y;
    }
#pragma unroll
    for (int j = 0; j < W / 2; ++j) v[2 * j] = dev::bf16_lo(u[j]), v[2 * j + 1] = dev::bf16_hi(u[j]);
}
template <int W>
__device__ __forceinline__ void load_row(float (&v)[W], const float* p) {
#pragma unroll
    for (int q = 0; q < W; q += 4) {
        const float4 u = *reinterpret_cast<const float4*>(p + q);
        v[q] = u.x, v[q + 1] = u.y, v[q + 2] = u.z, v[q + 3] = u.w;
    }
}

// Pre-activations kept for the backward pass.  fp32: as they are.  bf16 contexts: the upper 24
// bits of the fp32 sums (a sign, 8 exponent bits, 15 fraction bits), 16 in one array and 8 in another
// of the same shape.  They are cut there, not rounded: by less than 2^-15 of the value, 1/128 of the
// rounding of dg and du that follows.
// Rounded to bf16 they would be a third rounding of that size in the gradients, after those of
// dg, du and of the result (relative error of dWg and dx 0.0030 against 0.0023); all 32 bits
// would cost another third of the bytes.
template <int W>
__device__ __forceinline__ void keep_row(float* p, uint8_t*, int64_t i, const float (&v)[W]) {
    store_row<W>(p + i, v);
}
template <int W>
__device__ __forceinline__ void keep_row(uint16_t* hi, uint8_t* lo, int64_t i, const float (&v)[W]) {
    uint32_t h[W / 2], l[W / 4];
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
        const uint32_t a = __float_as_uint(v[2 * j]), b = __float_as_uint(v[2 * j + 1]);
        h[j] = __builtin_amdgcn_perm(b, a, 0x07060302);              // upper halves
        const uint32_t two = __builtin_amdgcn_perm(b, a, 0x0C0C0501);  // their next bytes
        l[j / 2] = j % 2 ? l[j / 2] | two << 16 : two;
    }
    if constexpr (W == 8) {
        *reinterpret_cast<uint4*>(hi + i) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint2*>(lo + i) = make_uint2(l[0], l[1]);
    } else {
        *reinterpret_cast<uint2*>(hi + i) = make_uint2(h[0], h[1]);
        *reinterpret_cast<uint32_t*>(lo + i) = l[0];
    }
}
template <int W>
__device__ __forceinline__ void kept_row(float (&v)[W], const float* p, const uint8_t*, int64_t i) {
    load_row<W>(v, p + i);
}
template <int W>
__device__ __forceinline__ void kept_row(float (&v)[W], const uint16_t* hi, const uint8_t* lo, int64_t i) {
    uint32_t h[W / 2], l[W / 4];
    if constexpr (W == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(hi + i);
        const uint2 r = *reinterpret_cast<const uint2*>(lo + i);
        h[0] = q.x, h[1] = q.y, h[2] = q.z, h[3] = q.w, l[0] = r.x, l[1] = r.y;
    } else {
        const uint2 q = *reinterpret_cast<const uint2*>(hi + i);
        h[0] = q.x, h[1] = q.y, l[0] = *reinterpret_cast<const uint32_t*>(lo + i);
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const uint32_t up = j % 2 ? h[j / 2] & 0xFFFF0000u : h[j / 2] << 16;
        v[j] = __uint_as_float(up | (l[j / 4] >> (8 * (j % 4)) & 255u) << 8);
    }
}

// The sigmoid of the block's kernels.  fp32: expf and a division.  bf16: hardware exp2 and
// reciprocal (about one fp32 step each, and the argument's rounding times its size; the results are
// rounded to bf16, 2^16 times coarser).  Either way the result is 0 from about z = -88 down, where
// e^-z overflows to infinity.
template <int TYPE>
__device__ __forceinline__ float sigmoid_of(float z) {
    if constexpr (TYPE == kF32) return sigmoid(z);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// Epilogues of integer products, and those whose results are one scaled number a column.
template <int EPI>
constexpr bool kScaled = EPI == kScale || EPI == kScale32 || EPI == kGate8;
template <int EPI>
constexpr bool kPlainScale = EPI == kScale || EPI == kScale32;

// Scales of the columns a lane finishes (and of the up columns): loaded once, used for every row.
template <int EPI, int W>
struct ColumnScales {
    float s[kScaled<EPI> ? W : 1], up[EPI == kGate8 ? W : 1];
    __device__ __forceinline__ void load(const Product& p, int n) {
        if constexpr (kScaled<EPI>) {
#pragma unroll
            for (int j = 0; j < W; ++j) s[j] = p.col_scale[n + j < p.N ? n + j : p.N - 1];
        }
        if constexpr (EPI == kGate8) {
#pragma unroll
            for (int j = 0; j < W; ++j) up[j] = p.col_scale[n + 16 + j < p.N ? n + 16 + j : p.N - 1];
        }
    }
};

// What finishing row m, columns n .. n + W - 1 reads: its row scale, or its gate and up values.
// Loaded apart from the finishing, so that a kernel can have the next row's loads ahead of this
// row's stores (a wait for a load waits for every older store).
template <int TYPE, int EPI, int W>
struct RowInputs {
    // first * last is the row's scale.  One above 2^60 is applied last: times a sum (below 2^31) it
    // could overflow although the column's scale brings the result back into range.
    float first, last, g[EPI == kDGate ? W : 1], u[EPI == kDGate ? W : 1];
    __device__ __forceinline__ void set_scale(float s) {
        const bool big = s > 1.1529215e18f;
        first = big ? 1.0f : s;
        last = big ? s : 1.0f;
    }
    __device__ __forceinline__ void load(const Product& p, int64_t m, int n) {
        if constexpr (kScaled<EPI>) set_scale(p.row_scale[m]);
        if constexpr (EPI == kDGate) {
            typedef typename Elem<TYPE>::T E;
            const int64_t i = m * 2 * p.N + n / 16 * 32 + n % 16;
            kept_row<W>(g, static_cast<const E*>(p.gu), p.gu_low, i);
            kept_row<W>(u, static_cast<const E*>(p.gu), p.gu_low, i + 16);
        }
    }
};

// Row m, columns n .. n + W - 1 (v; the up sums in u).  n < N; only kScale, kScale32 may reach
// past N.  STREAM: results past the caches.
template <int TYPE, int EPI, int W, bool STREAM, class S>
__device__ __forceinline__ void finish(const Product& p, int64_t m, int n, const S (&v)[W], const S (&u)[W],
                                       const ColumnScales<EPI, W>& cs, const RowInputs<TYPE, EPI, W>& in) {
    typedef typename Elem<TYPE>::T E;
    if constexpr (EPI == kStore) {
        float f[W];
#pragma unroll
        for (int j = 0; j < W; ++j) f[j] = float(v[j]);
        store_row<W>(static_cast<E*>(p.out) + m * p.ldo + n, f);
    } else if constexpr (kPlainScale<EPI>) {
        typedef typename std::conditional<EPI == kScale32, float, uint16_t>::type O;
        float f[W];
#pragma unroll
        for (int j = 0; j < W; ++j) f[j] = float(v[j]) * in.first * cs.s[j] * in.last;
        O* o = static_cast<O*>(p.out) + m * p.ldo + n;
        if (p.vec_out && n + W <= p.N) {
            store_row<W, STREAM>(o, f);
            return;
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
            if (n + j < p.N) put(o + j, f[j]);
    } else if constexpr (EPI == kGate) {
        // n is the gate column (n % 32 < 16) of inner index n / 32 * 16 + n % 16
        float h[W];
#pragma unroll
        for (int j = 0; j < W; ++j) h[j] = v[j] * sigmoid_of<TYPE>(v[j]) * u[j];
        if (p.gu) {
            keep_row<W>(static_cast<E*>(p.gu), p.gu_low, m * p.N + n, v);
            keep_row<W>(static_cast<E*>(p.gu), p.gu_low, m * p.N + n + 16, u);
        }
        store_row<W>(static_cast<E*>(p.out) + m * p.ldo + n / 32 * 16 + n % 16, h);
    } else if constexpr (EPI == kGate8) {
        // the same from integer sums, in fp32 throughout (h's codes are decided on it)
        float h[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float g = float(v[j]) * in.first * cs.s[j] * in.last, up = float(u[j]) * in.first * cs.up[j] * in.last;
            h[j] = silu(g) * up;
        }
        store_row<W, STREAM>(static_cast<float*>(p.out) + m * p.ldo + n / 32 * 16 + n % 16, h);
    } else {
        // v = dh, n an inner index
        const int64_t o = m * 2 * p.N + n / 16 * 32 + n % 16;
        float dg[W], du[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float s = sigmoid_of<TYPE>(in.g[j]);
            // (v last: a shut gate's factor is 0, and v g or v u may leave fp32)
            dg[j] = v[j] * (in.u[j] * silu_grad(in.g[j], s));
            du[j] = v[j] * (in.g[j] * s);
        }
        store_row<W>(static_cast<E*>(p.out) + o, dg);
        store_row<W>(static_cast<E*>(p.out) + o + 16, du);
    }
}

// Columns of one row that take part in W results: the gated epilogues pair two runs of 16.
template <int EPI>
constexpr bool kPaired = paired(EPI);

}  // namespace dense
}  // namespace moe
