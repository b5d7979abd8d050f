// Device helpers of the products with 4-bit weights.
#pragma once

#include "device_common.h"
#include "i4.h"

namespace moe {
namespace i4 {

typedef __attribute__((ext_vector_type(2))) float f32x2;

// The list of experts that a kernel takes (its 2 KB are copied at each launch): dense kernels have none.
struct NoList {};
template <int KIND>
struct ListType {
    using Type = NoList;
};
template <>
struct ListType<kGateUp> {
    using Type = ExpertList;
};
template <>
struct ListType<kDown> {
    using Type = ExpertList;
};
template <int KIND>
using ListOf = typename ListType<KIND>::Type;
template <int KIND>
const ListOf<KIND>& list_of(const ExpertList* list) {
    static const NoList none{};
    if constexpr (KIND == kGateUp || KIND == kDown)
        return *list;
    else
        return none;
}

// A group's word: s, and its zero point.  (Bytes as e4m3 numbers: 0..15 are 2^-9 times themselves,
// the subnormal numbers and the first binade, so the conversion instructions turn codes into numbers.)
__device__ __forceinline__ float word_scale(uint32_t w) { return __builtin_amdgcn_cvt_f32_fp8(int(w), 0); }
__device__ __forceinline__ float word_zero(uint32_t w) { return float((w >> 8) & 255u); }

// 2^(e - 127); 255 is NaN
__device__ __forceinline__ float row_scale(uint32_t e) {
    return __uint_as_float(e == 255u ? 0x7FC00000u : e == 0u ? 0x00400000u : e << 23);
}

// The 8 weights of 8 codes as bf16, in order: 512 s2 (code / 512) + off with s2 = 512 s S, off = -z s S.
__device__ __forceinline__ dev::u32x4 decode8(uint32_t codes, float s2, float off) {
    const uint32_t e = codes & 0x0F0F0F0Fu, o = codes >> 4 & 0x0F0F0F0Fu;
    const f32x2 e0 = __builtin_amdgcn_cvt_pk_f32_fp8(int(e), false), e1 = __builtin_amdgcn_cvt_pk_f32_fp8(int(e), true);
    const f32x2 o0 = __builtin_amdgcn_cvt_pk_f32_fp8(int(o), false), o1 = __builtin_amdgcn_cvt_pk_f32_fp8(int(o), true);
    return dev::u32x4{dev::pack_bf16x2(fmaf(e0[0], s2, off), fmaf(o0[0], s2, off)),
                      dev::pack_bf16x2(fmaf(e0[1], s2, off), fmaf(o0[1], s2, off)),
                      dev::pack_bf16x2(fmaf(e1[0], s2, off), fmaf(o1[0], s2, off)),
                      dev::pack_bf16x2(fmaf(e1[1], s2, off), fmaf(o1[1], s2, off))};
}

// silu(g) u in fp32 from the hardware's exp2 and reciprocal (a step each, and the argument's rounding
// times its size; the result is rounded to bf16, 2^16 times coarser); 0 from about g = -88 down
__device__ __forceinline__ float gated(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g)) * u;
}

// The entry of a list: bytes from slot 0 to its blob, whether it is the shared expert.
__device__ __forceinline__ int64_t blob_offset(const Product& p, int ent) {
    return (ent & 1023) == kSharedTag ? p.shared : int64_t(ent >> 10) * p.stride;
}
__device__ __forceinline__ Rows rows_at(const Rows& w, int64_t bytes) {
    Rows r = w;
    r.codes += bytes;
    r.words = reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(w.words) + bytes);
    r.exps += bytes;
    return r;
}

// Row of x and row of out of place base + r of an entry (the shared expert's places begin at T top_k).
template <int KIND>
__device__ __forceinline__ int64_t row_in(const Product& p, bool shared, int base, int r) {
    if (KIND == kGateUp) return shared ? base + r - int64_t(p.T) * p.top_k : p.perm[base + r] / p.top_k;
    if (KIND == kDown) return int64_t(base) + r;
    return r;
}
template <int KIND>
__device__ __forceinline__ int64_t row_out(const Product& p, bool shared, int base, int r) {
    if (KIND == kDown && !shared) return p.perm[base + r];
    if (KIND == kGateUp || KIND == kDown) return int64_t(base) + r;
    return r;
}

}  // namespace i4
}  // namespace moe
