// Device helpers of both routers: ordered keys, the scan of counts, and the grouping of few pairs.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"
#include "internal.h"

namespace moe {
namespace routing {

using dev::kWave;

constexpr int kRouteWaves = 16;              // tokens per workgroup in the large-T route kernel
constexpr int kBlock = kRouteWaves * kWave;  // 1024 threads
static_assert(kBlock == kPermChunk, "one pair per thread per permutation chunk");

// Order-preserving key of a logit: larger logit -> larger unsigned key; -0 and +0 share a key.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of cnt[0..E) by wave 0 into off[0..E]; other waves idle.
__device__ inline void wave0_scan(const int32_t* __restrict__ cnt, int E, int32_t* __restrict__ off_lds,
                           int32_t* __restrict__ off_global, int32_t* __restrict__ counts_global) {
    if (threadIdx.x >= kWave) return;
    const int lane = threadIdx.x;
    constexpr int kPer = kMaxExperts / kWave;  // 8 experts per lane
    int local[kPer];
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane * kPer + i;
        local[i] = e < E ? cnt[e] : 0;
        sum += local[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += o;
    }
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane * kPer + i;
        if (e < E) {
            off_lds[e] = run;
            if (off_global) off_global[e] = run;
            if (counts_global) counts_global[e] = local[i];
        }
        run += local[i];
    }
    if (lane == kWave - 1) {
        off_lds[E] = run;
        if (off_global) off_global[E] = run;
    }
}

// Grouping of up to 64 pairs by one workgroup, s_ids [n] in LDS (behind a barrier): counts and
// offsets by direct comparison, the rest by wave 0 with ballots.  For the pair of lane p with
// expert e: eq = lanes with expert e, lt = lanes with a smaller expert (bit-serial compare of the
// 10-bit ids, most significant bit first), so its position is |lt| + |eq below p|.
__device__ __forceinline__ void group_tiny(const int32_t* __restrict__ s_ids, int n, int E, int32_t* __restrict__ counts,
                           int32_t* __restrict__ offsets, int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
    const int tid = threadIdx.x;
    for (int e = tid; e < E; e += blockDim.x) {
        int c = 0, lt = 0;
        for (int p = 0; p < n; ++p) {
            const int v = s_ids[p];
            c += v == e;
            lt += v < e;
        }
        counts[e] = c;
        offsets[e] = lt;
    }
    if (tid == 0) offsets[E] = n;
    if (tid < kWave) {
        const bool valid = tid < n;
        const int e = valid ? s_ids[tid] : 0;
        uint64_t eq = __ballot(valid), lt = 0;
#pragma unroll
        for (int b = 9; b >= 0; --b) {
            const bool bit = (e >> b) & 1;
            const uint64_t b1 = __ballot(valid && bit);
            if (bit) {
                lt |= eq & ~b1;
                eq &= b1;
            } else {
                eq &= ~b1;
            }
        }
        const uint64_t below = tid == 0 ? 0ull : (~0ull >> (kWave - tid));
        if (valid) {
            const int pos = __popcll(lt) + __popcll(eq & below);
            perm[pos] = tid;
            inv[tid] = pos;
        }
    }
}

}  // namespace routing
}  // namespace moe
