// Device helpers of the routing kernels: ordered keys and their wave-wide maximum, and the stable
// counting sort of pairs by expert.
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
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Wave-wide maximum of an unsigned key, left in every lane: butterflies inside each row of
// 16 lanes (DPP quad swaps, rotations by 4 and 8), then row pairs and wave halves exchanged
// with permlane16_swap / permlane32_swap.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t a) {
    return max(a, uint32_t(__builtin_amdgcn_mov_dpp(int(a), CTRL, 0xF, 0xF, false)));
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t a) {
    a = dpp_umax<0xB1>(a);   // quad_perm [1,0,3,2]
    a = dpp_umax<0x4E>(a);   // quad_perm [2,3,0,1]
    a = dpp_umax<0x124>(a);  // row_ror:4
    a = dpp_umax<0x128>(a);  // row_ror:8
    const auto h16 = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    a = max(h16[0], h16[1]);
    const auto h32 = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    return max(h32[0], h32[1]);
}

// Lanes of the wave holding the same expert id (10-bit ids), among lanes with valid = 1.
__device__ __forceinline__ uint64_t match_expert(int e, bool valid) {
    uint64_t m = __ballot(valid);
#pragma unroll
    for (int b = 0; b < 10; ++b) {
        const bool bit = valid && ((e >> b) & 1);
        const uint64_t bb = __ballot(bit);
        m &= bit ? bb : ~bb;
    }
    return valid ? m : 0;
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

// Stable scatter of one chunk of up to 1024 pairs: pair p = p0 + tid with expert
// e = ids[tid].  run[e] is the output position of the chunk's first pair of expert
// e; it is advanced by the chunk's count.  wc: [16][E] per-wave counts (LDS).
__device__ inline void scatter_chunk(const int32_t* __restrict__ ids_src, int p0, int n_valid, int E,
                              int32_t* __restrict__ run, int32_t (*wc)[kMaxExperts],
                              int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const bool valid = tid < n_valid;
    const int e = valid ? ids_src[tid] : 0;
    const uint64_t m = match_expert(e, valid);
    const uint64_t lt = (lane == 0) ? 0ull : (~0ull >> (kWave - lane));
    const int rank = __popcll(m & lt);
    const int cw = __popcll(m);
    for (int i = tid; i < kRouteWaves * E; i += kBlock) wc[i / E][i % E] = 0;
    __syncthreads();
    if (valid && rank == 0) wc[wave][e] = cw;
    __syncthreads();
    if (valid) {
        int pos = run[e] + rank;
        for (int w2 = 0; w2 < wave; ++w2) pos += wc[w2][e];
        perm[pos] = p0 + tid;
        inv[p0 + tid] = pos;
    }
    __syncthreads();
    for (int ee = tid; ee < E; ee += kBlock) {
        int s = 0;
#pragma unroll
        for (int w2 = 0; w2 < kRouteWaves; ++w2) s += wc[w2][ee];
        run[ee] += s;
    }
    __syncthreads();
}

// Grouping of up to 4096 pairs by one workgroup: s_ids [n] in LDS (written by every thread that
// takes part; the call begins with a count and ends with every output stored).
__device__ inline void group_small(const int32_t* __restrict__ s_ids, int n, int E, int32_t* __restrict__ s_cnt,
                            int32_t* __restrict__ s_run, int32_t (*s_wc)[kMaxExperts], int32_t* __restrict__ counts,
                            int32_t* __restrict__ offsets, int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
    const int tid = threadIdx.x;
    for (int e = tid; e < E; e += kBlock) s_cnt[e] = 0;
    __syncthreads();
    for (int p = tid; p < n; p += kBlock) atomicAdd(&s_cnt[s_ids[p]], 1);
    __syncthreads();
    wave0_scan(s_cnt, E, s_run, offsets, counts);
    __syncthreads();
    for (int p0 = 0; p0 < n; p0 += kBlock) scatter_chunk(s_ids + p0, p0, n - p0, E, s_run, s_wc, perm, inv);
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
