// Router by scores, and its gradient (gfx950).
//
// Scores s_e = softmax(l)_e or 1 / (1 + e^-l_e); a bias b_e takes part in the choice and not in the
// gates: c_e = s_e + b_e.  Experts lie in groups of consecutive ids; a group counts as the sum of
// its one or two largest c_e, the best groups are kept, and of their experts the k with the
// largest c_e are chosen (without a bias: the largest logit, which is the same order, exact).
// Gates: scale * s_e, divided by the sum of the chosen scores where they are renormalised.
//
// The choice has to be that of the formula wherever it is run, so scores, biased values and group
// sums are 64-bit numbers: two experts closer than fp32's rounding of a score (2^-24) occur in every
// chunk of a few thousand tokens; closer than 2^-53 does not happen.  Equal values choose the lower
// id.  Gates are formed in 64 bits and rounded once.
//
// One wave takes one token.  Without groups lane l holds experts l + 64 i; with groups every group
// has `lanes` consecutive lanes (a power of two), each with every `lanes`-th of its experts.  A round of the
// top-k finds the largest key (order-preserving, its upper 32 bits first; the lower ones only
// where two are equal there) in a wave-wide maximum.
#include <hip/hip_runtime.h>

#include "route_common.h"

namespace moe {
namespace {

using namespace routing;

// The rule as the kernels use it: experts per group, and lanes per group.
struct Rule {
    int sigmoid, groups, size, keep, top, renorm, lanes;
    double scale;
};

Rule rule_of(const moe_route_rule& r, int E) {
    int lanes = kWave;
    while (lanes * r.n_groups > kWave) lanes /= 2;
    return Rule{r.score == MOE_SCORE_SIGMOID, r.n_groups, E / r.n_groups, r.keep_groups, r.group_top, r.renormalize,
                r.n_groups == 1 ? kWave : lanes, double(r.scale)};
}

// Order-preserving key of a 64-bit number: larger number, larger key; NaNs share the smallest one,
// (1, 0); (0, 0) is no number's.
struct Key {
    uint32_t hi, lo;
};
__device__ __forceinline__ Key key_of(double v) {
    if (v != v) return Key{1u, 0u};
    const uint64_t u = uint64_t(__double_as_longlong(v == 0.0 ? 0.0 : v));
    const uint64_t k = u >> 63 ? ~u : u | (uint64_t(1) << 63);
    return Key{uint32_t(k >> 32), uint32_t(k)};
}

__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t u = uint64_t(__double_as_longlong(v));
    const uint32_t hi = __builtin_amdgcn_readlane(int(u >> 32), lane), lo = __builtin_amdgcn_readlane(int(u), lane);
    return __longlong_as_double((long long)(uint64_t(hi) << 32 | lo));
}
__device__ __forceinline__ double sum_lanes(double v) {
#pragma unroll
    for (int d = kWave / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}
__device__ __forceinline__ double sigmoid64(double z) { return 1.0 / (1.0 + exp(-z)); }
// e^(l - m) with m the row's largest logit (-infinity: every score is 0)
__device__ __forceinline__ double share64(float l, float m) {
    return m == -INFINITY ? 0.0 : exp(double(l) - double(m));
}

template <int EPL>
__device__ __forceinline__ void scored_token(const float* __restrict__ lrow, const float* __restrict__ bias, int E, int k,
                                             const Rule& R, int32_t* __restrict__ ids_out, float* __restrict__ w_out,
                                             int32_t* __restrict__ lds_ids) {
    const int lane = dev::lane_id(), g = lane / R.lanes, r = lane % R.lanes;
    const int first = g * R.size + r;
    auto live = [&](int i) { return g < R.groups && r + R.lanes * i < R.size; };
    float l[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = live(i) ? lrow[first + R.lanes * i] : -INFINITY;
    float m = 0.0f;
    double den = 1.0;
    if (!R.sigmoid) {
        m = l[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
#pragma unroll
        for (int d = kWave / 2; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
    }
    double v[EPL];
    if (!R.sigmoid) {
        den = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            v[i] = live(i) ? share64(l[i], m) : 0.0;
            den += v[i];
        }
        den = sum_lanes(den);
        if (den == 0.0) den = 1.0;
    }
    uint32_t hi[EPL], lo[EPL];
    if (bias || R.groups > 1) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            v[i] = R.sigmoid ? sigmoid64(l[i]) : v[i] / den;
            if (bias && live(i)) v[i] += double(bias[first + R.lanes * i]);
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const Key q = bias ? key_of(v[i]) : Key{l[i] == l[i] ? order_key(l[i]) : 1u, 0u};
        hi[i] = live(i) ? q.hi : 0u;
        lo[i] = live(i) ? q.lo : 0u;
    }
    if (R.groups > 1) {
        // the two largest values of the lane, then of the group
        double a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (live(i)) {
                b = fmax(b, fmin(a, v[i]));
                a = fmax(a, v[i]);
            }
        for (int d = 1; d < R.lanes; d <<= 1) {
            const double oa = __shfl_xor(a, d, kWave), ob = __shfl_xor(b, d, kWave);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
        }
        const double mine = R.top == 2 && R.size > 1 ? a + b : a;
        int before = 0;
        for (int q = 0; q < R.groups; ++q) {
            const double other = lane_value(mine, q * R.lanes);
            before += other > mine || (other == mine && q < g) ? 1 : 0;
        }
        if (before >= R.keep) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) hi[i] = lo[i] = 0u;
        }
    }
    int my_e = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t best = hi[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) best = max(best, hi[i]);
        best = wave_umax(best);
        int n = 0;
        uint64_t at = 0;
        int slot = 0;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i) {
            const uint64_t b = __ballot(hi[i] == best);
            n += __popcll(b);
            if (b) at = b, slot = i;
        }
        if (n > 1) {                             // equal upper halves: lower halves, then the lowest id
            uint32_t low = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (hi[i] == best) low = max(low, lo[i]);
            low = wave_umax(low);
            uint32_t id = 0;                     // the largest of the complements
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (hi[i] == best && lo[i] == low && live(i)) id = max(id, ~uint32_t(first + R.lanes * i));
            id = ~wave_umax(id);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const uint64_t b = __ballot(live(i) && uint32_t(first + R.lanes * i) == id);
                if (b) at = b, slot = i;
            }
        }
        const int wl = __builtin_ctzll(at);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i == slot && lane == wl) hi[i] = lo[i] = 0u;
        if (lane == j) my_e = wl / R.lanes * R.size + wl % R.lanes + R.lanes * slot;
    }
    // gates
    const float my_l = lane < k ? lrow[my_e] : 0.0f;
    double s = lane < k ? (R.sigmoid ? sigmoid64(my_l) : share64(my_l, m) / den) : 0.0;
    if (R.renorm) {
        double total = 0.0;
        for (int j = 0; j < k; ++j) total += lane_value(s, j);
        if (total != 0.0) s /= total;
    }
    if (lane < k) {
        ids_out[lane] = my_e;
        w_out[lane] = float(s * R.scale);
        if (lds_ids) lds_ids[lane] = my_e;
    }
}

template <int EPL>
__device__ __forceinline__ void scored_tokens(const float* logits, const float* bias, int T, int E, int k, const Rule& R,
                                              int t0, int step, int32_t* ids, float* w, int32_t* lds_ids) {
    for (int t = t0 + int(threadIdx.x) / kWave; t < T; t += step)
        scored_token<EPL>(logits + int64_t(t) * E, bias, E, k, R, ids + int64_t(t) * k, w + int64_t(t) * k,
                          lds_ids ? lds_ids + int64_t(t) * k : nullptr);
}

// T*k <= 64, and <= 512: everything in one workgroup
template <int EPL>
__global__ __launch_bounds__(1024) void k_scored_tiny(const float* __restrict__ logits, const float* __restrict__ bias,
                                                      int T, int E, int k, const Rule R, int32_t* __restrict__ ids,
                                                      float* __restrict__ w, int32_t* __restrict__ counts,
                                                      int32_t* __restrict__ offsets, int32_t* __restrict__ perm,
                                                      int32_t* __restrict__ inv) {
    __shared__ int32_t s_ids[kWave];
    scored_tokens<EPL>(logits, bias, T, E, k, R, 0, blockDim.x / kWave, ids, w, s_ids);
    __syncthreads();
    group_tiny(s_ids, T * k, E, counts, offsets, perm, inv);
}
template <int EPL>
__global__ __launch_bounds__(kBlock) void k_scored_small(const float* __restrict__ logits, const float* __restrict__ bias,
                                                         int T, int E, int k, const Rule R, int32_t* __restrict__ ids,
                                                         float* __restrict__ w, int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ offsets, int32_t* __restrict__ perm,
                                                         int32_t* __restrict__ inv) {
    __shared__ int32_t s_ids[kSmallScored];
    __shared__ int32_t s_cnt[kMaxExperts];
    __shared__ int32_t s_run[kMaxExperts + 1];
    __shared__ int32_t s_wc[kRouteWaves][kMaxExperts];
    scored_tokens<EPL>(logits, bias, T, E, k, R, 0, kRouteWaves, ids, w, s_ids);
    group_small(s_ids, T * k, E, s_cnt, s_run, s_wc, counts, offsets, perm, inv);
}
template <int EPL>
__global__ __launch_bounds__(256) void k_scored(const float* __restrict__ logits, const float* __restrict__ bias, int T,
                                                int E, int k, const Rule R, int32_t* __restrict__ ids,
                                                float* __restrict__ w) {
    scored_tokens<EPL>(logits, bias, T, E, k, R, blockIdx.x * 4, T, ids, w, nullptr);
}

// Gradient of the logits from the gates', one wave a token.  With p the softmax or sigmoid score,
// S the sum of the chosen scores and a_j = p_j / S:
//   gates scale * a_j:  ds_j = scale (dw_j - sum_i dw_i a_i) / S;   gates scale * p_j:  ds_j = scale dw_j
//   sigmoid:  dl_j = ds_j p_j (1 - p_j) for the chosen, 0 for the others;
//   softmax:  dl_e = p_e (ds_e - sum_j ds_j p_j), ds_e = 0 for the others.  Renormalised, that is
//             scale a_j (dw_j - sum_i dw_i a_i) for the chosen and 0 for the others.
__global__ __launch_bounds__(256) void k_scored_backward(const float* __restrict__ logits, int T, int E, int k,
                                                         const Rule R, const int32_t* __restrict__ ids,
                                                         const float* __restrict__ dw, float* __restrict__ dlogits) {
    const int lane = dev::lane_id(), t = blockIdx.x * 4 + threadIdx.x / kWave;
    if (t >= T) return;
    const float* lrow = logits + int64_t(t) * E;
    float* drow = dlogits + int64_t(t) * E;
    int id = lane < k ? ids[int64_t(t) * k + lane] : -1;
    if (id >= E) id = -1;
    const bool mine = id >= 0;
    const double d = mine ? double(dw[int64_t(t) * k + lane]) * R.scale : 0.0;
    const float l = mine ? lrow[id] : -INFINITY;
    const bool whole = !R.sigmoid && !R.renorm;       // every logit takes part
    float m = l;
    if (whole)
        for (int e = lane; e < E; e += kWave) m = fmaxf(m, lrow[e]);
#pragma unroll
    for (int i = kWave / 2; i >= 1; i >>= 1) m = fmaxf(m, __shfl_xor(m, i, kWave));
    double den = 1.0;
    if (whole) {
        den = 0.0;
        for (int e = lane; e < E; e += kWave) den += share64(lrow[e], m);
        den = sum_lanes(den);
        if (den == 0.0) den = 1.0;
    }
    double p = mine ? (R.sigmoid ? sigmoid64(l) : share64(l, m) / den) : 0.0;
    double v, rest = 0.0;                             // rest: sum of ds_j p_j
    if (R.renorm) {
        double S = sum_lanes(p);
        if (S == 0.0) S = 1.0;
        const double a = p / S, x = d - sum_lanes(d * a);
        v = R.sigmoid ? x / S * p * sigmoid64(-double(l)) : a * x;
    } else if (R.sigmoid) {
        v = d * p * sigmoid64(-double(l));
    } else {
        rest = sum_lanes(d * p);
        v = p * (d - rest);
    }
    const float value = float(v);
    for (int e = lane; e < E; e += kWave) {
        float out = whole ? float(-share64(lrow[e], m) / den * rest) : 0.0f;
        for (int j = 0; j < k; ++j) {
            const float vj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(value), j));
            if (__builtin_amdgcn_readlane(id, j) == e) out = vj;
        }
        drow[e] = out;
    }
}

template <int EPL>
hipError_t launch_as(const moe_config& c, const Rule& R, const float* logits, const float* bias, int32_t T, int32_t* ids,
                     float* w, int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* ws, hipStream_t s) {
    const int E = c.n_experts, k = c.top_k;
    const int64_t n = int64_t(T) * k;
    if (n <= kWave) {
        const int waves = T < 1 ? 1 : T > 16 ? 16 : int(T);
        hipLaunchKernelGGL((k_scored_tiny<EPL>), dim3(1), dim3(waves * kWave), 0, s, logits, bias, T, E, k, R, ids, w,
                           counts, offsets, perm, inv);
        return hipGetLastError();
    }
    if (n <= kSmallScored) {
        hipLaunchKernelGGL((k_scored_small<EPL>), dim3(1), dim3(kBlock), 0, s, logits, bias, T, E, k, R, ids, w, counts,
                           offsets, perm, inv);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((k_scored<EPL>), dim3((T + 3) / 4), dim3(256), 0, s, logits, bias, T, E, k, R, ids, w);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? launch_permute(c, T, ids, counts, offsets, perm, inv, ws, s) : e;
}

}  // namespace

hipError_t launch_route_scored(const moe_config& c, const moe_route_rule& r, const float* logits, const float* bias,
                               int32_t T, int32_t* ids, float* w, int32_t* counts, int32_t* offsets, int32_t* perm,
                               int32_t* inv, void* ws, hipStream_t s) {
    const Rule R = rule_of(r, c.n_experts);
    const int per = (R.size + R.lanes - 1) / R.lanes;        // (16 at most: 512 experts, lanes > 32 / groups)
#define MOE_SCORED(N) return launch_as<N>(c, R, logits, bias, T, ids, w, counts, offsets, perm, inv, ws, s)
    if (per <= 1) MOE_SCORED(1);
    if (per <= 2) MOE_SCORED(2);
    if (per <= 4) MOE_SCORED(4);
    if (per <= 8) MOE_SCORED(8);
    if (per <= 16) MOE_SCORED(16);
#undef MOE_SCORED
    return hipErrorInvalidValue;
}

hipError_t launch_route_scored_backward(const moe_config& c, const moe_route_rule& r, const float* logits, int32_t T,
                                        const int32_t* ids, const float* dw, float* dlogits, hipStream_t s) {
    if (T == 0) return hipSuccess;
    hipLaunchKernelGGL(k_scored_backward, dim3((T + 3) / 4), dim3(256), 0, s, logits, T, c.n_experts, c.top_k,
                       rule_of(r, c.n_experts), ids, dw, dlogits);
    return hipGetLastError();
}

}  // namespace moe
