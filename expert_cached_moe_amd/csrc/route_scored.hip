// Router by scores, and its gradient (gfx950).
//
// Scores s_e = softmax(l)_e or 1 / (1 + e^-l_e); a bias b_e takes part in the choice and not in the
// gates: c_e = s_e + b_e.  Experts lie in groups of consecutive ids; a group counts as the sum of
// its one or two largest c_e, the best groups are kept, and of their experts the k with the
// largest c_e are chosen (without a bias: the largest logit, which is the same order, exact).
// Gates: scale * s_e, divided by the sum of the chosen scores where they are renormalised (softmax: that over the
// chosen logits).
//
// The choice has to be that of the formula wherever it is run, so scores, biased values and group
// sums are 64-bit numbers: two experts closer than fp32's rounding of a score (2^-24) occur in every
// chunk of a few thousand tokens, closer than 2^-51 only where scores are next to 1: sigmoids of 30 and more, which from
// 53 ln 2 = 36.74 up are 1.  Equal values choose the lower id; which of two unequal ones closer than 2^-51 (1 + e^-z and its
// reciprocal each 2^-53 off) comes first is left open.  Gates are formed in 64 bits and rounded once.
//
// W lanes take one token, 16 or, where few tokens are to be had, a wave; a lane holds consecutive
// experts, and with groups a group has a power of two of lanes to itself.  64-bit work is the same
// for both, a round of the top-k costs a wave the same for one token and for four: maxima of
// 32-bit keys in each lane and across the W, then the one key cleared.  The keys are the
// values rounded to fp32, in order; where two of the k + 1 largest are equal there the wave makes
// its choice again on the 64-bit values.
//
// More than 16 tokens or 64 pairs: workgroups of 4 tokens and more, 256 at most, count their pairs by expert, and the
// second kernel's workgroups, one for each, add up the counts for themselves: E x 256 bytes from L2
// in place of two further launches.  8,192 tokens, 256 experts in 8 groups, top 8: 14 us and 5 (a wave a
// token, sorted by three kernels: 20, and 11 for these); 515 tokens 7.5 and 5.  The bytes take 2 us: what bounds the
// first kernel is the length of a wave's program, read once (a token's 64-bit sigmoids, 8 rounds), and of the second a
// chain of reads of what other dies' workgroups wrote, sums and barriers.
#include <hip/hip_runtime.h>

#include "route_common.h"

namespace moe {
namespace {

using namespace routing;

// The rule as the kernels use it: experts of a group, lanes of a group of the W that take a token, experts of a lane, and
// whether these can be read four at a time.
struct Rule {
    int sigmoid, groups, size, keep, top, renorm, lanes, per, fours;
    double scale;
};

Rule rule_of(const moe_route_rule& r, int E, int W, const void* logits, const void* bias) {
    int lanes = W;
    while (lanes > 1 && lanes * r.n_groups > W) lanes /= 2;
    const int size = E / r.n_groups, per = (size + lanes - 1) / lanes;
    const bool fours = size % 4 == 0 && per > 2 && (uintptr_t(logits) | uintptr_t(bias)) % 16 == 0;
    return Rule{r.score == MOE_SCORE_SIGMOID, r.n_groups, size, r.keep_groups, r.group_top, r.renormalize, lanes,
                fours ? (per + 3) / 4 * 4 : per, fours, double(r.scale)};
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

// f over W consecutive lanes, left in each: mirrors of 8 and 16 lanes stand for the other four and eight, which hold one
// value by then.  Every lane combines the same pairs.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
    return uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __uint_as_float(moved<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
    const uint64_t u = uint64_t(__double_as_longlong(v));
    return __longlong_as_double((long long)(uint64_t(moved<CTRL>(uint32_t(u >> 32))) << 32 | moved<CTRL>(uint32_t(u))));
}
template <int D>                                     // lanes in pairs of rows of 16, or halves of the wave: the two values
__device__ __forceinline__ void both(uint32_t v, uint32_t& a, uint32_t& b) {
    const auto h = D == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false) : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = h[0], b = h[1];
}
template <int D>
__device__ __forceinline__ void both(float v, float& a, float& b) {
    uint32_t x, y;
    both<D>(__float_as_uint(v), x, y);
    a = __uint_as_float(x), b = __uint_as_float(y);
}
template <int D>
__device__ __forceinline__ void both(double v, double& a, double& b) {
    const uint64_t u = uint64_t(__double_as_longlong(v));
    uint32_t ah, bh, al, bl;
    both<D>(uint32_t(u >> 32), ah, bh);
    both<D>(uint32_t(u), al, bl);
    a = __longlong_as_double((long long)(uint64_t(ah) << 32 | al)), b = __longlong_as_double((long long)(uint64_t(bh) << 32 | bl));
}
template <int W, class V, class F>
__device__ __forceinline__ V across(V v, F f) {
    v = f(v, moved<0xB1>(v));                        // quad_perm [1,0,3,2]
    v = f(v, moved<0x4E>(v));                        // quad_perm [2,3,0,1]
    v = f(v, moved<0x141>(v));                       // row_half_mirror
    v = f(v, moved<0x140>(v));                       // row_mirror
    if constexpr (W >= 32) {
        V a, b;
        both<16>(v, a, b);
        v = f(a, b);
    }
    if constexpr (W == kWave) {
        V a, b;
        both<32>(v, a, b);
        v = f(a, b);
    }
    return v;
}
struct Add {
    __device__ double operator()(double a, double b) const { return a + b; }
};
struct Max {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};
__device__ __forceinline__ double sum_lanes(double v) { return across<kWave>(v, Add{}); }

// The two largest values of a group's lanes, from each lane's.
template <int CTRL>
__device__ __forceinline__ void merge_two(double& a, double& b) {
    const double oa = moved<CTRL>(a), ob = moved<CTRL>(b);
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
}
template <int D>
__device__ __forceinline__ void merge_rows(double& a, double& b) {
    double a0, a1, b0, b1;
    both<D>(a, a0, a1);
    both<D>(b, b0, b1);
    b = fmax(fmin(a0, a1), fmax(b0, b1));
    a = fmax(a0, a1);
}

// 1 / d for d in [1, 2^1000]: the estimate and two steps of Newton's iteration
__device__ __forceinline__ double reciprocal(double d) {
    double y = __builtin_amdgcn_rcp(d);
    y = fma(fma(-d, y, 1.0), y, y);
    return fma(fma(-d, y, 1.0), y, y);
}
// 1 / (1 + e^-z), from e^-|z|, at most 1
__device__ __forceinline__ double sigmoid64(double z) {
    const double e = exp(-fabs(z));
    return (z < 0.0 ? e : 1.0) * reciprocal(1.0 + e);
}
// e^(l - m) with m the row's largest logit (-infinity: every score is 0)
__device__ __forceinline__ double share64(float l, float m) { return exp(double(l) - (m == -INFINITY ? 0.0 : double(m))); }

// Token t of the W lanes (those with act; the others go along), logits lrow.  Returns the lane's expert: lane j < k of
// the W the j-th.
template <int W, int EPL>
__device__ __forceinline__ int scored_token(const float* __restrict__ lrow, const float* __restrict__ bias, bool act, int k,
                                            const Rule& R, int32_t* __restrict__ ids_out, float* __restrict__ w_out,
                                            volatile int32_t* picks) {
    const int lane = dev::lane_id(), l = lane % W, seg = lane - l;
    const int g = l / R.lanes, r = l % R.lanes;
    const int begin = r * R.per, first = g * R.size + begin;
    const int n = act && g < R.groups ? min(R.size - begin, R.per) : 0;
    auto live = [&](int i) { return i < n; };
    float x[EPL], b[EPL];
    auto read = [&](const float* row, float (&v)[EPL], float none) {
        if (EPL % 4 == 0 && R.fours) {
#pragma unroll
            for (int i = 0; i < EPL / 4; ++i) {
                const bool in = 4 * i < n;
                const float4 f = *reinterpret_cast<const float4*>(row + (in ? first + 4 * i : 0));
                v[4 * i] = in ? f.x : none, v[4 * i + 1] = in ? f.y : none;
                v[4 * i + 2] = in ? f.z : none, v[4 * i + 3] = in ? f.w : none;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float f = row[live(i) ? first + i : 0];
                v[i] = live(i) ? f : none;
            }
        }
    };
    read(lrow, x, -INFINITY);
    if (bias) read(bias, b, 0.0f);
    float m = 0.0f;
    double den = 1.0, v[EPL];
    if (!R.sigmoid) {
        m = x[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = fmaxf(m, x[i]);
        m = across<W>(m, Max{});
        den = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            v[i] = share64(x[i], m);                          // (0 where there is no expert)
            den += v[i];
        }
        den = across<W>(den, Add{});
        if (den == 0.0) den = 1.0;
    }
    uint32_t key[EPL];
    if (bias || R.groups > 1) {
        if (R.sigmoid) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) v[i] = sigmoid64(x[i]);
        } else {
            const double inv = reciprocal(den);
#pragma unroll
            for (int i = 0; i < EPL; ++i) v[i] *= inv;
        }
        if (bias) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) v[i] += double(b[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const float c = bias ? float(v[i]) : x[i];
        key[i] = live(i) ? (c == c ? order_key(c) : 1u) : 0u;
    }
    bool in = true;
    if (R.groups > 1) {
        double a = -INFINITY, b2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const double c = live(i) ? v[i] : -INFINITY;
            b2 = fmax(b2, fmin(a, c));
            a = fmax(a, c);
        }
        if (R.lanes > 1) merge_two<0xB1>(a, b2);
        if (R.lanes > 2) merge_two<0x4E>(a, b2);
        if (R.lanes > 4) merge_two<0x141>(a, b2);
        if (R.lanes > 8) merge_two<0x140>(a, b2);
        if constexpr (W == kWave)
            if (R.lanes > 16) merge_rows<16>(a, b2);          // (two groups: 32 lanes at most)
        const double mine = R.top == 2 && R.size > 1 ? a + b2 : a;
        int before = 0;
#pragma unroll 8
        for (int q = 0; q < R.groups; ++q) {
            const double other = __shfl(mine, seg + q * R.lanes, kWave);
            before += other > mine || (other == mine && q < g) ? 1 : 0;
        }
        in = before < R.keep;
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = in ? key[i] : 0u;
    }
    auto best_key = [&] {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
        return best;
    };
    // the lowest lane of the W with the flag (one has it)
    auto lowest = [&](bool flag) {
        const uint64_t mask = __ballot(flag);
        return W == kWave ? int(__builtin_ctzll(mask)) : int(__builtin_ctz(uint32_t(mask >> seg)));
    };
    // (the j-th pick of the W's token: its lane leaves it in LDS; nothing waits for it before the last)
    uint32_t last = 0;
    bool tie = false;
    for (int j = 0; j < k; ++j) {
        const uint32_t own = best_key(), best = across<W>(own, Max{});
        tie |= best == last;
        last = best;
        const int wl = lowest(own == best);
        bool left = l == wl;
        int at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool eq = key[i] == best, hit = eq && left;
            left = left && !eq;
            key[i] = hit ? 0u : key[i];
            at = hit ? i : at;
        }
        if (l == wl) picks[seg + j] = first + at;
    }
    if (bias) {
        tie |= across<W>(best_key(), Max{}) == last;
        if (__any(tie && act)) {
            // values, larger first, then ids, lower first
            uint64_t taken = 0;
            for (int j = 0; j < k; ++j) {
                Key best{0, 0};
                int at = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const Key q = key_of(v[i]);
                    if (live(i) && in && !(taken >> i & 1) && (q.hi > best.hi || (q.hi == best.hi && q.lo > best.lo))) best = q, at = i;
                }
                const uint32_t hi = across<W>(best.hi, Max{}), lo = across<W>(best.hi == hi ? best.lo : 0u, Max{});
                const int wl = lowest(best.hi == hi && best.lo == lo);
                if (l == wl) taken |= uint64_t(1) << at;
                if (l == wl) picks[seg + j] = first + at;
            }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int mine = l < k ? picks[lane] : 0;
    // gates
    const bool chosen = act && l < k;
    const float my_l = chosen ? lrow[mine] : 0.0f;
    // (renormalised softmax: of the chosen logits alone.  Where the largest is not among them they can lie so far below it
    // that their parts of the whole row's sum are 0)
    const bool alone = R.renorm && !R.sigmoid;
    if (alone) m = across<16>(chosen ? my_l : -INFINITY, Max{});
    double s = chosen ? (R.sigmoid ? sigmoid64(my_l) : share64(my_l, m) / (alone ? 1.0 : den)) : 0.0;
    if (R.renorm) {
        const double total = across<16>(s, Add{});            // k <= 16
        if (total != 0.0) s /= total;
    }
    if (chosen) {
        ids_out[l] = mine;
        w_out[l] = float(s * R.scale);
    }
    return mine;
}
// Tokens of a workgroup up to which its counts are bytes: 256 workgroups have 65,280 then, so that sums fit 16 bits.
constexpr int kByteTokens = 255;
static_assert(kMaxTopK <= 16, "a token's gates have a lane each");

// Tokens t0.. of [t0, t1), a wave's 64 / W at a time; each(t, expert) for the lanes of the chosen.
template <int W, int EPL, class Each>
__device__ __forceinline__ void scored_tokens(const float* logits, const float* bias, int t0, int t1, int E, int k, const Rule& R,
                                              int32_t* ids, float* w, int32_t* s_picks, Each each) {
    constexpr int P = kWave / W;
    const int wave = threadIdx.x / kWave, waves = blockDim.x / kWave, l = dev::lane_id() % W;
    for (int tw = t0 + wave * P; tw < t1; tw += waves * P) {
        const int t = tw + dev::lane_id() / W;
        const bool act = t < t1;
        const int64_t row = act ? t : tw;
        const int e = scored_token<W, EPL>(logits + row * E, bias, act, k, R, ids + row * k, w + row * k, s_picks + wave * kWave);
        if (act && l < k) each(t * k + l, e);
    }
}

// T <= 16 and T*k <= 64: everything in one workgroup, a wave a token
template <int EPL>
__global__ __launch_bounds__(1024) void k_scored_tiny(const float* __restrict__ logits, const float* __restrict__ bias,
                                                      int T, int E, int k, const Rule R, int32_t* __restrict__ ids,
                                                      float* __restrict__ w, int32_t* __restrict__ counts,
                                                      int32_t* __restrict__ offsets, int32_t* __restrict__ perm,
                                                      int32_t* __restrict__ inv) {
    __shared__ int32_t s_ids[kWave], s_picks[1024];
    scored_tokens<kWave, EPL>(logits, bias, 0, T, E, k, R, ids, w, s_picks, [&](int p, int e) { s_ids[p] = e; });
    __syncthreads();
    group_tiny(s_ids, T * k, E, counts, offsets, perm, inv);
}
// Counts of a workgroup's pairs by expert: row blockIdx.x of rows, a byte each up to 255 tokens, 16 bits above; `parts` pieces
// of 8 experts, or of 4.
template <int W, int EPL>
__global__ __launch_bounds__(512) void k_scored(const float* __restrict__ logits, const float* __restrict__ bias, int T, int E,
                                                int k, const Rule R, int32_t* __restrict__ ids, float* __restrict__ w,
                                                int each, int parts, uint2* __restrict__ rows) {
    __shared__ int32_t s_cnt[kMaxExperts], s_picks[512];
    for (int e = threadIdx.x; e < kMaxExperts; e += blockDim.x) s_cnt[e] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * each;
    scored_tokens<W, EPL>(logits, bias, t0, min(t0 + each, T), E, k, R, ids, w, s_picks, [&](int, int e) { atomicAdd(&s_cnt[e], 1); });
    __syncthreads();
    const bool bytes = each <= kByteTokens;
    auto four = [&](int e) {
        return uint32_t(s_cnt[e] | s_cnt[e + 1] << 8 | s_cnt[e + 2] << 16) | uint32_t(s_cnt[e + 3]) << 24;
    };
    for (int q = threadIdx.x; q < parts; q += blockDim.x)
        rows[int64_t(blockIdx.x) * parts + q] =
            bytes ? make_uint2(four(8 * q), four(8 * q + 4))
                  : make_uint2(uint32_t(s_cnt[4 * q] | s_cnt[4 * q + 1] << 16), uint32_t(s_cnt[4 * q + 2] | s_cnt[4 * q + 3] << 16));
}

// The pairs of workgroup blockIdx.x of k_scored to their places: an expert's first is behind the pairs of smaller experts and
// those of earlier rows; the others follow by their token, a bit in the expert's mask of 64 tokens (a token has an
// expert once).
//
// The counts of all rows are read by every workgroup, so they are short: with bytes 8,192 tokens of 256 experts take 18.5 us
// for both kernels, with 16 bits 21.9; 2,048 tokens 12.5 and 15.6.
// Sums of bytes stay below 2^16 and go two to a register: the even experts of a word, and the odd ones.
template <bool BYTES>
__global__ __launch_bounds__(kBlock) void k_scored_place(const int32_t* __restrict__ ids, int T, int k, int E, int each,
                                                         int parts, const uint2* __restrict__ rows,
                                                         int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                         int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
    __shared__ int32_t s_cnt[kMaxExperts], s_run[kMaxExperts + 1], s_before[kMaxExperts];
    __shared__ unsigned long long s_mask[kMaxExperts];
    __shared__ uint4 s_part[2][kBlock];                       // all, those before: [group of rows][piece]
    const int tid = threadIdx.x, groups = min(kBlock / parts, 64), q = tid % parts, g = tid / parts;
    const int t0 = blockIdx.x * each, t1 = min(t0 + each, T), own = tid / k;
    auto expert = [&](int t) { return own < 64 && t + own < t1 ? ids[int64_t(t) * k + tid] : -1; };
    int e = expert(t0);
    for (int i = tid; i < E; i += kBlock) s_mask[i] = 0;
    if (g < groups) {
        uint4 all = make_uint4(0, 0, 0, 0), before = all;
#pragma unroll 8
        for (int row = g; row < int(gridDim.x); row += groups) {
            const uint2 c = rows[row * parts + q];
            const uint4 v = BYTES ? make_uint4(c.x & 0x00FF00FFu, c.x >> 8 & 0x00FF00FFu, c.y & 0x00FF00FFu, c.y >> 8 & 0x00FF00FFu)
                                  : make_uint4(c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16);
            const uint32_t in = row < int(blockIdx.x) ? ~0u : 0u;
            all = make_uint4(all.x + v.x, all.y + v.y, all.z + v.z, all.w + v.w);
            before = make_uint4(before.x + (v.x & in), before.y + (v.y & in), before.z + (v.z & in), before.w + (v.w & in));
        }
        s_part[0][g * parts + q] = all;
        s_part[1][g * parts + q] = before;
    }
    __syncthreads();
    const unsigned long long bit = 1ull << (own & 63);
    if (e >= 0) atomicOr(&s_mask[e], bit);
    for (int i = tid; i < 2 * E; i += kBlock) {
        const int which = i >= E ? 1 : 0, c = i - which * E;
        int sum = 0;
        if constexpr (BYTES) {
            // expert 8 p + i: word (i / 4) * 2 + i % 2 of piece p, half i / 2 % 2
            const uint16_t* from = reinterpret_cast<const uint16_t*>(s_part[which]) + (c & ~7) + (c & 4) + (c & 1) * 2 + (c >> 1 & 1);
#pragma unroll 8
            for (int j = 0; j < groups; ++j) sum += from[j * parts * 8];
        } else {
            const int32_t* from = reinterpret_cast<const int32_t*>(s_part[which]) + c;
#pragma unroll 8
            for (int j = 0; j < groups; ++j) sum += from[j * parts * 4];
        }
        (which ? s_before : s_cnt)[c] = sum;
    }
    __syncthreads();
    const bool whole = blockIdx.x == 0;
    wave0_scan(s_cnt, E, s_run, whole ? offsets : nullptr, whole ? counts : nullptr);
    __syncthreads();
    if (e >= 0) {
        const int to = s_run[e] + s_before[e] + __popcll(s_mask[e] & (bit - 1));
        perm[to] = t0 * k + tid;
        inv[t0 * k + tid] = to;
    }
    for (int t = t0 + 64; t < t1; t += 64) {
        __syncthreads();
        for (int i = tid; i < E; i += kBlock) {
            s_before[i] += __popcll(s_mask[i]);
            s_mask[i] = 0;
        }
        e = expert(t);
        __syncthreads();
        if (e >= 0) atomicOr(&s_mask[e], bit);
        __syncthreads();
        if (e >= 0) {
            const int to = s_run[e] + s_before[e] + __popcll(s_mask[e] & (bit - 1));
            perm[to] = t * k + tid;
            inv[t * k + tid] = to;
        }
    }
}

// Gradient of the logits from the gates', one wave a token.  With p the softmax or sigmoid score,
// S the sum of the chosen scores and a_j = p_j / S:
//   gates scale * a_j:  ds_j = scale (dw_j - sum_i dw_i a_i) / S;   gates scale * p_j:  ds_j = scale dw_j
//   sigmoid:  dl_j = ds_j p_j (1 - p_j) for the chosen, 0 for the others.  Renormalised, ds_j p_j is formed as
//             scale (dw_j - sum_i dw_i a_i) a_j: S can be as small as the least 64-bit number, a quotient by it infinite;
//   softmax:  dl_e = p_e (ds_e - sum_j ds_j p_j), ds_e = 0 for the others.  Renormalised, that is
//             scale a_j (dw_j - sum_i dw_i a_i) for the chosen and 0 for the others.
__global__ __launch_bounds__(256) void k_scored_backward(const float* __restrict__ logits, int T, int E, int k,
                                                         const Rule R, const int32_t* __restrict__ ids,
                                                         const float* __restrict__ dw, float* __restrict__ dlogits) {
    constexpr int kPer = kMaxExperts / kWave;
    __shared__ float s_row[4][kMaxExperts];
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
    float m = l, x[kPer];
    if (whole) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            x[i] = lane + kWave * i < E ? lrow[lane + kWave * i] : -INFINITY;
            m = fmaxf(m, x[i]);
        }
    }
    m = across<kWave>(m, Max{});
    double den = 1.0, q[kPer];
    if (whole) {
        den = 0.0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (kWave * i < E) den += q[i] = lane + kWave * i < E ? share64(x[i], m) : 0.0;
        den = sum_lanes(den);
        if (den == 0.0) den = 1.0;
    }
    double p = mine ? (R.sigmoid ? sigmoid64(l) : share64(l, m) / den) : 0.0;
    double v, rest = 0.0;                             // rest: sum of ds_j p_j
    if (R.renorm) {
        double S = sum_lanes(p);
        if (S == 0.0) S = 1.0;
        const double a = p / S, x = a * (d - sum_lanes(d * a));
        v = R.sigmoid ? x * sigmoid64(-double(l)) : x;
    } else if (R.sigmoid) {
        v = d * p * sigmoid64(-double(l));
    } else {
        rest = sum_lanes(d * p);
        v = p * (d - rest);
    }
    // the row in LDS, the chosen over it
    float* row = s_row[threadIdx.x / kWave];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (lane + kWave * i < E) row[lane + kWave * i] = whole ? float(-q[i] / den * rest) : 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (mine) row[id] = float(v);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int e = lane; e < E; e += kWave) drow[e] = row[e];
}

template <int W, int EPL>
hipError_t launch_as(const moe_config& c, const moe_route_rule& r, const float* logits, const float* bias, int32_t T, int32_t* ids,
                     float* w, int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, void* ws, hipStream_t s) {
    const int E = c.n_experts, k = c.top_k;
    const Rule R = rule_of(r, E, W, logits, bias);
    if (scored_alone(T, k)) {
        if constexpr (W == kWave) {
            hipLaunchKernelGGL((k_scored_tiny<EPL>), dim3(1), dim3((T < 1 ? 1 : T) * kWave), 0, s, logits, bias, T, E, k, R, ids, w,
                               counts, offsets, perm, inv);
            return hipGetLastError();
        }
        return hipErrorInvalidValue;
    }
    const int each = scored_each(T), blocks = int((int64_t(T) + each - 1) / each);
    const int waves = each * W / kWave < 8 ? each * W / kWave : 8, parts = each <= kByteTokens ? (E + 7) / 8 : (E + 3) / 4;
    uint2* rows = reinterpret_cast<uint2*>(static_cast<char*>(ws) + ws_layout(c, T).scored);
    hipLaunchKernelGGL((k_scored<W, EPL>), dim3(blocks), dim3(waves * kWave), 0, s, logits, bias, T, E, k, R, ids, w, each,
                       parts, rows);
    const auto place = each <= kByteTokens ? &k_scored_place<true> : &k_scored_place<false>;
    hipLaunchKernelGGL(place, dim3(blocks), dim3(kBlock), 0, s, ids, T, k, E, each, parts, rows, counts, offsets, perm, inv);
    return hipGetLastError();
}

// More tokens than this: 16 lanes a token, 32 where a lane of 16 would have more than 16 experts (registers).  256 experts in
// 8 groups, top 8: 2,048 tokens 18.4 us against 15.5 on waves, 4,096 19.0 against 20.5, 30,000 53 against 84; 512 experts,
// 8,192 tokens: 34 us on 32 lanes, 38 on waves (each 3 less since counts are bytes).
constexpr int kManyTokens = 2048;

// Experts of a lane where W lanes take a token.
int per_lane(const moe_route_rule& r, int E, int W, const void* logits, const void* bias) {
    return rule_of(r, E, W, logits, bias).per;
}

}  // namespace

hipError_t launch_route_scored(const moe_config& c, const moe_route_rule& r, const float* logits, const float* bias,
                               int32_t T, int32_t* ids, float* w, int32_t* counts, int32_t* offsets, int32_t* perm,
                               int32_t* inv, void* ws, hipStream_t s) {
#define MOE_SCORED(W, N) \
    if (per <= N) return launch_as<W, N>(c, r, logits, bias, T, ids, w, counts, offsets, perm, inv, ws, s)
    int per = per_lane(r, c.n_experts, 16, logits, bias);
    if (T > kManyTokens && r.n_groups <= 16) {                // (a group has a lane to itself)
        MOE_SCORED(16, 4);
        MOE_SCORED(16, 8);
        MOE_SCORED(16, 12);
        MOE_SCORED(16, 16);
    }
    per = per_lane(r, c.n_experts, 32, logits, bias);
    if (T > kManyTokens && r.n_groups <= 32 && per > 8) {
        MOE_SCORED(32, 16);
    }
    per = per_lane(r, c.n_experts, kWave, logits, bias);      // (16 at most: 512 experts, lanes > 32 / groups)
    MOE_SCORED(kWave, 1);
    MOE_SCORED(kWave, 2);
    MOE_SCORED(kWave, 4);
    MOE_SCORED(kWave, 8);
    MOE_SCORED(kWave, 16);
#undef MOE_SCORED
    return hipErrorInvalidValue;
}

hipError_t launch_route_scored_backward(const moe_config& c, const moe_route_rule& r, const float* logits, int32_t T,
                                        const int32_t* ids, const float* dw, float* dlogits, hipStream_t s) {
    if (T == 0) return hipSuccess;
    hipLaunchKernelGGL(k_scored_backward, dim3((T + 3) / 4), dim3(256), 0, s, logits, T, c.n_experts, c.top_k,
                       rule_of(r, c.n_experts, kWave, nullptr, nullptr), ids, dw, dlogits);
    return hipGetLastError();
}

}  // namespace moe
