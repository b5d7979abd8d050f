// Products of few tokens with weights contiguous along K: the weight stream.
//
// With few tokens the time is that of reading the weights once.  A workgroup owns 8 R rows of
// the weights and all tokens; its waves split K among them by 128-byte slices (wave w takes
// slices w, w + W, ...), kDepth slices in flight a wave, and meet once, to add their sums in
// LDS in a fixed order.
//
// Weights go straight into the registers of the 16x16 matrix instructions, 8 rows of one whole
// 128-byte line each a load: lane l holds row l % 8, 16-byte piece (l / 16) + 4 (l % 16 / 8).
// To the instruction those are 16 rows of 64 bytes: rows 0-7 are the weight rows' first halves,
// rows 8-15 their second halves.  The activations are held the same way (columns 0-7: 8 tokens'
// first halves, 8-15 their second halves), so of the 16 x 16 sums the two 8 x 8 blocks on the
// diagonal are those of the two halves, and are added at the end; the other two are dropped.
// That leaves half of the instruction's work unused, which a stream does not miss, and needs
// neither a pass through LDS nor loads of half lines: streaming 201 MB as 16 rows of 64 bytes a
// load reads 4.0-5.9 TB/s, as 8 whole lines 6.6 TB/s, as 1 KiB of one row 6.7 TB/s (workgroups
// of 16 rows, non-temporal; of 32 rows 4.9 TB/s).
//
// WALK: a workgroup walks groups of 8 R rows; the next group's first weights are requested before
// the sums of the current one are added, and where K is one pass (ONE: kDepth slices a wave) x
// stays in registers for all groups.  That saves reading x for every group, which from 9 tokens on
// is as much as the weights, and the last workgroups do not end alone (100003 x 4096 codes, kernel
// times: at 8 tokens 73 us, 5.6 TB/s, without a walk and 67 with it).
//
// A pass is 4 KiB of each row.  Workgroups that all begin with the first pass read every other 4 KiB
// of rows of 8 KiB, and then the rest, at the rate of half-used memory channels.  So group g begins
// with pass g % passes (100003 x 8192 codes at 8 tokens 136 us against 169, 6.0 TB/s; 8192 x 8192
// bf16 block at one token 74 against 84; rows of other lengths gained little).
//
// AHEAD (K of several passes, up to 16 rows a workgroup): the next pass's weights and activations
// are requested before the current one's products, in registers of their own (1 token, 100003 x
// 8192 codes 118 us against 139, 4096 x 12288 11.2 against 12.5; with 32 rows the registers cost
// more: 8 tokens, 100003 x 8192 147 against 136).
//
// Measured: 4096 x 12288 bf16 block at one token, 302 MB in 50.6 us (31.5 and 17.2), 6.0 TB/s;
// 100003 x 4096 codes at 8 tokens, 410 MB in 65-67 us, 6.2 TB/s; 2048 x 2048 codes at one token
// 5.1 us, latency.
//
// QUANT: x comes as numbers and every workgroup quantises it for itself, into LDS, while its
// first weights are on the way: T K conversions in each workgroup against a launch and a pass
// through memory, for T K up to kMaxQuant and few outputs.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "dense_common.h"
#include "dense_epilogue.h"

namespace moe {
namespace dense {
namespace {

using dev::kWave;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
constexpr uint32_t kOutside = 0xFFFFFFF0u, kRange = 0x80000000u;
constexpr int kSlice = 128, kDepth = 4, kThreads = 512, kWaves = kThreads / kWave;
static_assert(kWaves * kSlice * kDepth == kFewPass, "a pass of K");
enum { kNoQuant = 0, kQuantBF16 = 1, kQuantF32 = 2 };
constexpr int kMaxQuant = kFewQuant, kQuantVec = kMaxQuant / 8 / kThreads;   // vectors of 8 a thread
constexpr int kCodePad = 16;             // bytes between the code rows: other banks

__device__ __forceinline__ dev::f32x4 mma(const dev::u32x4& a, const dev::u32x4& b, const dev::f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ dev::f32x4 mma_f32(const dev::u32x4& a, const dev::u32x4& b, dev::f32x4 c) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[q]), __uint_as_float(b[q]), c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ i32x4 mma(const dev::u32x4& a, const dev::u32x4& b, const i32x4& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}
template <int TYPE> struct FewAcc { typedef dev::f32x4 T; };
template <> struct FewAcc<kI8> { typedef i32x4 T; };

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, kRange, 0x00027000);
}
constexpr int kStream = 2;               // cache policy of a non-temporal load
template <int POLICY>
__device__ __forceinline__ dev::u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(dev::u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, POLICY));
}

// Barrier over LDS alone: the next weights stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// MT: 8-token tiles; R: 8-row weight tiles of a workgroup.  Gated epilogues: R / 2 tiles of gate
// rows, then those of their up rows (16 rows on in the weights).
template <int TYPE, int EPI, int MT, int R, int QUANT, bool WALK, bool ONE, bool AHEAD>
__global__ void __launch_bounds__(kThreads) k_few(const Product p0, int groups) {
    typedef typename FewAcc<TYPE>::T Acc;
    constexpr int ES = TYPE == kI8 ? 1 : TYPE == kBF16 ? 2 : 4;
    constexpr bool GATE = kPaired<EPI>;
    static_assert(!GATE || R == 2 || R == 4, "gate and up tiles");
    static_assert(WALK || !ONE, "x is kept for the groups of a walk");
    static_assert(!AHEAD || !WALK, "a walk has its next group ahead");
    static_assert(QUANT == kNoQuant || MT == 1, "x quantised on the way: up to 8 tokens");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ uint32_t s_top[8];
    __shared__ float s_scale[8];
    Product p = p0;
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const int T = int(p.M);
    const uint32_t kb = uint32_t(p.K) * ES;
    const int l8 = lane % 8;
    const uint32_t piece = uint32_t(lane / 16 + 4 * (lane % 16 / 8)) * 16;
    // first row of group g, and of its tile r from there; gated: a group has 4 R inner indices
    auto first_row = [&](int g) { return GATE && R == 2 ? int64_t(g) / 2 * 32 + g % 2 * 8 : int64_t(g) * 8 * R; };
    auto tile_row = [](int r) { return GATE ? r / (R / 2) * 16 + r % (R / 2) * 8 : r * 8; };
    uint32_t xo[MT];
    // numbers to quantise: vector v of a thread is 8 numbers of row qrow[v]
    constexpr int NV = QUANT == kNoQuant ? 1 : kQuantVec;
    uint4 qv[NV][QUANT == kQuantF32 ? 2 : 1];
    int qrow[NV], qcol[NV];
    if constexpr (QUANT != kNoQuant) {
        const int per = p.K / 8;
        const __amdgpu_buffer_rsrc_t rx = rsrc(p.a);
        const uint32_t es = QUANT == kQuantF32 ? 4 : 2;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = v * kThreads + tid;
            qrow[v] = i / per;
            qcol[v] = i % per * 8;
            const uint32_t o = qrow[v] < T ? (uint32_t(qrow[v]) * uint32_t(p.lda) + qcol[v]) * es : kOutside;
#pragma unroll
            for (int q = 0; q < int(es) / 2; ++q) {
                const dev::u32x4 u = load16<0>(rx, qrow[v] < T ? o + 16 * q : kOutside);
                qv[v][q] = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
        if (tid < 8) s_top[tid] = 0;
    }
    const __amdgpu_buffer_rsrc_t rx = rsrc(p.a);
#pragma unroll
    for (int m = 0; m < MT; ++m)
        xo[m] = uint32_t(min(m * 8 + l8, T - 1)) * (QUANT != kNoQuant ? p.K + kCodePad : uint32_t(p.lda * ES));
    constexpr uint32_t kStride = kWaves * kSlice, kPass = kStride * kDepth;
    // K goes in passes; group g begins with pass g % passes
    constexpr bool SINGLE = ONE || (!WALK && !AHEAD);
    const int passes = SINGLE ? 1 : int((kb + kPass - 1) / kPass);
    int begin = SINGLE ? 0 : int(blockIdx.x) % passes;
    auto at = [&](int pass) {
        const int q = pass + begin;
        return uint32_t(wave * kSlice) + uint32_t(q >= passes ? q - passes : q) * kPass;
    };
    dev::u32x4 w[AHEAD ? 2 : 1][kDepth][R];
    auto load_w = [&](dev::u32x4 (&w)[kDepth][R], int g, uint32_t s) {
        const int64_t n0 = first_row(g), left = p.N - 1 - n0;   // rows past N repeat the last one
        const __amdgpu_buffer_rsrc_t rw = rsrc(static_cast<const uint8_t*>(p.b) + n0 * p.ldb * ES);
        uint32_t wo[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = tile_row(r) + l8;
            wo[r] = uint32_t(row < left ? row : int(left)) * uint32_t(p.ldb * ES);
        }
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            const uint32_t k = s + d * kStride + piece;         // past K: zeros
#pragma unroll
            for (int r = 0; r < R; ++r) w[d][r] = load16<kStream>(rw, k < kb ? wo[r] + k : kOutside);
        }
    };
    dev::u32x4 x[AHEAD ? 2 : 1][kDepth][MT];
    auto load_x = [&](dev::u32x4 (&x)[kDepth][MT], uint32_t s) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            const uint32_t k = s + d * kStride + piece;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if constexpr (QUANT != kNoQuant)                // (any codes do past K: the weights are zeros there)
                    x[d][m] = *reinterpret_cast<const dev::u32x4*>(lds + (k < kb ? xo[m] + k : 0));
                else
                    x[d][m] = load16<0>(rx, k < kb ? xo[m] + k : kOutside);
            }
        }
    };
    int g = blockIdx.x;
    if constexpr (AHEAD && QUANT == kNoQuant) load_x(x[0], at(0));
    load_w(w[0], g, at(0));
    if constexpr (QUANT != kNoQuant) {
        float f[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (QUANT == kQuantF32) {
                const uint32_t u[8] = {qv[v][0].x, qv[v][0].y, qv[v][0].z, qv[v][0].w,
                                       qv[v][1].x, qv[v][1].y, qv[v][1].z, qv[v][1].w};
#pragma unroll
                for (int j = 0; j < 8; ++j) f[v][j] = __uint_as_float(u[j]);
            } else {
                const uint32_t u[4] = {qv[v][0].x, qv[v][0].y, qv[v][0].z, qv[v][0].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) f[v][2 * j] = dev::bf16_lo(u[j]), f[v][2 * j + 1] = dev::bf16_hi(u[j]);
            }
        }
        __syncthreads();                                        // s_top is clear
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[v][j]) & 0x7FFFFFFFu);
            const int first = __builtin_amdgcn_readfirstlane(qrow[v]);
            if (first >= T) break;
            if (__all(qrow[v] == first)) {                      // one row in the wave: one update
#pragma unroll
                for (int d = kWave / 2; d >= 1; d >>= 1) top = max(top, uint32_t(__shfl_xor(int(top), d, kWave)));
                if (lane == 0) atomicMax(&s_top[first], top);
            } else if (qrow[v] < T) {
                atomicMax(&s_top[qrow[v]], top);
            }
        }
        __syncthreads();
        if (tid < T) s_scale[tid] = row_scale(s_top[tid]);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (qrow[v] >= T) break;
            const float sc = row_scale(s_top[qrow[v]]), inv = inverse_scale(sc);
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j / 4] |= uint32_t(quantize_one(f[v][j], sc, inv) & 255) << (8 * (j % 4));
            *reinterpret_cast<uint2*>(lds + qrow[v] * (p.K + kCodePad) + qcol[v]) = make_uint2(c[0], c[1]);
        }
        __syncthreads();
        p.row_scale = s_scale;
    }
    // LDS: the codes, then two areas of sums, [wave][half][m][r][16]
    constexpr int kSums = 2 * kWaves * MT * R * 16;
    Acc* red0 = reinterpret_cast<Acc*>(lds + (QUANT != kNoQuant ? T * (p.K + kCodePad) : 0));
    Acc acc[MT][R];
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[m][r] = Acc{0, 0, 0, 0};
    };
    auto products = [&](const dev::u32x4 (&w)[kDepth][R], const dev::u32x4 (&x)[kDepth][MT]) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if constexpr (TYPE == kF32) acc[m][r] = mma_f32(w[d][r], x[d][m], acc[m][r]);
                    else acc[m][r] = mma(w[d][r], x[d][m], acc[m][r]);
                }
    };
    // results: thread `tid` finishes 4 columns of one token.  What that reads is requested before
    // the next weights (a wait for a load waits for every older one).
    constexpr int PER = GATE ? 2 : 1, RES = R / PER, ITEMS = MT * RES * 16;    // RES: tiles of results
    static_assert(ITEMS <= kThreads, "one item a thread");
    const int ent = tid % 16, rm = tid / 16 / RES, rr = tid / 16 % RES, rt = rm * 8 + ent % 8;
    ColumnScales<EPI, 4> cs;
    RowInputs<TYPE, EPI, 4> in;
    auto column = [&](int g) { return first_row(g) + rr * 8 + 4 * (ent / 8); };
    auto request = [&](int g) {
        if (tid < ITEMS && rt < T && column(g) < p.N) {
            cs.load(p, int(column(g)));
            in.load(p, rt, int(column(g)));
        }
    };
    // Sums of the diagonal blocks: lanes 0-7 and 16-23 (rows 0-7, first halves), 40-47 and
    // 56-63 (rows 8-15, second halves) as entry lane % 8 + 8 (lane / 16 % 2) of half lane / 32.
    auto reduce = [&](int g, int turn) {
        Acc* red = red0 + (turn & 1) * kSums;
        if ((lane % 16) / 8 == lane / 32) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    red[(((wave * 2 + lane / 32) * MT + m) * R + r) * 16 + l8 + 8 * (lane / 16 % 2)] = acc[m][r];
        }
        // (the other area's readers are past it: they met at the barrier before this one)
        lds_barrier();
        if (tid >= ITEMS) return;
        Acc sum[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int tile = rm * R + rr + q * RES;
            sum[q] = red[tile * 16 + ent];
#pragma unroll
            for (int v = 1; v < 2 * kWaves; ++v) sum[q] += red[(v * MT * R + tile) * 16 + ent];
        }
        if (rt >= T || column(g) >= p.N) return;
        typename Elem<TYPE>::Acc v[4], u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = sum[0][e], u[e] = sum[PER - 1][e];
        finish<TYPE, EPI, 4, false>(p, rt, int(column(g)), v, u, cs, in);
    };
    if constexpr (ONE) load_x(x[0], at(0));
    for (int turn = 0; g < groups; ++turn) {
        const int next = g + int(gridDim.x);
        clear();
        if constexpr (AHEAD) {
            if constexpr (QUANT != kNoQuant) load_x(x[0], at(0));
            for (int pass = 0;; pass += 2) {
                if (pass + 1 < passes) load_x(x[1], at(pass + 1)), load_w(w[1], g, at(pass + 1));
                products(w[0], x[0]);
                if (pass + 1 >= passes) break;
                if (pass + 2 < passes) load_x(x[0], at(pass + 2)), load_w(w[0], g, at(pass + 2));
                products(w[1], x[1]);
                if (pass + 2 >= passes) break;
            }
        } else {
            for (int pass = 0;;) {
                if constexpr (!ONE) load_x(x[0], at(pass));
                products(w[0], x[0]);
                if (++pass >= passes) break;
                load_w(w[0], g, at(pass));
            }
        }
        if constexpr (!SINGLE && WALK) begin = next % passes;
        request(g);
        if (WALK && next < groups) load_w(w[0], next, at(0));
        reduce(g, turn);
        if (!WALK) break;
        g = next;
    }
}

template <int TYPE, int EPI, int MT, int R, int QUANT, bool WALK>
hipError_t launch_few_as(const Product& p, bool one, hipStream_t s) {
    const int64_t groups = (int64_t(p.N) + 8 * R - 1) / (8 * R);
    const int lds = (WALK ? 2 : 1) * 2 * kWaves * MT * R * 16 * 16 + (QUANT ? int(p.M) * (p.K + kCodePad) : 0);
    if constexpr (!WALK) {
        static_assert(R <= 2, "registers for the next pass");
        if (one)
            hipLaunchKernelGGL((k_few<TYPE, EPI, MT, R, QUANT, false, false, false>), dim3(unsigned(groups)),
                               dim3(kThreads), lds, s, p, int(groups));
        else
            hipLaunchKernelGGL((k_few<TYPE, EPI, MT, R, QUANT, false, false, true>), dim3(unsigned(groups)),
                               dim3(kThreads), lds, s, p, int(groups));
    } else {
        // 32 rows: a workgroup a CU (its registers hold 128 KiB of weights); 16: up to four, each the
        // same number of groups
        const int64_t most = int64_t(compute_units()) * (R == 4 ? 1 : 4), turns = (groups + most - 1) / most;
        const dim3 grid(unsigned(R == 4 ? std::min(groups, most) : (groups + turns - 1) / turns));
        if (one)
            hipLaunchKernelGGL((k_few<TYPE, EPI, MT, R, QUANT, true, true, false>), grid, dim3(kThreads), lds, s, p, int(groups));
        else
            hipLaunchKernelGGL((k_few<TYPE, EPI, MT, R, QUANT, true, false, false>), grid, dim3(kThreads), lds, s, p, int(groups));
    }
    return hipGetLastError();
}

template <int TYPE, int EPI>
hipError_t choose_few(const Product& p, int quant, hipStream_t s) {
    const Few f = plan_few(p.sizes(), elem_bytes(TYPE), kPaired<EPI>, quant != kNoQuant, compute_units());
    if constexpr (TYPE == kI8) {
        if (quant == kQuantBF16) return launch_few_as<TYPE, EPI, 1, 2, kQuantBF16, false>(p, f.one, s);
        if constexpr (EPI != kGate8) {           // (gate and up read bf16 activations)
            if (quant == kQuantF32) return launch_few_as<TYPE, EPI, 1, 2, kQuantF32, false>(p, f.one, s);
        }
    }
    if constexpr (!kPaired<EPI>) {
        if (f.r == 1) return launch_few_as<TYPE, EPI, 1, 1, kNoQuant, false>(p, f.one, s);
    }
    if (f.mt == 1 && f.walk) return launch_few_as<TYPE, EPI, 1, 4, kNoQuant, true>(p, f.one, s);
    if (f.mt == 1) return launch_few_as<TYPE, EPI, 1, 2, kNoQuant, false>(p, f.one, s);
    if (f.mt == 2 && f.r == 4) return launch_few_as<TYPE, EPI, 2, 4, kNoQuant, true>(p, f.one, s);
    if (f.mt == 2) return launch_few_as<TYPE, EPI, 2, 2, kNoQuant, true>(p, f.one, s);
    return launch_few_as<TYPE, EPI, 4, 2, kNoQuant, true>(p, f.one, s);
}

}  // namespace

hipError_t launch_few(int type, int epi, const Product& p, hipStream_t s, int x_type, bool quant) {
    if (p.M > kFewTokens) return hipErrorInvalidValue;
    const int q = !quant ? kNoQuant : x_type == MOE_A_F32 ? kQuantF32 : kQuantBF16;
    if (quant && (type != kI8 || p.M > 8 || p.M * p.K > kFewQuant)) return hipErrorInvalidValue;
    if (epi == kGate8 && q == kQuantF32) return hipErrorInvalidValue;
    if (type == kI8) {
        if (epi == kScale) return choose_few<kI8, kScale>(p, q, s);
        if (epi == kScale32) return choose_few<kI8, kScale32>(p, q, s);
        if (epi == kGate8) return choose_few<kI8, kGate8>(p, q, s);
    } else if (type == kBF16) {
        if (epi == kStore) return choose_few<kBF16, kStore>(p, q, s);
        if (epi == kGate) return choose_few<kBF16, kGate>(p, q, s);
    } else {
        if (epi == kStore) return choose_few<kF32, kStore>(p, q, s);
        if (epi == kGate) return choose_few<kF32, kGate>(p, q, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace dense
}  // namespace moe
