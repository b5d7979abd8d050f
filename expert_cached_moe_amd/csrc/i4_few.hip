// Products of few rows of x with 4-bit weights, dense and by expert: the stream of codes.
//
// The time is that of reading the codes once, so the work on a code has to be small: at 6 TB/s a CU
// receives a code for every 0.8 cycles of one lane.  The 4x4x4 matrix instruction does 16 products of
// 4 x 4 with 4 k each, one in every four lanes.  A wave loads 4 weight rows x 512 codes at a time: lane l
// holds 32 codes, a piece, of row l % 4, and block l / 4 of the instruction has one k range of 32, so one
// group.  Codes become bf16 numbers 0..15 by three masks and shifts and four conversions per eight (bytes
// 0..15 are e4m3 numbers 2^-9 times themselves), eight instructions of the matrix unit sum x * code over
// the piece for four tokens, started with -z * (sum of x), which gives sum x * (code - z); four
// multiply-adds add that, times s and the row's power of two, to the sums.  So a code takes 1.2 operations of a lane
// for up to 4 tokens and 1.4 for 8, of the 3.3 that there is time for; scaling every weight would take 2.4.  The power of
// two takes part in each step, and not once at the end, because sums without it leave fp32 at one end or the other: of x
// from 2^103 up in rows of small weights, or of x below 2^-94 in rows of large ones (it costs 1-3%).
//
// The waves of a workgroup split K (by chunks of 512); sums meet once a
// unit of rows, across the blocks in registers, across the waves in LDS, in a fixed order.  Every tile's
// registers are loaded again as soon as it is used, with the next chunk or the next unit of rows.  The stream still
// stops once a pass: the loop's registers are copied at its back edge and behind it, so the compiler waits there until all
// weights of the next pass have landed, before this unit's sums are reduced.  With K above 4096 there are several passes
// (8 waves of 512), and x is read again in each pass of each unit, its loads under branches, with no weights in flight.
// These waits bound the kernel, and where few workgroups have a row's passes to walk, their number.
//
// Measured (kernel): 2048 x 2048 at one token 4.0-4.6 us (launch, one trip to memory, the sums; its 2.2 MB take 0.4), 100003 x
// 4096 at 4 tokens 48-50 (220 MB at 4.5 TB/s; 33 at the rate of a bare read), at 8 tokens 71, at 4 fp32 tokens 71; 32768 x 12288
// at one token 46, at 4 tokens 58 (214 MB: 32 at the rate of a bare read); 7 experts of 4096 x 1536 at one token 19 and 9.9
// (50 and 25 MB).  Twice the rows a wave (more bytes in flight, fewer waves) 3% slower, half of them 14-30%.
//
// Experts: each workgroup lists the entries that have rows, from the offsets, in blocks of 4 rows at most, and walks their
// units.  Blocks of 8 cost more registers, so waves, for the few entries that fill them (256 experts of 4096 x 1536 with
// the shared one, top 6, 8 tokens: 157 us against 118; 128 of 2048 x 768, top 8: 48.5 and 48.9).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "dense.h"
#include "i4_common.h"

namespace moe {
namespace i4 {
namespace {

using dev::kWave;

typedef __attribute__((ext_vector_type(4))) short s16x4;

constexpr int kChunk = 512, kMaxWaves = 8, kStream = 2;       // cache policy of a non-temporal load
constexpr int kFewBlocks = kFewTokens * kMaxTopK + 2;          // of up to 4 rows: a block a pair at most, the shared expert's two
constexpr uint32_t kOutside = 0xFFFFFFF0u, kRange = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, kRange, 0x00027000);
}

// Barrier over LDS alone: loads of weights stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, false));
}

// Four codes as bf16 numbers, divided by 512 (so that sums of 32 stay in range whatever x is), from bytes (even codes of four in `even`, odd ones in `odd`; HIGH: the upper two of each)
template <bool HIGH>
__device__ __forceinline__ s16x4 codes4(uint32_t even, uint32_t odd) {
    const uint2 u = make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(even), 1.0f, HIGH)),
                               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(odd), 1.0f, HIGH)));
    return __builtin_bit_cast(s16x4, u);
}

// 512 times a group's scale times its row's 2^(e - 127); 255 is NaN
__device__ __forceinline__ float row_and_group(uint32_t word, uint32_t e) {
    return __builtin_amdgcn_ldexpf(word_scale(e == 255u ? 0x7Fu : word), int(e) - 118);
}

// Waves on a SIMD: what the registers allow.
template <int MAXMT, int P>
constexpr int kWavesPerSimd = MAXMT * P == 1 ? 4 : MAXMT * P <= 3 ? 3 : 2;

struct Few {
    int kw;                  // waves along K
    int units;               // of an entry: runs of 4 R rows (gated: 2 R gate rows and their up rows)
    int entries;             // dense: runs of 4 MT tokens; experts: entries of the list
};

// What a unit of rows is: an entry's rows of x, and its weights.
struct Entry {
    int64_t offset;          // bytes of its blob from slot 0
    int base, count;
    bool shared;
};

template <int KIND, int MAXMT, int R, int P>
__global__ void __launch_bounds__(kMaxWaves* kWave) __attribute__((amdgpu_waves_per_eu(kWavesPerSimd<MAXMT, P>)))
k_i4_few(const Product p, const ListOf<KIND> list, const Few f) {
    constexpr bool GATE = KIND == kGateUp, EXPERTS = KIND == kGateUp || KIND == kDown;
    __shared__ int4 s_entry[EXPERTS ? kFewBlocks : 1];
    __shared__ int s_waves[kMaxWaves];
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int j = lane % 4, block = lane / 4;
    const int units = f.units, chunks = (p.K + kChunk - 1) / kChunk, passes = (chunks + f.kw - 1) / f.kw;
    const int pieces = p.K / 32;

    int total = f.entries * units;
    if constexpr (EXPERTS) {
        // entries with rows, in the list's order (the same list in every workgroup); one of more rows is several
        // of 4 MAXMT
        int active = 0;
        for (int i0 = 0; i0 < list.n; i0 += blockDim.x) {
            const int i = i0 + tid;
            int base = 0, count = 0, ent = 0;
            if (i < list.n) {
                ent = list.ent[i];
                const int e = ent & 1023;
                base = e == kSharedTag ? int(p.T) * p.top_k : p.offsets[e];
                count = e == kSharedTag ? int(p.T) : p.offsets[e + 1] - base;
            }
            const int blocks = (count + 4 * MAXMT - 1) / (4 * MAXMT);
            int incl = blocks;
            if (__any(blocks > 1)) {
#pragma unroll
                for (int d = 1; d < kWave; d <<= 1) {
                    const int o = __shfl_up(incl, d, kWave);
                    if (lane >= d) incl += o;
                }
            } else {
                incl = __popcll(__ballot(blocks) << (63 - lane));
            }
            if (i0) __syncthreads();                          // the last turn's sums are read
            if (lane == kWave - 1) s_waves[wave] = incl;
            __syncthreads();
            int first = active + incl - blocks;
            for (int w = 0; w < int(blockDim.x) / kWave; ++w) {
                const int n = s_waves[w];
                if (w < wave) first += n;
                active += n;
            }
            for (int q = 0; q < blocks; ++q)
                if (first + q < kFewBlocks)                   // (the host has seen to it)
                    s_entry[first + q] = make_int4(ent, base + q * 4 * MAXMT, min(count - q * 4 * MAXMT, 4 * MAXMT), 0);
        }
        __syncthreads();
        total = __builtin_amdgcn_readfirstlane(active) * units;
    }
    auto entry_of = [&](int u) {
        const int a = u / units;
        if constexpr (EXPERTS) {
            const int4 s = s_entry[a];
            const int ent = __builtin_amdgcn_readfirstlane(s.x);
            return Entry{blob_offset(p, ent), __builtin_amdgcn_readfirstlane(s.y), __builtin_amdgcn_readfirstlane(s.z),
                         (ent & 1023) == kSharedTag};
        } else {
            const int t0 = a * 4 * MAXMT;
            return Entry{0, t0, int(p.T) - t0 < 4 * MAXMT ? int(p.T) - t0 : 4 * MAXMT, false};
        }
    };
    // first row of a unit, and row of tile r from there
    auto first_row = [](int unit) {
        return GATE ? unit / (8 / R) * 32 + unit % (8 / R) * (2 * R) : unit * (4 * R);
    };
    auto tile_row = [](int r) { return GATE ? r / (R / 2) * 16 + r % (R / 2) * 4 : r * 4; };

    dev::u32x4 w[R];
    uint32_t word[R], ex[R];
    __amdgpu_buffer_rsrc_t rc = rsrc(p.w.codes), rg = rsrc(p.w.words), re = rsrc(p.w.exps);
    uint32_t first = 0, left = 0;                               // first row of the unit, and rows behind it
    auto aim = [&](int u) {
        const Entry e = entry_of(u);
        const int n0 = first_row(u % units);
        const Rows rows = rows_at(p.w, e.offset);
        rc = rsrc(rows.codes + int64_t(n0) * (p.K / 2));
        rg = rsrc(rows.words + int64_t(n0 & ~15) * p.w.groups);
        re = rsrc(rows.exps + n0);
        first = uint32_t(n0);
        left = uint32_t(p.N - 1 - n0);
    };
    // (from the first word of the unit's run of 16 rows)
    auto word_of = [&](uint32_t row, uint32_t group) {
        const uint32_t n = first + row, run = n & ~15u, rest = uint32_t(p.N) - run;
        return (run - (first & ~15u)) * uint32_t(p.w.groups) + group * (rest < 16 ? rest : 16u) + (n - run);
    };
    auto load = [&](int r, int pass) {
        const int piece = (pass * f.kw + wave) * 16 + block;
        const uint32_t row = min(uint32_t(tile_row(r) + j), left);
        const bool in = piece < pieces;
        w[r] = __builtin_bit_cast(dev::u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            rc, in ? row * uint32_t(p.K / 2) + uint32_t(piece) * 16 : kOutside, 0, kStream));
        word[r] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(
            rg, in ? word_of(row, uint32_t(piece) * 32 >> p.w.shift) * 2 : kOutside, 0, 0));
        ex[r] = uint8_t(__builtin_amdgcn_raw_buffer_load_b8(re, row, 0, 0));
    };

    // this workgroup's units.  Experts: a run of them, so that it changes entries seldom; else all workgroups
    // walk through the weights side by side (100003 x 4096 at one token 53.4 us against 55.1)
    const int share = total / int(gridDim.x), more = total % int(gridDim.x), id = int(blockIdx.x);
    const int step = EXPERTS ? 1 : int(gridDim.x);
    int u = EXPERTS ? id * share + (id < more ? id : more) : id;
    const int end = EXPERTS ? u + share + (id < more ? 1 : 0) : total;
    if (u >= end) return;
    aim(u);
#pragma unroll
    for (int r = 0; r < R; ++r) load(r, 0);

    // x of the wave's chunk: 4 tokens a tile, in the order of the codes, and its sums; where K is one pass
    // they stay for all units of an entry
    s16x4 x[P][MAXMT][8];
    dev::f32x4 xs[MAXMT];
    const uint16_t* xr[MAXMT];
    int turn = 0;
    auto run = [&](auto mt_, const Entry& e, int u, bool fresh) {
        constexpr int MT = decltype(mt_)::value, V = R * MT * 4, Q = V / 4;
        const int next = u + step;
        dev::f32x4 y[MT][R];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (fresh) {
                const int t = min(4 * m + j, e.count - 1);
                xr[m] = p.x + (EXPERTS ? row_in<KIND>(p, e.shared, e.base, t) : int64_t(e.base) + t) * p.ldx;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) y[m][r] = dev::f32x4{0, 0, 0, 0};
        }
        // results: a thread's items are a row each (gated: a gate row) of one token
        constexpr int ROWS = GATE ? 2 * R : 4 * R, ITEMS = ROWS * MT * 4;
        const int threads = blockDim.x;
        struct Item {
            int n, t, at, up;                                   // row of the weights, token, places in the sums
            bool live;
        };
        auto item = [&](int q) {
            const int i = q * threads + tid, row = i % ROWS, t = i / ROWS, tile = row / 4;
            const int n = first_row(u % units) + tile_row(tile) + row % 4;
            const int v = ((t / 4) * R + tile) * 4 + t % 4;     // of tile's value; its up row's: R / 2 tiles on
            auto place = [&](int v) { return (v / Q * 4 + row % 4) * Q + v % Q; };
            return Item{n, t, place(v), place(v + 2 * R), i < ITEMS && t < e.count && n < p.N};
        };
        // its row of out
        auto row_of = [&](const Item& i) {
            return i.live ? int32_t(EXPERTS ? row_out<KIND>(p, e.shared, e.base, i.t) : int64_t(e.base) + i.t) : 0;
        };
        int32_t first = 0;
        for (int pass = 0; pass < passes; ++pass) {
            const int piece = (pass * f.kw + wave) * 16 + block;
            if (fresh || passes > 1) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int a = 0; a < P; ++a) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint4 d = make_uint4(0, 0, 0, 0);
                            if (piece < pieces) d = *reinterpret_cast<const uint4*>(xr[m] + a * p.plane + piece * 32 + q * 8);
                            // x0 x2 x1 x3, x4 x6 x5 x7: the order of the codes
                            x[a][m][2 * q] = __builtin_bit_cast(s16x4, make_uint2(__builtin_amdgcn_perm(d.y, d.x, 0x05040100),
                                                                                  __builtin_amdgcn_perm(d.y, d.x, 0x07060302)));
                            x[a][m][2 * q + 1] = __builtin_bit_cast(s16x4, make_uint2(__builtin_amdgcn_perm(d.w, d.z, 0x05040100),
                                                                                      __builtin_amdgcn_perm(d.w, d.z, 0x07060302)));
                        }
                    }
                    const s16x4 unit = __builtin_bit_cast(s16x4, make_uint2(0x3B003B00u, 0x3B003B00u));
                    xs[m] = dev::f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int a = P - 1; a >= 0; --a)
#pragma unroll
                        for (int q = 0; q < 8; ++q) xs[m] = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(x[a][m][q], unit, xs[m], 0, 0, 0);
                }
            }
            const bool last = pass + 1 == passes;
            if (last) {
                // (ahead of the next unit's weights: a wait for a load waits for every older one; a thread has one item
                // with four waves along K and more)
                first = row_of(item(0));
                if (next < end) aim(next);
            }
            const int ahead = last ? 0 : pass + 1;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float s = row_and_group(word[r], ex[r]), z = -word_zero(word[r]);
                s16x4 b[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t even = w[r][q] & 0x0F0F0F0Fu, odd = w[r][q] >> 4 & 0x0F0F0F0Fu;
                    b[2 * q] = codes4<false>(even, odd);
                    b[2 * q + 1] = codes4<true>(even, odd);
                }
                if (!last || next < end) load(r, ahead);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    dev::f32x4 d = {z * xs[m][0], z * xs[m][1], z * xs[m][2], z * xs[m][3]};
#pragma unroll
                    for (int a = P - 1; a >= 0; --a)
#pragma unroll
                        for (int q = 0; q < 8; ++q) d = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(x[a][m][q], b[q], d, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[m][r][i] = fmaf(s, d[i], y[m][r][i]);
                }
            }
        }
        // sums over the blocks: halves of the values to the lanes of each half and each other row of 16 lanes,
        // then all four blocks of a row add up
        float v[V];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[(m * R + r) * 4 + i] = y[m][r][i];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) v[i] = dev::swap_add<32>(v[i], v[i + V / 2]);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) v[i] = dev::swap_add<16>(v[i], v[i + V / 4]);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) v[i] += dpp<0x128>(v[i]);      // row_ror:8
#pragma unroll
        for (int i = 0; i < V / 4; ++i) v[i] += dpp<0x124>(v[i]);      // row_ror:4
        float* mine = red + (turn & 1) * (kMaxWaves * R * MAXMT * 16);
        if (lane % 16 < 4) {
            float* d = mine + wave * (V * 4) + (lane / 16 * 4 + j) * Q;
#pragma unroll
            for (int i = 0; i < Q; ++i) d[i] = v[i];
        }
        // (the other area's readers are past it: they met at the barrier before this one)
        lds_barrier();
        ++turn;
        for (int q = 0; q * threads < ITEMS; ++q) {
            const Item i = item(q);
            if (!i.live) continue;
            const int64_t to = q == 0 ? first : row_of(i);
            float sum = 0.0f, up = 0.0f;
#pragma unroll 8
            for (int k = 0; k < f.kw; ++k) {
                sum += mine[i.at + k * (V * 4)];
                if constexpr (GATE) up += mine[i.up + k * (V * 4)];
            }
            if constexpr (GATE) {
                static_cast<uint16_t*>(p.out)[to * p.ldo + i.n / 32 * 16 + i.n % 16] = dev::f32_to_bf16_bits(gated(sum, up));
            } else if constexpr (KIND == kOut32) {
                static_cast<float*>(p.out)[to * p.ldo + i.n] = sum;
            } else {
                static_cast<uint16_t*>(p.out)[to * p.ldo + i.n] = dev::f32_to_bf16_bits(sum);
            }
        }
    };
    int had = -1;
    for (; u < end; u += step) {
        const Entry e = entry_of(u);
        const bool fresh = u / units != had;
        had = u / units;
        if constexpr (MAXMT >= 2) {
            if (e.count > 4) run(std::integral_constant<int, 2>{}, e, u, fresh);
        }
        if (e.count <= 4) run(std::integral_constant<int, 1>{}, e, u, fresh);
    }
}

template <int KIND, int MAXMT, int R, int P>
hipError_t launch_as(const Product& p, const ExpertList* list, hipStream_t s) {
    const int n_cu = dense::compute_units();
    const int chunks = (p.K + kChunk - 1) / kChunk;
    Few f;
    // waves along K: all of a row in one pass where there are enough
    f.kw = chunks < kMaxWaves ? chunks : kMaxWaves;
    f.units = int((int64_t(p.N) + 4 * R - 1) / (4 * R));
    f.entries = list ? 0 : int((p.T + 4 * MAXMT - 1) / (4 * MAXMT));
    const int per_cu = std::max(1, 4 * kWavesPerSimd<MAXMT, P> / f.kw);
    const int64_t units = int64_t(f.units) * (list ? std::min<int64_t>(2 * list->n, p.T * p.top_k + 2) : f.entries);
    const int64_t grid = std::min<int64_t>(units, int64_t(n_cu) * per_cu);
    const int lds = 2 * kMaxWaves * R * MAXMT * 16 * 4;
    hipLaunchKernelGGL((k_i4_few<KIND, MAXMT, R, P>), dim3(unsigned(grid)), dim3(f.kw * kWave), lds, s, p,
                       list_of<KIND>(list), f);
    return hipGetLastError();
}

template <int KIND, int P>
hipError_t choose(const Product& p, const ExpertList* list, hipStream_t s) {
    if constexpr (KIND == kOut16 || KIND == kOut32)
        if (p.T > 4) return launch_as<KIND, 2, 4, P>(p, list, s);
    return launch_as<KIND, 1, 4, P>(p, list, s);
}

}  // namespace

hipError_t launch_i4_few(int kind, const Product& p, const ExpertList* list, hipStream_t s) {
    if (p.T == 0) return hipSuccess;
    if (list && p.T > kFewTokens) return hipErrorInvalidValue;      // (more blocks than a workgroup lists)
    const bool parts = p.planes == 3;
    switch (kind) {
        case kOut16: return parts ? choose<kOut16, 3>(p, nullptr, s) : choose<kOut16, 1>(p, nullptr, s);
        case kOut32: return parts ? choose<kOut32, 3>(p, nullptr, s) : choose<kOut32, 1>(p, nullptr, s);
        case kGateUp: return choose<kGateUp, 1>(p, list, s);
        default: return choose<kDown, 1>(p, list, s);
    }
}

}  // namespace i4
}  // namespace moe
