// Products of many rows of x with 4-bit weights: 256 x 256 tiles on the matrix cores, dense and by expert.
//
// 8 waves, two on each SIMD, in two groups that take turns: while one group runs the matrix instructions
// of half a slice of K (32 of them, 512 cycles of the matrix unit), the other reads its fragments of the
// next half from LDS; a barrier ends each turn.  A slice is 64 of K, 32 KiB of either operand, in a ring of
// five places that is all of the LDS.  x comes straight into its place by loads into LDS; the weights
// come as codes, 16 bytes a thread and slice, requested two slices before they are decoded and four before they are
// multiplied (the wait for those of an even slice is one for all loads, so also for the odd slice's behind them,
// requested a turn earlier), and become exact bf16 weights in the reading turns: 32 codes of one group a thread, 16 in each turn, 38 vector operations and two 16-byte
// LDS writes, beside 12 fragment reads.  A turn's LDS traffic, 48 KiB read and 8 written by a group,
// takes 448 of its 512 cycles.  So the codes are decoded once a tile, the weights never pass through
// memory, and the matrix units are fed as by a product of bf16 weights.
//
// Measured: 8,192 x 4096 x 8192 435-466 us (1.18-1.26 PFLOP/s; 380 at the rate of a library product of 8192^3); a slice takes
// 1.6 us with few tiles and 1.8-1.9 with every CU busy, a tile 8-10 besides for its start and its results.  128 experts of
// 2048 x 768, top 8, 8,192 tokens 503 and 317: of the tiles of experts with 512 rows on average a fifth is empty, and the 12
// slices of the down product are 22 of a tile's 32 us.
//
// In slice j of a group's turns, B of slice j lies at place u, x at u + 1, those of the next slice behind
// them; in the reading turns x of slice j + 1 is requested into u + 3 and the weights of slice j + 2 are
// written to u + 4 = u - 1: the places of slice j - 1, which both groups have read.
#include <hip/hip_runtime.h>

#include <atomic>
#include <type_traits>

#include "i4_common.h"

namespace moe {
namespace i4 {
namespace {

using dev::kWave;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;
typedef uint32_t __attribute__((ext_vector_type(4), aligned(4))) words4;
// (bf16 results lie on 2 bytes where rows have an odd number of them: 5012 x 480 x 84667 542 us, 974 in single stores)
typedef uint32_t __attribute__((ext_vector_type(4), aligned(2))) halves8;

constexpr int kXcds = 8, kGroupM = 8, kSlice = 128, kThreads = 512, kB = 256;
constexpr int WN = 2, TM = 64, TN = 128, FM = 4, FN = 8;       // waves 4 x 2 of 64 x 128
constexpr int kPlace = 256 * kSlice, kPlaces = 5, kLds = kPlace * kPlaces;
constexpr int kFinishRow = TN * 4 + 16;
static_assert(8 * 16 * kFinishRow <= kLds && kLds <= 160 * 1024, "LDS of a CU");

__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }
// vector memory operations that may be in flight, LDS operations (15: any)
constexpr int wait_for(int vm, int lgkm) { return (vm & 15) | (7 << 4) | (lgkm << 8) | ((vm >> 4) << 14); }

__device__ __forceinline__ dev::f32x4 mma(const bf16x8& a, const bf16x8& b, const dev::f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ void fence_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void lanes_in_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// A 16-byte write to LDS.  In assembly: the compiler takes one to depend on every load into LDS in flight and
// waits for all of them first.  (Its data is read as it is issued; the turn's own wait covers it.)
__device__ __forceinline__ void write16(uint8_t* to, const dev::u32x4& v) {
    asm volatile("ds_write_b128 %0, %1" ::"v"(uint32_t(reinterpret_cast<uintptr_t>((lds_void*)to))), "v"(v) : "memory");
}

template <int KIND>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
k_i4_turns(const Product p, const ListOf<KIND> list, const int4* __restrict__ map, int n_tiles, int m_tiles) {
    constexpr bool EXPERTS = KIND == kGateUp || KIND == kDown, GATE = KIND == kGateUp;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];

    // workgroup b serves XCD b % 8, each XCD a contiguous run of the tiles' order
    const int total = (EXPERTS ? reinterpret_cast<const int*>(map)[0] : m_tiles) * n_tiles;
    const int per = (total + kXcds - 1) / kXcds, lid = int(blockIdx.x) % kXcds * per + int(blockIdx.x) / kXcds;
    if (int(blockIdx.x) / kXcds >= per || lid >= total) return;
    int base = 0, left, n0;
    int64_t r0;
    bool shared = false;
    Rows w = p.w;
    if constexpr (EXPERTS) {
        const int4 rec = map[1 + lid / n_tiles];
        n0 = lid % n_tiles * kB;
        r0 = int64_t(rec.y) * kB;
        base = rec.z;
        left = rec.w - int(r0);
        const int ent = list.ent[rec.x];
        shared = (ent & 1023) == kSharedTag;
        w = rows_at(p.w, blob_offset(p, ent));
    } else {
        // groups of kGroupM row tiles, columns slowest: the tiles in flight on an XCD share operands in its L2
        const int grp = lid / (kGroupM * n_tiles), in = lid % (kGroupM * n_tiles);
        const int gm = min(kGroupM, m_tiles - grp * kGroupM);
        r0 = int64_t(grp * kGroupM + in % gm) * kB;
        n0 = in / gm * kB;
        left = int(min(p.T - r0, int64_t(kB)));
    }
    const int rows = min(left, kB);

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int wm = wave / WN, wn = wave % WN;
    const bool mine = wm * TM < rows;                         // (a wave without rows computes nothing)
    const bool second = wave >= 4;                            // (SIMD i has waves i and i + 4)

    // x: a wave's loads of a slice are 4 times 8 rows; chunk c of row r at slot c ^ row_swz(r).  Where K ends in
    // the middle of a slice, the lanes of its second half read the first again: it is not used.
    const uint16_t* xa[4];
    const int slices = (p.K + 63) / 64, n = slices * p.planes;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = (wave + 8 * q) * 8 + lane / 8, c = lane % 8 ^ row_swz(r), rr = min(r, rows - 1);
        const int64_t from = EXPERTS ? row_in<KIND>(p, shared, base, int(r0) + rr) : r0 + rr;
        xa[q] = p.x + from * p.ldx + c * 8 + (p.planes - 1) * p.plane;        // smallest parts first
    }
    const bool odd = p.K % 64 != 0;
    int slice_x = 0;                                          // next to request
    auto place = [&](int u) { return lds + (u >= kPlaces ? u - kPlaces : u) * kPlace; };
    auto issue_x = [&](int u) {
        uint8_t* d = place(u) + wave * 1024;
        const bool cut = odd && slice_x + 1 == slices;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = (wave + 8 * q) * 8 + lane / 8, c = lane % 8 ^ row_swz(r);
            __builtin_amdgcn_global_load_lds((global_void*)(xa[q] - (cut && c >= 4 ? 32 : 0)), (lds_void*)(d + q * 8192), 16, 0, 0);
            xa[q] += 64;
        }
        if (++slice_x == slices) {
            slice_x = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) xa[q] -= p.plane + slices * 64;
        }
    };
    // weights: thread t has half t % 2 of row t / 2
    const int half_b = tid % 2, br = tid / 2;
    const int64_t nb = min(n0 + br, p.N - 1);
    const uint8_t* codes = w.codes + nb * (p.K / 2) + half_b * 16;
    const WordAt wa = word_at(nb, p.N, w.groups);
    const uint16_t* words = w.words + wa.first;
    const float S = row_scale(w.exps[nb]);
    // (words are widened where they are used, so that their loads stay in flight)
    dev::u32x4 code[2];                                       // of slices of even and odd number
    uint16_t word[2];
    int slice_w = 0;
    auto load_w = [&](dev::u32x4& code, uint16_t& word) {
        const int k = min(slice_w * 64 + half_b * 32, p.K - 32);       // (past K: any codes; not used)
        code = *reinterpret_cast<const dev::u32x4*>(codes + (k - half_b * 32) / 2);
        word = words[(k >> w.shift) * wa.step];
        if (++slice_w == slices) slice_w = 0;
    };
    float s2 = 0, off = 0;
    auto scales = [&](uint32_t word) {
        const float s = word_scale(word) * S;
        off = -word_zero(word) * s;
        s2 = s * 512.0f;
    };
    auto put_w = [&](int u, int q, const dev::u32x4& code) {
        write16(place(u) + br * kSlice + ((half_b * 4 + q) ^ row_swz(br)) * 16, decode8(code[q], s2, off));
    };
    const int at0 = (lane % 16) * kSlice + ((lane / 16 ^ row_swz(lane % 16)) << 4);
    auto read = [&](const uint8_t* from, int half, auto& v) {
        constexpr int NF = sizeof(v) / sizeof(bf16x8);
#pragma unroll
        for (int i = 0; i < NF; ++i) v[i] = *reinterpret_cast<const bf16x8*>(from + (at0 ^ half << 6) + i * 16 * kSlice);
    };
    dev::f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int k = 0; k < FN; ++k) acc[i][k] = dev::f32x4{0, 0, 0, 0};

    load_w(code[0], word[0]);
    load_w(code[1], word[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        scales(word[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) put_w(2 * i, q, code[i]);
    }
    issue_x(1);
    load_w(code[0], word[0]);
    load_w(code[1], word[1]);
    __builtin_amdgcn_s_waitcnt(wait_for(0, 0));
    fence_barrier();
    if (second) fence_barrier();                              // half a period behind
    int u = 0, now = 0;                                       // place of the slice's weights, its number in the plane
    // slice j of even or odd number; ahead: four and more follow
    auto turns = [&](auto odd_, auto ahead_, int j) {
        constexpr int P = decltype(odd_)::value;
        constexpr bool AHEAD = decltype(ahead_)::value;
        const uint8_t *pb = place(u) + wn * TN * kSlice, *px = place(u + 1) + wm * TM * kSlice;
        const bool put = AHEAD || j + 2 < n, whole = !(odd && now + 1 == slices);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            bf16x8 fa[FM], fb[FN];
            read(px, half, fa);
            read(pb, half, fb);
            __builtin_amdgcn_sched_barrier(0);                // (the reads first: the decoding runs while they do)
            if (half == 0) scales(word[P]);
            if (put) {
                put_w(u + 4, half * 2, code[P]);
                put_w(u + 4, half * 2 + 1, code[P]);
            }
            if (half == 0 && (AHEAD || j + 1 < n)) issue_x(u + 3);      // (after the wait for the codes)
            if (half == 1 && AHEAD) load_w(code[P], word[P]);
            // x of slice j + 1 has landed at the end of the slice's last turn: a reading turn of the second
            // group, a computing turn of the first; the codes behind it may be in flight
            if (half == 1 && second) __builtin_amdgcn_s_waitcnt(wait_for(AHEAD ? 2 : 0, 0));
            else __builtin_amdgcn_s_waitcnt(wait_for(63, 0));
            fence_barrier();
            if (mine && (half == 0 || whole)) {
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int k = 0; k < FN; ++k) acc[i][k] = mma(fb[k], fa[i], acc[i][k]);
                __builtin_amdgcn_s_setprio(0);
            }
            if (half == 1 && !second) __builtin_amdgcn_s_waitcnt(wait_for(AHEAD ? 2 : 0, 15));
            fence_barrier();
        }
        if (++now == slices) now = 0;
        u = u + 2 >= kPlaces ? u + 2 - kPlaces : u + 2;
    };
    typedef std::integral_constant<int, 0> Even;
    typedef std::integral_constant<int, 1> Odd;
    int j = 0;
    for (; j + 5 < n; j += 2) {
        turns(Even{}, std::true_type{}, j);
        turns(Odd{}, std::true_type{}, j + 1);
    }
    // (the codes of the last four slices are in registers or LDS but for that of a fifth)
    if (j + 4 < n) {
        turns(Even{}, std::true_type{}, j);
        turns(Odd{}, std::false_type{}, j + 1);
        j += 2;
    }
    for (; j < n; j += 2) {
        turns(Even{}, std::false_type{}, j);
        if (j + 1 < n) turns(Odd{}, std::false_type{}, j + 1);
    }
    if (!second) fence_barrier();

    // results: 16 rows of the wave at a time through LDS, to come back as consecutive columns of a row
    uint8_t* st = lds + wave * (16 * kFinishRow);
    constexpr int W = KIND == kOut32 ? 4 : 8;
    constexpr int LPR = TN / (GATE ? 2 * W : W), RPP = kWave / LPR;
    const int lr = lane / LPR, lc = lane % LPR;
    const int col = GATE ? lc * W / 16 * 32 + lc * W % 16 : lc * W;
    const int nn = n0 + wn * TN + col;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        lanes_in_order();
#pragma unroll
        for (int k = 0; k < FN; ++k)
            *reinterpret_cast<dev::f32x4*>(st + (lane % 16) * kFinishRow + (lane / 16) * 16 + k * 64) = acc[i][k];
        lanes_in_order();
#pragma unroll
        for (int ps = 0; ps < 16 / RPP; ++ps) {
            const int rr = ps * RPP + lr, r = wm * TM + i * 16 + rr;
            if (r >= rows || nn >= p.N) continue;
            float v[W];
            const float* f = reinterpret_cast<const float*>(st + rr * kFinishRow) + col;
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = GATE ? gated(f[e], f[16 + e]) : f[e];
            const int64_t to = EXPERTS ? row_out<KIND>(p, shared, base, int(r0) + r) : r0 + r;
            if constexpr (KIND == kOut32) {
                float* o = static_cast<float*>(p.out) + to * p.ldo + nn;
                if (nn + W <= p.N) {
                    *reinterpret_cast<words4*>(o) = __builtin_bit_cast(dev::u32x4, dev::f32x4{v[0], v[1], v[2], v[3]});
                } else {
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (nn + e < p.N) o[e] = v[e];
                }
            } else {
                uint16_t* o = static_cast<uint16_t*>(p.out) + to * p.ldo + (GATE ? nn / 32 * 16 + nn % 16 : nn);
                if (EXPERTS || nn + W <= p.N) {
                    *reinterpret_cast<halves8*>(o) =
                        dev::u32x4{dev::pack_bf16x2(v[0], v[1]), dev::pack_bf16x2(v[2], v[3]), dev::pack_bf16x2(v[4], v[5]),
                                   dev::pack_bf16x2(v[6], v[7])};
                } else {
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (nn + e < p.N) o[e] = dev::f32_to_bf16_bits(v[e]);
                }
            }
        }
    }
}

// Lets a kernel use more than 64 KiB of LDS, once on each device.
hipError_t allow_lds(const void* kernel, std::atomic<uint64_t>& done) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <int KIND>
hipError_t launch_as(const Product& p, const ExpertList* list, const void* map, int64_t max_tiles, hipStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    const int64_t nt = (p.N + kB - 1) / kB, mt = list ? max_tiles : (p.T + kB - 1) / kB;
    const int64_t blocks = (nt * mt + kXcds - 1) / kXcds * kXcds;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0x7FFFFFFF / kThreads) return hipErrorInvalidValue;
    const auto kernel = &k_i4_turns<KIND>;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), allowed);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(unsigned(blocks)), dim3(kThreads), kLds, s, p, list_of<KIND>(list),
                       static_cast<const int4*>(map), int(nt), int(mt));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_i4_turns(int kind, const Product& p, const ExpertList* list, const void* map, int64_t max_tiles,
                           hipStream_t s) {
    if (p.T == 0) return hipSuccess;
    switch (kind) {
        case kOut16: return launch_as<kOut16>(p, nullptr, nullptr, 0, s);
        case kOut32: return launch_as<kOut32>(p, nullptr, nullptr, 0, s);
        case kGateUp: return launch_as<kGateUp>(p, list, map, max_tiles, s);
        default: return launch_as<kDown>(p, list, map, max_tiles, s);
    }
}

}  // namespace i4
}  // namespace moe
