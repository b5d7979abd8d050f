// Products with 4-bit weights in tiles on the matrix cores, dense and by expert.
//
// A workgroup of four waves owns 64 or 128 rows of x and 128 of the weights and walks K in slices of 64.
// The rows of x are loaded straight into LDS (rows of 128 bytes, 16-byte chunk c of row r at slot
// c ^ ((r >> 1) & 7), so the 16 rows of a fragment read fall on different banks).  The weights come as
// codes, one 16-byte load a thread and slice, a slice ahead; a thread turns its 32 codes, which share a
// group, into 32 exact bf16 weights and writes them into LDS the same way, so each code is decoded once
// in a workgroup.  fp32 activations are three bf16 parts, walked one after the
// other, the smallest first: sums stay small, and their roundings, until the last.
//
// Experts: records of the tile map (k_i4_map) name an entry of the list and its rows; rows of x are
// gathered by the pairs' tokens, results scattered to the pairs.
#include <hip/hip_runtime.h>

#include "i4_common.h"

namespace moe {
namespace i4 {
namespace {

using dev::kWave;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;
typedef uint32_t __attribute__((ext_vector_type(4), aligned(4))) words4;

constexpr int kXcds = 8, kSlice = 128, kBN = 128, kThreads = 256;

__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ dev::f32x4 mma(const bf16x8& a, const bf16x8& b, const dev::f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Between LDS writes and reads of one wave's lanes: the LDS takes them in order, the compiler has to.
__device__ __forceinline__ void lanes_in_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

template <int KIND, int BM>
__global__ void __launch_bounds__(kThreads) k_i4_tile(const Product p, const ExpertList list, const int4* __restrict__ map,
                                                      int n_tiles, int m_tiles) {
    constexpr bool EXPERTS = KIND == kGateUp || KIND == kDown;
    constexpr int WM = BM / 64, WN = 4 / WM, TN = kBN / WN, FM = 4, FN = TN / 16;      // waves: WM x WN of 64 x TN
    constexpr int STAGE = (BM + kBN) * kSlice;
    constexpr int A_LOADS = BM / 32;                                                  // 1 KiB loads of a wave a slice
    constexpr int FROW = TN * 4 + 16;                                                 // staged rows of sums
    static_assert(4 * 16 * FROW <= 2 * STAGE, "room for the results");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];

    // tile: workgroup b serves XCD b % 8, each XCD a contiguous run of the order, row tiles fastest
    const int total = (EXPERTS ? reinterpret_cast<const int*>(map)[0] : m_tiles) * n_tiles;
    const int per = (total + kXcds - 1) / kXcds, lid = int(blockIdx.x) % kXcds * per + int(blockIdx.x) / kXcds;
    if (int(blockIdx.x) / kXcds >= per || lid >= total) return;
    int mt, n0, base = 0, left;
    bool shared = false;
    Rows w = p.w;
    if constexpr (EXPERTS) {
        // (the row tiles of an entry are neighbours in the map: columns slower inside an entry would
        // need its extent; the map's order with columns slowest of all reads x of an entry once an XCD)
        const int4 rec = map[1 + lid / n_tiles];
        mt = rec.y;
        n0 = lid % n_tiles * kBN;
        base = rec.z;
        left = rec.w - mt * BM;
        const int ent = list.ent[rec.x];
        shared = (ent & 1023) == kSharedTag;
        w = rows_at(p.w, blob_offset(p, ent));
    } else {
        mt = lid % m_tiles;
        n0 = lid / m_tiles * kBN;
        const int64_t l = p.T - int64_t(mt) * BM;
        left = l < BM ? int(l) : BM;
    }
    const int rows = left < BM ? left : BM;
    const int64_t r0 = int64_t(mt) * BM;

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int wm = wave / WN, wn = wave % WN;
    // rows of x: load q of the wave is 8 rows of the tile
    const uint16_t* xa[A_LOADS];
#pragma unroll
    for (int q = 0; q < A_LOADS; ++q) {
        const int r = (wave + 4 * q) * 8 + lane / 8, c = lane % 8 ^ row_swz(r);
        const int64_t from = EXPERTS ? row_in<KIND>(p, shared, base, int(r0) + min(r, rows - 1)) : r0 + min(r, rows - 1);
        xa[q] = p.x + from * p.ldx + c * 8;
    }
    const int half = tid % 2, br = tid / 2;
    const int64_t n = min(n0 + br, p.N - 1);
    const uint8_t* codes = w.codes + n * (p.K / 2) + half * 16;
    const uint16_t* words = w.words + n * w.groups;
    const float S = row_scale(w.exps[n]);
    uint8_t* const b_row = lds + BM * kSlice + br * kSlice;

    const int slices = (p.K + 63) / 64, nk = slices * p.planes;
    uint4 code = make_uint4(0, 0, 0, 0);
    uint32_t word = 0;
    auto load_codes = [&](int s) {
        const int k = s * 64 + half * 32;
        if (k < p.K) {
            code = *reinterpret_cast<const uint4*>(codes + s * 32);
            word = words[k >> w.shift];
        }
    };
    auto put_codes = [&](int stage) {
        const float s = word_scale(word) * S, off = -word_zero(word) * s, s2 = s * 512.0f;
        uint8_t* d = b_row + stage * STAGE;
        const uint32_t c[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<dev::u32x4*>(d + ((half * 4 + q) ^ row_swz(br)) * 16) = decode8(c[q], s2, off);
    };
    auto load_x = [&](int plane, int s, int stage) {
        const int64_t o = (p.planes - 1 - plane) * p.plane + s * 64;     // smallest parts first
        uint8_t* d = lds + stage * STAGE;
#pragma unroll
        for (int q = 0; q < A_LOADS; ++q) {
            const int r = (wave + 4 * q) * 8 + lane / 8;
            if (s * 64 + (lane % 8 ^ row_swz(r)) * 8 < p.K)       // (the second half of the last slice may lie past K)
                __builtin_amdgcn_global_load_lds((global_void*)(xa[q] + o), (lds_void*)(d + (wave + 4 * q) * 1024), 16, 0, 0);
        }
    };
    dev::f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = dev::f32x4{0, 0, 0, 0};

    int plane = 0, s = 0;                                         // of the slice after the current one
    load_codes(0);
    load_x(0, 0, 0);
    put_codes(0);
    auto advance = [&]() {
        if (++s == slices) s = 0, ++plane;
    };
    int now = 0;                                                  // slice in its plane
    advance();
    if (nk > 1) load_codes(s);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int it = 0; it < nk; ++it) {
        const int stage = it & 1;
        const bool more = it + 1 < nk;
        if (more) load_x(plane, s, stage ^ 1);
        const uint8_t* a = lds + stage * STAGE + wm * 64 * kSlice;
        const uint8_t* b = lds + stage * STAGE + (BM + wn * TN) * kSlice;
        const int row = lane % 16, g = lane / 16;
        const int halves = now * 64 + 32 < p.K ? 2 : 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h < halves) {
                bf16x8 fa[FM], fb[FN];
                const int at = ((h * 4 + g) ^ row_swz(row)) * 16 + row * kSlice;
#pragma unroll
                for (int i = 0; i < FM; ++i) fa[i] = *reinterpret_cast<const bf16x8*>(a + i * 16 * kSlice + at);
#pragma unroll
                for (int j = 0; j < FN; ++j) fb[j] = *reinterpret_cast<const bf16x8*>(b + j * 16 * kSlice + at);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) acc[i][j] = mma(fb[j], fa[i], acc[i][j]);
            }
        }
        if (more) {
            put_codes(stage ^ 1);
            now = s;
            advance();
            if (it + 2 < nk) load_codes(s);
        }
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
    }

    // results: 16 rows of the wave at a time through LDS, to come back as consecutive columns of a row
    uint8_t* st = lds + wave * (16 * FROW);
    constexpr bool GATE = KIND == kGateUp;
    constexpr int W = KIND == kOut32 ? 4 : 8;                     // results a lane
    constexpr int LPR = TN / (GATE ? 2 * W : W), RPP = kWave / LPR < 16 ? kWave / LPR : 16;
    const int lr = lane / LPR, lc = lane % LPR;
    const int col = GATE ? lc * W / 16 * 32 + lc * W % 16 : lc * W;
    const int nn = n0 + wn * TN + col;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        lanes_in_order();
#pragma unroll
        for (int j = 0; j < FN; ++j)
            *reinterpret_cast<dev::f32x4*>(st + (lane % 16) * FROW + (lane / 16) * 16 + j * 64) = acc[i][j];
        lanes_in_order();
#pragma unroll
        for (int ps = 0; ps < 16 / RPP; ++ps) {
            const int rr = ps * RPP + lr % RPP, r = wm * 64 + i * 16 + rr;
            if (lr >= RPP || r >= rows || nn >= p.N) continue;
            float v[W];
            const float* f = reinterpret_cast<const float*>(st + rr * FROW) + col;
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = GATE ? gated(f[e], f[16 + e]) : f[e];
            const int64_t to = EXPERTS ? row_out<KIND>(p, shared, base, int(r0) + r) : r0 + r;
            if constexpr (KIND == kOut32) {
                float* o = static_cast<float*>(p.out) + to * p.ldo + nn;
                if (nn + W <= p.N) {
                    *reinterpret_cast<words4*>(o) =
                        __builtin_bit_cast(dev::u32x4, dev::f32x4{v[0], v[1], v[2], v[3]});
                } else {
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (nn + e < p.N) o[e] = v[e];
                }
            } else {
                uint16_t* o = static_cast<uint16_t*>(p.out) + to * p.ldo + (GATE ? nn / 32 * 16 + nn % 16 : nn);
                if (EXPERTS || (p.wide && nn + W <= p.N)) {
                    *reinterpret_cast<words4*>(o) =
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

// The tile map: one workgroup, one thread an entry (513 at most).
__global__ __launch_bounds__(1024) void k_i4_map(const ExpertList list, const int32_t* __restrict__ offsets, int T, int top_k,
                                                 int tile, int4* __restrict__ map) {
    __shared__ int s_sum[16];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    int count = 0, base = 0;
    if (tid < list.n) {
        const int e = list.ent[tid] & 1023;
        base = e == kSharedTag ? T * top_k : offsets[e];
        count = e == kSharedTag ? T : offsets[e + 1] - base;
    }
    const int tiles = (count + tile - 1) / tile;
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += o;
    }
    if (lane == kWave - 1) s_sum[wave] = incl;
    __syncthreads();
    int first = incl - tiles, total = 0;
    for (int w = 0; w < 16; ++w) {
        if (w < wave) first += s_sum[w];
        total += s_sum[w];
    }
    for (int i = 0; i < tiles; ++i) map[1 + first + i] = make_int4(tid, i, base, count);
    if (tid == 0) reinterpret_cast<int*>(map)[0] = total;
}

template <int KIND, int BM>
hipError_t launch_as(const Product& p, const ExpertList* list, const void* map, int64_t max_tiles, hipStream_t s) {
    static const ExpertList none{};
    const int64_t nt = (p.N + kBN - 1) / kBN, mt = list ? max_tiles : (p.T + BM - 1) / BM;
    const int64_t blocks = (nt * mt + kXcds - 1) / kXcds * kXcds;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0x7FFFFFFF / kThreads) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_i4_tile<KIND, BM>), dim3(unsigned(blocks)), dim3(kThreads), 0, s, p, list ? *list : none,
                       static_cast<const int4*>(map), int(nt), int(mt));
    return hipGetLastError();
}

}  // namespace

int64_t map_tiles(int n, int64_t rows, int tile) { return rows / tile + n; }

hipError_t launch_i4_map(const ExpertList& list, const int32_t* offsets, int64_t T, int top_k, int rows, void* map,
                         hipStream_t s) {
    hipLaunchKernelGGL(k_i4_map, dim3(1), dim3(1024), 0, s, list, offsets, int(T), top_k, rows, static_cast<int4*>(map));
    return hipGetLastError();
}

hipError_t launch_i4_tiles(int kind, const Product& p, const ExpertList* list, const void* map, int64_t max_tiles,
                           hipStream_t s) {
    if (p.T == 0) return hipSuccess;
    switch (kind) {
        case kOut16: return launch_as<kOut16, kTileRows>(p, nullptr, nullptr, 0, s);
        case kOut32: return launch_as<kOut32, kTileRows>(p, nullptr, nullptr, 0, s);
        case kGateUp: return launch_as<kGateUp, kTileRows>(p, list, map, max_tiles, s);
        default: return launch_as<kDown, kTileRows>(p, list, map, max_tiles, s);
    }
}

}  // namespace i4
}  // namespace moe
