// Products of 9 to some 128 rows of x with 4-bit weights, dense and by expert: a stream of codes that feeds
// 16x16x32 matrix instructions.
//
// A wave owns 32 rows of the weights and up to 128 of x.  Waves share the work two ways: WN of them have rows of
// their own and the same k, WK of them the same rows and slices of 64 k by turns.  With few rows of
// weights in all, a workgroup has 32 or 64 of them and its waves split K, so that the chip is full; with
// many, its waves have rows of their own and share x, which is what has to be read again for every run of rows:
// T K numbers for each 32 WN rows.
//
// Everything comes by loads straight into LDS, S slices ahead and counted by the wave itself: x as rows of 128
// bytes (16-byte chunk c of row r at slot c ^ ((r >> 1) & 7)), the codes as rows of 32 bytes, the groups'
// words one in four bytes.  A lane turns 16 codes of a weight row, one group, into two fragments of exact bf16
// weights, once for all rows of x.  Sums of the waves meet in LDS at the end, in a fixed order.
//
// Measured (bf16 x): 4096 x 4096 at 32 rows 8.4 us, at 128 11.2, at 512 27; 4096 x 12288 at 256 rows 50; 77 fp32 rows of 1568 to 1037
// 10.4 (75 walks of a slice: the codes are read and decoded once for each of the three parts of x).  What bounds them is the
// time of a slice with its wait and decoding, 0.9-1.5 us, not the matrix unit: a wave has 32 rows of the weights, so each fragment of
// x feeds two matrix instructions only; and K is not split over workgroups, so that with fewer tiles than CUs some are idle.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "dense.h"
#include "i4_common.h"

namespace moe {
namespace i4 {
namespace {

using dev::kWave;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((address_space(3))) void lds_void;
typedef uint32_t __attribute__((ext_vector_type(4), aligned(4))) words4;
typedef uint32_t __attribute__((ext_vector_type(2), aligned(2))) halves4;   // (odd rows of bf16 results lie on 2 bytes)

constexpr int kSlice = 128;                  // bytes of a row of x in a slice

__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }
constexpr int wait_for(int vm, int lgkm) { return (vm & 15) | (7 << 4) | (lgkm << 8) | ((vm >> 4) << 14); }

__device__ __forceinline__ dev::f32x4 mma(const bf16x8& a, const bf16x8& b, const dev::f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
constexpr uint32_t kRange = 0xFFFF0000u;     // of the buffer descriptors
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(kRange), 0x00027000);
}
// A lane's 16 bytes to its place of the wave's KiB; its two bytes into four of the wave's 256.  `at`: the lane's offset,
// `from`: the slice's.
__device__ __forceinline__ void load16_lds(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t at, uint32_t from) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, at, from, 0, 0);
}
__device__ __forceinline__ void load2_lds(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t at, uint32_t from) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 2, at, from, 0, 0);
}

template <int MF_, int WK_, int WN_, int S_>
struct Mid {
    static constexpr int MF = MF_, WK = WK_, WN = WN_, S = S_;
    static constexpr int NW = WK * WN, kThreads = NW * kWave, BM = MF * 16, BN = 32 * WN;
    static constexpr int X = BM * kSlice, W = 32 * 32, WORDS = 256;              // bytes of a slice
    static constexpr int kStage = WK * X + NW * (W + WORDS);
    static constexpr int XL = X / 1024 / WN;                                     // a wave's loads of x
    static constexpr int kPassRows = WK == 1 && BM > 32 ? 32 : BM, kRow = 36, kSums = NW * kPassRows * kRow * 4;   // staged sums
    static constexpr int kLds = S * kStage > kSums ? S * kStage : kSums;
    static_assert(XL * WN * 1024 == X && kLds <= 160 * 1024, "LDS of a CU");
    static constexpr int kWavesPerSimd = NW * (160 * 1024 / kLds) / 4 < 1 ? 1 : NW * (160 * 1024 / kLds) / 4 > 4 ? 4 : NW * (160 * 1024 / kLds) / 4;
};

// The tile of a workgroup: row tiles fastest, those of one run of weights are neighbours.
struct At {
    int64_t r0;              // first row of x, in the entry
    int n0, base, left;      // first row of the weights; first place of the entry; rows from r0 on
    bool shared, any;
    Rows w;
};
template <int KIND, class C>
__device__ __forceinline__ At tile_at(const Product& p, const ListOf<KIND>& list, const int4* map, int n_tiles, int m_tiles) {
    const int id = blockIdx.x;
    At at;
    at.w = p.w;
    at.base = 0;
    at.shared = false;
    at.any = true;
    if constexpr (KIND == kGateUp || KIND == kDown) {
        const int tiles = reinterpret_cast<const int*>(map)[0];
        at.any = id < tiles * n_tiles;
        if (!at.any) return at;
        const int4 rec = map[1 + id / n_tiles];
        at.n0 = id % n_tiles * C::BN;
        at.r0 = int64_t(rec.y) * C::BM;
        at.base = rec.z;
        at.left = rec.w - int(at.r0);
        const int ent = list.ent[rec.x];
        at.shared = (ent & 1023) == kSharedTag;
        at.w = rows_at(p.w, blob_offset(p, ent));
    } else {
        at.r0 = int64_t(id % m_tiles) * C::BM;
        at.n0 = id / m_tiles * C::BN;
        at.left = int(min(p.T - at.r0, int64_t(C::BM)));
    }
    return at;
}

// Sums of the waves, [wave][row of x][32 weight rows] in LDS, added in the waves' order, and finished.
template <int KIND, class C>
__device__ __forceinline__ void finish_sums(const Product& p, const dev::f32x4 (&acc)[C::MF][2], uint8_t* lds, int64_t r0, int n0,
                                            int base, bool shared, int rows) {
    constexpr bool EXPERTS = KIND == kGateUp || KIND == kDown, GATE = KIND == kGateUp;
    constexpr int MF = C::MF, WK = C::WK, WN = C::WN;
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, j = lane % 16, kb = lane / 16;
    __builtin_amdgcn_s_waitcnt(0);
    float* red = reinterpret_cast<float*>(lds);
    // (nothing to add where no waves share rows: then 32 rows at a time, which leaves LDS for a second workgroup)
    constexpr int PF = C::kPassRows / 16;
#pragma unroll
    for (int i0 = 0; i0 < MF; i0 += PF) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PF; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f)
                *reinterpret_cast<dev::f32x4*>(red + (wave * C::kPassRows + i * 16 + j) * C::kRow + f * 16 + kb * 4) = acc[i0 + i][f];
        __syncthreads();
        constexpr int PER = (GATE ? 4 : 8) * WN;                  // items of 4 results in a row of x
        const int left = min(rows - i0 * 16, C::kPassRows);
        for (int i = tid; i < left * PER; i += C::kThreads) {
            const int r = i0 * 16 + i / PER, c = i % PER, cw = c / (PER / WN), col = c % (PER / WN) * 4;
            auto sum = [&](int at) {
                const float* from = red + (cw * C::kPassRows + i / PER) * C::kRow + at;
                dev::f32x4 t = *reinterpret_cast<const dev::f32x4*>(from);
#pragma unroll
                for (int k = 1; k < WK; ++k) t += *reinterpret_cast<const dev::f32x4*>(from + k * WN * C::kPassRows * C::kRow);
                return t;
            };
            dev::f32x4 v = sum(col);
            const int nn = n0 + cw * 32 + col;
            if (nn >= p.N) continue;
            if constexpr (GATE) {
                const dev::f32x4 up = sum(col + 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = gated(v[e], up[e]);
            }
            const int64_t to = EXPERTS ? row_out<KIND>(p, shared, base, int(r0) + r) : r0 + r;
            if constexpr (KIND == kOut32) {
                float* o = static_cast<float*>(p.out) + to * p.ldo + nn;
                if (nn + 4 <= p.N) {
                    *reinterpret_cast<words4*>(o) = __builtin_bit_cast(dev::u32x4, v);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (nn + e < p.N) o[e] = v[e];
                }
            } else {
                uint16_t* o = static_cast<uint16_t*>(p.out) + to * p.ldo + (GATE ? nn / 32 * 16 + nn % 16 : nn);
                if (EXPERTS || nn + 4 <= p.N) {
                    *reinterpret_cast<halves4*>(o) = halves4{dev::pack_bf16x2(v[0], v[1]), dev::pack_bf16x2(v[2], v[3])};
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (nn + e < p.N) o[e] = dev::f32_to_bf16_bits(v[e]);
                }
            }
        }
    }
}

template <int KIND, int MF, int WK, int WN, int S>
__global__ void __launch_bounds__((Mid<MF, WK, WN, S>::kThreads))
    __attribute__((amdgpu_waves_per_eu((Mid<MF, WK, WN, S>::kWavesPerSimd))))
k_i4_mid(const Product p, const ListOf<KIND> list, const int4* __restrict__ map, int n_tiles, int m_tiles) {
    typedef Mid<MF, WK, WN, S> C;
    constexpr bool EXPERTS = KIND == kGateUp || KIND == kDown;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const At at = tile_at<KIND, C>(p, list, map, n_tiles, m_tiles);
    if (!at.any) return;
    const Rows& w = at.w;
    const int64_t r0 = at.r0;
    const int n0 = at.n0, base = at.base, rows = min(at.left, C::BM);
    const bool shared = at.shared;

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int wn = wave % WN, wk = wave / WN;
    const int j = lane % 16, kb = lane / 16;
    const int slices = (p.K + 63) / 64, n = (slices * p.planes + WK - 1) / WK;
    const bool odd = p.K % 64 != 0;
    // x: offsets of the lane's 16 bytes in row r of the tile.  Where K ends in the middle of a slice its second half is
    // the first again, with weights 0 (a token's own numbers: an infinity times 0 does no harm to another).
    uint32_t xo[C::XL];
    int64_t x0 = 0;                                           // (dense: offsets from the tile's first row)
    if (!EXPERTS) x0 = r0;
    else if (KIND == kDown) x0 = base + r0;
#pragma unroll
    for (int q = 0; q < C::XL; ++q) {
        const int r = (wn + WN * q) * 8 + lane / 8, rr = min(r, rows - 1);
        const int64_t from = KIND == kGateUp ? row_in<KIND>(p, shared, base, int(r0) + rr) : int64_t(rr);
        xo[q] = uint32_t(from * p.ldx * 2) + (lane % 8 ^ row_swz(r)) * 16;
    }
    const uint16_t* xp = p.x + x0 * p.ldx;
    const int nb = n0 + wn * 32;                              // the wave's first weight row
    const int first_row = min(nb, p.N - 1), row_l = min(nb + lane / 2, p.N - 1) - first_row;
    const uint32_t co = uint32_t(row_l) * uint32_t(p.K / 2) + lane % 2 * 16;
    const WordAt wa = word_at(first_row + row_l, p.N, w.groups);
    const uint32_t wo = uint32_t(wa.first - int64_t(first_row & ~15) * w.groups + (lane % 2 * 32 >> w.shift) * wa.step) * 2;
    const __amdgpu_buffer_rsrc_t rc = rsrc(w.codes + int64_t(first_row) * (p.K / 2)),
                                 rg = rsrc(w.words + int64_t(first_row & ~15) * w.groups);
    float E[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) E[f] = row_scale(w.exps[min(nb + f * 16 + j, p.N - 1)]);

    // LDS of a stage: x of the WK slices, then codes and words of each wave
    auto x_at = [&](int stage) { return lds + stage * C::kStage + wk * C::X; };
    auto w_at = [&](int stage) { return lds + stage * C::kStage + WK * C::X + wave * (C::W + C::WORDS); };
    int plane = p.planes - 1, slice = wk;                     // of the next request; smallest parts first
    auto settle = [&](int& slice, int& plane) {
        while (slice >= slices && plane > 0) slice -= slices, --plane;
    };
    settle(slice, plane);
    auto issue = [&](int stage) {
        // (past the end: the last slice again, with weights 0)
        const int s = min(slice, slices - 1);
        const __amdgpu_buffer_rsrc_t rx = rsrc(xp + plane * p.plane);
        uint8_t *dx = x_at(stage) + wn * 1024, *dw = w_at(stage);
        if (odd && s + 1 == slices) {
#pragma unroll
            for (int q = 0; q < C::XL; ++q) {
                const int c = lane % 8 ^ row_swz((wn + WN * q) * 8 + lane / 8);
                load16_lds(rx, dx + q * (WN * 1024), xo[q] - (c >= 4 ? 64 : 0), s * 128);
            }
            load16_lds(rc, dw, co - lane % 2 * 16, s * 32);
            load2_lds(rg, dw + C::W, wo + ((s * 64 >> w.shift) - (lane % 2 * 32 >> w.shift)) * wa.step * 2, 0);
        } else {
#pragma unroll
            for (int q = 0; q < C::XL; ++q) load16_lds(rx, dx + q * (WN * 1024), xo[q], s * 128);
            load16_lds(rc, dw, co, s * 32);
            load2_lds(rg, dw + C::W, wo + (s * 64 >> w.shift) * wa.step * 2, 0);
        }
        slice += WK;
        settle(slice, plane);
    };
    dev::f32x4 acc[MF][2];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int f = 0; f < 2; ++f) acc[i][f] = dev::f32x4{0, 0, 0, 0};

    constexpr int kLoads = C::XL + 2;
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s);
    int now = wk, now_plane = p.planes - 1, stage = 0, ahead = S - 1;
    for (int it = 0; it < n; ++it) {
        // this slice has landed, and every wave is past the one whose place the next request takes
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(wait_for((S - 2) * kLoads, 0));
        asm volatile("" ::: "memory");
        if constexpr (WN > 1) __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t *x = x_at(stage), *wl = w_at(stage);
        uint2 c[2];
        uint32_t word[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int r = f * 16 + j;
            c[f] = *reinterpret_cast<const uint2*>(wl + r * 32 + kb * 8);
            word[f] = *reinterpret_cast<const uint32_t*>(wl + C::W + (r * 2 + kb / 2) * 4);
        }
        // k of instruction q in lane block kb: 16 kb + 8 q on, chunk 2 kb + q
        auto read_x = [&](int i, int q) {
            return *reinterpret_cast<const bf16x8*>(x + (i * 16 + j) * kSlice + ((2 * kb + q) ^ row_swz(j)) * 16);
        };
        constexpr int EARLY = MF < 4 ? MF : 4;                // fragments read ahead of the decoding
        bf16x8 fa[EARLY][2];
#pragma unroll
        for (int i = 0; i < EARLY; ++i) fa[i][0] = read_x(i, 0), fa[i][1] = read_x(i, 1);
        __builtin_amdgcn_sched_barrier(0);
        issue(ahead);
        settle(now, now_plane);
        const uint32_t live = now >= slices ? 0u : odd && now + 1 == slices && kb >= 2 ? 0u : ~0u;
        bf16x8 fb[2][2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const uint32_t wd = word[f] & live;               // (0: scale 0)
            const float s = word_scale(wd) * E[f], off = -word_zero(wd) * s, s2 = s * 512.0f;
            fb[f][0] = __builtin_bit_cast(bf16x8, decode8(c[f].x, s2, off));
            fb[f][1] = __builtin_bit_cast(bf16x8, decode8(c[f].y, s2, off));
        }
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const bf16x8 a = i < EARLY ? fa[i < EARLY ? i : 0][q] : read_x(i, q);
#pragma unroll
                for (int f = 0; f < 2; ++f) acc[i][f] = mma(fb[f][q], a, acc[i][f]);
            }
        now += WK;
        stage = stage + 1 == S ? 0 : stage + 1;
        ahead = ahead + 1 == S ? 0 : ahead + 1;
    }

    finish_sums<KIND, C>(p, acc, lds, at.r0, at.n0, at.base, at.shared, rows);
}

// The same with whole lines of codes in registers: a wave's 32 rows by blocks of 128 k, 16 bytes a lane and 16 rows, so
// that the 32 codes of a lane share a group, D blocks ahead; x alone goes through LDS, in D + 1 stages.  Half the
// waits, words and addresses for a code: for products whose time is the decoding, many rows of weights or many experts.
// Measured: 100003 x 4096 at 32 rows 71 us, at 64 92, at 128 147 (two workgroups read 256 KB of LDS a block, 2,048 cycles, as many as
// their matrix instructions take, and the decoding comes on top); 128 experts of 2048 x 768, top 8, at 16 tokens 36 and 21 (166 MB at
// 2.9 TB/s), at 64 tokens 86 in all, at 256 94, at 2,048 291.
template <int MF_, int D_>
struct Wide {
    static constexpr int MF = MF_, WK = 1, WN = 4, D = D_;
    static constexpr int NW = WN, kThreads = NW * kWave, BM = MF * 16, BN = 32 * WN;
    static constexpr int kStage = BM * 256;
    static constexpr int XL = kStage / 1024 / WN;
    static constexpr int kPassRows = BM > 32 ? 32 : BM, kRow = 36, kSums = NW * kPassRows * kRow * 4;
    static constexpr int kLds = (D + 1) * kStage > kSums ? (D + 1) * kStage : kSums;
    static_assert(XL * WN * 1024 == kStage && (D == 1 || D == 2), "loads of a stage, registers of a block");
    static constexpr int kPerCu = 160 * 1024 / kLds < 1 ? 1 : 160 * 1024 / kLds;
    static constexpr int kWavesPerSimd = NW * kPerCu / 4 < 1 ? 1 : NW * kPerCu / 4 > 4 ? 4 : NW * kPerCu / 4;
};
constexpr uint32_t kOutside = 0xFFFFFFF0u;   // an offset past kRange: zeros, also into LDS

template <int KIND, int MF, int D>
__global__ void __launch_bounds__((Wide<MF, D>::kThreads)) __attribute__((amdgpu_waves_per_eu((Wide<MF, D>::kWavesPerSimd))))
k_i4_wide(const Product p, const ListOf<KIND> list, const int4* __restrict__ map, int n_tiles, int m_tiles) {
    typedef Wide<MF, D> C;
    constexpr int WN = C::WN;
    constexpr bool EXPERTS = KIND == kGateUp || KIND == kDown;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const At at = tile_at<KIND, C>(p, list, map, n_tiles, m_tiles);
    if (!at.any) return;
    const int rows = min(at.left, C::BM);
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
    const int wn = wave, j = lane % 16, kb = lane / 16;
    const int blocks = (p.K + 127) / 128, n = blocks * p.planes;

    // x: 16 lanes a row of 256 bytes, 4 rows a load; 16-byte chunk c of row r at slot c ^ (r % 16)
    uint32_t xo[C::XL];
    int64_t x0 = 0;
    if (!EXPERTS) x0 = at.r0;
    else if (KIND == kDown) x0 = at.base + at.r0;
#pragma unroll
    for (int q = 0; q < C::XL; ++q) {
        const int r = (wn + WN * q) * 4 + lane / 16, rr = min(r, rows - 1);
        const int64_t from = KIND == kGateUp ? row_in<KIND>(p, at.shared, at.base, int(at.r0) + rr) : int64_t(rr);
        xo[q] = uint32_t(from * p.ldx * 2);
    }
    const uint16_t* xp = p.x + x0 * p.ldx;
    const int nb = at.n0 + wn * 32, first_row = min(nb, p.N - 1);
    const __amdgpu_buffer_rsrc_t rc = rsrc(at.w.codes + int64_t(first_row) * (p.K / 2)),
                                 rg = rsrc(at.w.words + int64_t(first_row & ~15) * at.w.groups);
    uint32_t co[2], wo[2];
    int step[2];
    float E[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const int row = min(nb + f * 16 + j, p.N - 1);
        co[f] = uint32_t(row - first_row) * uint32_t(p.K / 2) + kb * 16;
        const WordAt wa = word_at(row, p.N, at.w.groups);
        wo[f] = uint32_t(wa.first - int64_t(first_row & ~15) * at.w.groups + (kb * 32 >> at.w.shift) * wa.step) * 2;
        step[f] = __builtin_amdgcn_readfirstlane(wa.step * 2);      // (one run of 16 rows: one step)
        E[f] = row_scale(at.w.exps[row]);
    }
    int x_plane = p.planes - 1, x_block = 0, w_block = 0, w_plane = p.planes - 1;
    auto settle = [&](int& block, int& plane) {
        if (block >= blocks && plane > 0) block -= blocks, --plane;
    };
    auto issue_x = [&](int stage) {
        const __amdgpu_buffer_rsrc_t rx = rsrc(xp + x_plane * p.plane);
        uint8_t* d = lds + stage * C::kStage + wn * 1024;
#pragma unroll
        for (int q = 0; q < C::XL; ++q) {
            const int r = (wn + WN * q) * 4 + lane / 16, c = lane % 16 ^ (r % 16);
            load16_lds(rx, d + q * (WN * 1024), x_block * 128 + c * 8 < p.K ? xo[q] + c * 16 : kOutside, x_block * 256);
        }
        ++x_block;
        settle(x_block, x_plane);
    };
    dev::u32x4 code[D][2];
    uint16_t word[D][2];
    auto load_w = [&](dev::u32x4 (&c)[2], uint16_t (&g)[2]) {
        const bool in = w_block * 128 + kb * 32 < p.K;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            c[f] = __builtin_bit_cast(dev::u32x4, __builtin_amdgcn_raw_buffer_load_b128(rc, in ? co[f] : kOutside, w_block * 64, 0));
            g[f] = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(rg, in ? wo[f] : kOutside, (w_block * 128 >> at.w.shift) * step[f], 0));
        }
        ++w_block;
        settle(w_block, w_plane);
    };
    dev::f32x4 acc[MF][2];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int f = 0; f < 2; ++f) acc[i][f] = dev::f32x4{0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < D; ++d) {
        issue_x(d);
        asm volatile("" ::: "memory");
        load_w(code[d], word[d]);
        asm volatile("" ::: "memory");
    }
    int stage = 0, ahead = D;
    auto block = [&](auto slot_) {
        constexpr int slot = decltype(slot_)::value;
        // this block has landed, and every wave is past the one whose place the next request takes
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(wait_for((D - 1) * (C::XL + 4), 0));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        issue_x(ahead);
        const uint8_t* x = lds + stage * C::kStage;
        float s2[2], off[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const float s = word_scale(word[slot][f]) * E[f];
            off[f] = -word_zero(word[slot][f]) * s;
            s2[f] = s * 512.0f;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // k of instruction q in lane block kb: 32 kb + 8 q on
            bf16x8 fa[MF], fb[2];
#pragma unroll
            for (int i = 0; i < MF; ++i)
                fa[i] = *reinterpret_cast<const bf16x8*>(x + (i * 16 + j) * 256 + ((4 * kb + q) ^ j) * 16);
#pragma unroll
            for (int f = 0; f < 2; ++f) fb[f] = __builtin_bit_cast(bf16x8, decode8(code[slot][f][q], s2[f], off[f]));
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int f = 0; f < 2; ++f) acc[i][f] = mma(fb[f], fa[i], acc[i][f]);
        }
        asm volatile("" ::: "memory");
        load_w(code[slot], word[slot]);
        stage = stage == D ? 0 : stage + 1;
        ahead = ahead == D ? 0 : ahead + 1;
    };
    // (past the end blocks are zeros)
    for (int it = 0; it < n; it += D) {
        block(std::integral_constant<int, 0>{});
        if constexpr (D > 1) block(std::integral_constant<int, 1>{});
    }
    finish_sums<KIND, C>(p, acc, lds, at.r0, at.n0, at.base, at.shared, rows);
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
    for (int w = 0; w < int(blockDim.x) / kWave; ++w) {
        if (w < wave) first += s_sum[w];
        total += s_sum[w];
    }
    for (int i = 0; i < tiles; ++i) map[1 + first + i] = make_int4(tid, i, base, count);
    if (tid == 0) reinterpret_cast<int*>(map)[0] = total;
}

hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <int KIND, class C, class F>
hipError_t launch_as(F kernel, const Product& p, const ExpertList* list, const void* map, int64_t max_tiles, hipStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    const int64_t nt = (p.N + C::BN - 1) / C::BN, mt = list ? max_tiles : (p.T + C::BM - 1) / C::BM, blocks = nt * mt;
    if (blocks == 0) return hipSuccess;
    if (blocks > 0x7FFFFFFF / C::kThreads) return hipErrorInvalidValue;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), C::kLds, allowed);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(unsigned(blocks)), dim3(C::kThreads), C::kLds, s, p, list_of<KIND>(list),
                       static_cast<const int4*>(map), int(nt), int(mt));
    return hipGetLastError();
}
template <int KIND, int MF, int WK, int WN, int S>
hipError_t mid(const Product& p, const ExpertList* list, const void* map, int64_t max_tiles, hipStream_t s) {
    return launch_as<KIND, Mid<MF, WK, WN, S>>(&k_i4_mid<KIND, MF, WK, WN, S>, p, list, map, max_tiles, s);
}
template <int KIND, int MF, int D>
hipError_t wide(const Product& p, const ExpertList* list, const void* map, int64_t max_tiles, hipStream_t s) {
    return launch_as<KIND, Wide<MF, D>>(&k_i4_wide<KIND, MF, D>, p, list, map, max_tiles, s);
}

template <int KIND>
hipError_t choose(int kind, const Product& p, const ExpertList* list, const void* map, int64_t max_tiles, hipStream_t s) {
    switch (kind) {
        case kMid32x32: return mid<KIND, 2, 8, 1, 3>(p, list, map, max_tiles, s);
        case kMid64x32: return mid<KIND, 4, 8, 1, 2>(p, list, map, max_tiles, s);
        case kMid128x32: return mid<KIND, 8, 4, 1, 2>(p, list, map, max_tiles, s);
        case kMid64x64: return mid<KIND, 4, 4, 2, 3>(p, list, map, max_tiles, s);
        case kMid128x64: return mid<KIND, 8, 4, 2, 2>(p, list, map, max_tiles, s);
        case kMid32x128: return wide<KIND, 2, 2>(p, list, map, max_tiles, s);
        case kMid64x128: return wide<KIND, 4, 2>(p, list, map, max_tiles, s);
        case kMid128x128: return wide<KIND, 8, 1>(p, list, map, max_tiles, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_i4_map(const ExpertList& list, const int32_t* offsets, int64_t T, int top_k, int rows, void* map,
                         hipStream_t s) {
    hipLaunchKernelGGL(k_i4_map, dim3(1), dim3((list.n + kWave - 1) / kWave * kWave), 0, s, list, offsets, int(T), top_k, rows, static_cast<int4*>(map));
    return hipGetLastError();
}

hipError_t launch_i4_mid(int what, int kind, const Product& p, const ExpertList* list, const void* map, int64_t max_tiles,
                         hipStream_t s) {
    if (p.T == 0) return hipSuccess;
    switch (what) {
        case kOut16: return choose<kOut16>(kind, p, nullptr, nullptr, 0, s);
        case kOut32: return choose<kOut32>(kind, p, nullptr, nullptr, 0, s);
        case kGateUp: return choose<kGateUp>(kind, p, list, map, max_tiles, s);
        default: return choose<kDown>(kind, p, list, map, max_tiles, s);
    }
}

}  // namespace i4
}  // namespace moe
