// Products of the dense operators on the matrix cores: fp32, bf16 and 8-bit integers.
//
// C[m][n] = sum_k A(m, k) B(n, k) in tiles of BM x BN.  One K slice is 128 bytes of K (32 fp32,
// 64 bf16 or 128 codes), so a row segment of an operand that is contiguous along K is one cache
// line and all types move the same bytes per slice; a fragment is 16 bytes a lane from each
// operand: one 16x16 matrix instruction for bf16 (32 k) and for codes (64 k) in the same time,
// four for fp32 (4 k each; which k an instruction takes does not matter while both operands
// agree), eight times as long.  Slices are loaded straight into LDS by buffer loads.
//
// Two kernels: k_mma_turns on 256 x 256 tiles, k_mma on 128 x 128 and 64 x 64 ones, where larger
// tiles would leave CUs idle; with few of those, K is split over workgroups and k_join adds the
// parts.  Measured (8,192 tokens through the 4096 x 12288 block, kernel times at their least, cards
// differ by up to 7%): bf16 down 0.55 ms, 1.50 PFLOP/s, the matrix units busy 79% of the cycles at
// 1.8 GHz, where power holds the clock; gate and up 1.20 ms, 1.38 PFLOP/s, 70%; dx 1.12 ms, 1.47
// PFLOP/s, 76%; both weights' gradients 1.82 ms, 1.36 PFLOP/s, 67%; dg and du 0.73 ms, 1.13
// PFLOP/s, 56% (1 GB of pre-activations read and results written when all CUs end a tile together).
// In 8 bits down 280 us, 2.95 POP/s, gate and up 666 us, 2.48 POP/s.  A library product of 8192^3
// reaches 1.45 PFLOP/s and 2.36 POP/s on the same card.
//
// Operands contiguous along K lie in LDS as rows of 128 bytes, 16-byte chunk c of row r at slot
// c ^ ((r >> 1) & 7): two rows share a 256-byte window of the banks, so the 16 rows of a
// fragment read fall on different banks.  Operands contiguous along the other dimension (the
// gradients' products) lie as rows of one k; their fragments are read with the transposing LDS
// read, 4 k of 16 columns a group of 16 lanes, and the 32-byte units of row k are permuted by
// bits 0, 1 and 3 of k, so the 8 rows that 32 lanes read fall on different banks.  fp32 reads them
// 4 bytes a lane instead, 16 columns of one k a group of 16 lanes, 64-byte units permuted by
// bits 2 and 3 of k.
//
// The weights' operand goes first into the instruction, so a lane ends with four consecutive
// columns of one row, and gate and up sums of an inner index are in one lane.
//
// Rows past M or N are read from the last row (their sums are dropped), and the part of the last
// slice past K is zeros: a buffer load whose offset is out of range writes zeros to LDS.
//
// Workgroup b serves XCD b % 8; each XCD takes a contiguous run of the tile order, which walks
// groups of 8 row tiles, so the tiles in flight on an XCD share operands in its L2.
#include <hip/hip_runtime.h>

#include <atomic>
#include <type_traits>

#include "dense_common.h"
#include "dense_epilogue.h"

namespace moe {
namespace dense {
namespace {

using dev::kWave;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kXcds = 8, kGroupM = 8;
constexpr int kSlice = kSliceBytes;
constexpr uint32_t kOutside = 0xFFFFFFF0u;        // a buffer offset past every range
constexpr uint32_t kRange = 0x80000000u;          // range of the buffer descriptors: 2 GiB

template <int TYPE> struct Frag;
template <> struct Frag<kBF16> {
    typedef bf16x8 V;
    typedef dev::f32x4 Acc;
    static constexpr int ES = 2;
};
template <> struct Frag<kI8> {
    typedef i32x4 V;
    typedef i32x4 Acc;
    static constexpr int ES = 1;
};
template <> struct Frag<kF32> {
    typedef dev::f32x4 V;
    typedef dev::f32x4 Acc;
    static constexpr int ES = 4;
};
__device__ __forceinline__ dev::f32x4 mma(const dev::f32x4& a, const dev::f32x4& b, dev::f32x4 c) {
#pragma unroll
    for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[q], b[q], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ dev::f32x4 mma(const bf16x8& a, const bf16x8& b, const dev::f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mma(const i32x4& a, const i32x4& b, const i32x4& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// permutation (of 16-byte chunks, by whole 32-byte units) of row k of an operand that is not
// contiguous along K: rows of 256 bytes and more all start on the same bank and have 8 units to
// permute; rows of 128 bytes (X = 64) alternate between the halves of the banks and have 4.
// fp32: by 64-byte units.
template <int X, int ES>
__device__ __forceinline__ int chunk_swz(int k) {
    if (ES == 4) return ((k >> 2) & 3) << 2;
    return (X == 64 ? ((k >> 1) & 1) | ((k >> 2) & 2) : (k & 3) | ((k >> 1) & 4)) << 1;
}

// permutation of the chunks of row r of an operand that is contiguous along K: rows of 128 bytes
// share the 256 bytes of the banks by two
__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }

// A wave's loads of a slice of one operand into LDS (256 rows, 8 waves): four times 1 KiB, 8 KiB
// apart.
struct SliceLoads {
    uint32_t lds;
    i32x4 rsrc;
    uint32_t off[4];
};

// One operand's tile: X rows (tokens or weights) by one slice of K, X * 128 bytes in LDS.
// KC: contiguous along K.
template <int X, bool KC, int ES, int NW>
struct Side {
    static constexpr int Q = X * kSlice / 1024 / NW;          // 1 KiB loads of a wave per slice
    static constexpr int KS = kSlice / ES;                    // k in a slice
    static constexpr int CPS = kSlice / 16;                   // 16-byte chunks of a row's slice
    static_assert(Q * NW * 1024 == X * kSlice, "loads split over the waves");
    static_assert(KC || ES >= 2, "transposing reads: 16-bit elements; fp32 reads single values");

    const uint8_t* base;     // (uniform) first row / column of the tile at the next slice to load
    int64_t step;            // bytes from slice to slice
    uint32_t off[Q];         // this lane's offsets from base

    // x0: the tile's first row, n_rows rows in all; ld elements between rows (KC) or between k;
    // first: the first slice to load
    __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t x0, int64_t n_rows, int first) {
        const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
        const uint32_t ldb = uint32_t(ld) * ES;
        base = static_cast<const uint8_t*>(p) + (KC ? x0 * ld * ES : x0 * ES);
        step = KC ? kSlice : int64_t(KS) * ld * ES;
        base += first * step;
        const int left = int(n_rows - x0 < X ? n_rows - x0 : X);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int i = wave + NW * q;                  // 1 KiB block of the tile
            if constexpr (KC) {
                const int r = (i * 64 + lane) / CPS, c = lane % CPS ^ row_swz(r);
                off[q] = uint32_t(r < left ? r : left - 1) * ldb + c * 16;
            } else {
                constexpr int CPR = X * ES / 16;          // 16-byte chunks of a k row
                const int k = (i * 64 + lane) / CPR, c = (i * 64 + lane) % CPR;
                const int col = (c ^ chunk_swz<X, ES>(k)) * (16 / ES);
                off[q] = uint32_t(k) * ldb + (col < left ? col : 0) * ES;
            }
        }
    }
    // the loads of the next slice for an assembly block; their offsets once k_left k are left
    __device__ __forceinline__ SliceLoads next(uint8_t* lds) {
        static_assert(Q == 4 && NW == 8, "as SliceLoads has them");
        const uint64_t b = reinterpret_cast<uint64_t>(base);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        SliceLoads l{uint32_t(reinterpret_cast<uintptr_t>((lds_void*)lds)) + wave * 1024,
                     i32x4{int(b), int(b >> 32) & 0xFFFF, int(kRange), 0x00027000},
                     {off[0], off[1], off[2], off[3]}};
        base += step;
        return l;
    }
    __device__ __forceinline__ void end_of_k(int k_left) {
#pragma unroll
        for (int q = 0; q < Q; ++q) off[q] = k_left > 0 ? tail(q, k_left) : kOutside;
    }
    // offset of load q when only k_left k of the slice exist
    __device__ __forceinline__ uint32_t tail(int q, int k_left) const {
        const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, i = wave + NW * q;
        bool in;
        if constexpr (KC) {
            const int r = (i * 64 + lane) / CPS, c = lane % CPS ^ row_swz(r);
            in = c * (16 / ES) < k_left;
        } else {
            in = (i * 64 + lane) / (X * ES / 16) < k_left;
        }
        return in ? off[q] : kOutside;
    }
    __device__ __forceinline__ void issue(uint8_t* lds, int k_left) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, kRange, 0x00027000);
        auto load = [&](int q, uint32_t o) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + (wave + NW * q) * 1024), 16, o, 0, 0, 0);
        };
        if (k_left >= KS) {
#pragma unroll
            for (int q = 0; q < Q; ++q) load(q, off[q]);
        } else {
#pragma unroll
            for (int q = 0; q < Q; ++q) load(q, tail(q, k_left));
            asm volatile("");           // (a path of its own: no selects among every slice's loads)
        }
        base += step;
    }
};

// Transposing reads of N fragments from the LDS offsets at[i] and, for their second halves,
// at[i] + OFF.  In assembly, with their wait: the compiler takes the builtin to depend on every
// load into LDS in flight and waits for all of them first, which undoes the requests ahead.
template <int OFF>
__device__ __forceinline__ void read_transposed(const uint32_t (&at)[1], s16x4 (&lo)[1], s16x4 (&hi)[1]) {
    asm volatile("ds_read_b64_tr_b16 %0, %2\n\tds_read_b64_tr_b16 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0]) : "v"(at[0]), "n"(OFF) : "memory");
}
template <int OFF>
__device__ __forceinline__ void read_transposed(const uint32_t (&at)[2], s16x4 (&lo)[2], s16x4 (&hi)[2]) {
    asm volatile("ds_read_b64_tr_b16 %0, %4\n\tds_read_b64_tr_b16 %1, %4 offset:%6\n\t"
                 "ds_read_b64_tr_b16 %2, %5\n\tds_read_b64_tr_b16 %3, %5 offset:%6\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]) : "v"(at[0]), "v"(at[1]), "n"(OFF) : "memory");
}
template <int OFF>
__device__ __forceinline__ void read_transposed(const uint32_t (&at)[4], s16x4 (&lo)[4], s16x4 (&hi)[4]) {
    asm volatile("ds_read_b64_tr_b16 %0, %8\n\tds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
                 "ds_read_b64_tr_b16 %2, %9\n\tds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
                 "ds_read_b64_tr_b16 %4, %10\n\tds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
                 "ds_read_b64_tr_b16 %6, %11\n\tds_read_b64_tr_b16 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]), "=&v"(hi[2]), "=&v"(lo[3]), "=&v"(hi[3])
                 : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(OFF) : "memory");
}
// Transposing reads of 8 fragments, and of 8 and 4 of two operands, with the loads of a slice issued
// among them, and the wait for the reads.  All loads before the reads delay those, all after
// them end late: dx of the 4096 x 12288 block 1267 us before, 1220 after, 1210 among them.
template <int OFF>
__device__ __forceinline__ void read_transposed_and_load(const uint32_t (&at)[8], s16x4 (&lo)[8], s16x4 (&hi)[8],
                                                     const SliceLoads& ld) {
    asm volatile("s_mov_b32 m0, %25\n\tds_read_b64_tr_b16 %0, %16\n\tds_read_b64_tr_b16 %1, %16 offset:%24\n\t"
                 "ds_read_b64_tr_b16 %2, %17\n\tds_read_b64_tr_b16 %3, %17 offset:%24\n\t"
                 "buffer_load_dwordx4 %27, %26, 0 offen lds\n\ts_add_u32 m0, %25, 0x2000\n\t"
                 "ds_read_b64_tr_b16 %4, %18\n\tds_read_b64_tr_b16 %5, %18 offset:%24\n\t"
                 "ds_read_b64_tr_b16 %6, %19\n\tds_read_b64_tr_b16 %7, %19 offset:%24\n\t"
                 "buffer_load_dwordx4 %28, %26, 0 offen lds\n\ts_add_u32 m0, %25, 0x4000\n\t"
                 "ds_read_b64_tr_b16 %8, %20\n\tds_read_b64_tr_b16 %9, %20 offset:%24\n\t"
                 "ds_read_b64_tr_b16 %10, %21\n\tds_read_b64_tr_b16 %11, %21 offset:%24\n\t"
                 "buffer_load_dwordx4 %29, %26, 0 offen lds\n\ts_add_u32 m0, %25, 0x6000\n\t"
                 "ds_read_b64_tr_b16 %12, %22\n\tds_read_b64_tr_b16 %13, %22 offset:%24\n\t"
                 "ds_read_b64_tr_b16 %14, %23\n\tds_read_b64_tr_b16 %15, %23 offset:%24\n\t"
                 "buffer_load_dwordx4 %30, %26, 0 offen lds\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]), "=&v"(hi[2]),
                   "=&v"(lo[3]), "=&v"(hi[3]), "=&v"(lo[4]), "=&v"(hi[4]), "=&v"(lo[5]), "=&v"(hi[5]),
                   "=&v"(lo[6]), "=&v"(hi[6]), "=&v"(lo[7]), "=&v"(hi[7])
                 : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5]), "v"(at[6]),
                   "v"(at[7]), "n"(OFF), "s"(ld.lds), "s"(ld.rsrc), "v"(ld.off[0]), "v"(ld.off[1]),
                   "v"(ld.off[2]), "v"(ld.off[3])
                 : "memory", "m0", "scc");
}
template <int OFF, int OFF2>
__device__ __forceinline__ void read_transposed_and_load(const uint32_t (&at)[8], s16x4 (&lo)[8], s16x4 (&hi)[8],
                                                     const uint32_t (&at2)[4], s16x4 (&lo2)[4], s16x4 (&hi2)[4],
                                                     const SliceLoads& ld) {
    asm volatile("s_mov_b32 m0, %38\n\tds_read_b64_tr_b16 %0, %24\n\tds_read_b64_tr_b16 %1, %24 offset:%36\n\t"
                 "ds_read_b64_tr_b16 %2, %25\n\tds_read_b64_tr_b16 %3, %25 offset:%36\n\t"
                 "ds_read_b64_tr_b16 %4, %26\n\tds_read_b64_tr_b16 %5, %26 offset:%36\n\t"
                 "buffer_load_dwordx4 %40, %39, 0 offen lds\n\ts_add_u32 m0, %38, 0x2000\n\t"
                 "ds_read_b64_tr_b16 %6, %27\n\tds_read_b64_tr_b16 %7, %27 offset:%36\n\t"
                 "ds_read_b64_tr_b16 %8, %28\n\tds_read_b64_tr_b16 %9, %28 offset:%36\n\t"
                 "ds_read_b64_tr_b16 %10, %29\n\tds_read_b64_tr_b16 %11, %29 offset:%36\n\t"
                 "buffer_load_dwordx4 %41, %39, 0 offen lds\n\ts_add_u32 m0, %38, 0x4000\n\t"
                 "ds_read_b64_tr_b16 %12, %30\n\tds_read_b64_tr_b16 %13, %30 offset:%36\n\t"
                 "ds_read_b64_tr_b16 %14, %31\n\tds_read_b64_tr_b16 %15, %31 offset:%36\n\t"
                 "ds_read_b64_tr_b16 %16, %32\n\tds_read_b64_tr_b16 %17, %32 offset:%37\n\t"
                 "buffer_load_dwordx4 %42, %39, 0 offen lds\n\ts_add_u32 m0, %38, 0x6000\n\t"
                 "ds_read_b64_tr_b16 %18, %33\n\tds_read_b64_tr_b16 %19, %33 offset:%37\n\t"
                 "ds_read_b64_tr_b16 %20, %34\n\tds_read_b64_tr_b16 %21, %34 offset:%37\n\t"
                 "ds_read_b64_tr_b16 %22, %35\n\tds_read_b64_tr_b16 %23, %35 offset:%37\n\t"
                 "buffer_load_dwordx4 %43, %39, 0 offen lds\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]), "=&v"(hi[2]),
                   "=&v"(lo[3]), "=&v"(hi[3]), "=&v"(lo[4]), "=&v"(hi[4]), "=&v"(lo[5]), "=&v"(hi[5]),
                   "=&v"(lo[6]), "=&v"(hi[6]), "=&v"(lo[7]), "=&v"(hi[7]), "=&v"(lo2[0]), "=&v"(hi2[0]),
                   "=&v"(lo2[1]), "=&v"(hi2[1]), "=&v"(lo2[2]), "=&v"(hi2[2]), "=&v"(lo2[3]), "=&v"(hi2[3])
                 : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5]), "v"(at[6]),
                   "v"(at[7]), "v"(at2[0]), "v"(at2[1]), "v"(at2[2]), "v"(at2[3]), "n"(OFF), "n"(OFF2),
                   "s"(ld.lds), "s"(ld.rsrc), "v"(ld.off[0]), "v"(ld.off[1]), "v"(ld.off[2]), "v"(ld.off[3])
                 : "memory", "m0", "scc");
}

// This lane's fragment reads of one operand: rows x0 + 16 i + lane % 16 of the tile.
template <int X, bool KC, int ES>
struct Reader {
    uint32_t at[2];          // byte offset for the first and second 64 bytes of K
    __device__ __forceinline__ void init(int x0) {
        const int lane = threadIdx.x % kWave, j = lane % 16, g = lane / 16;
        if constexpr (KC) {
            at[0] = (x0 + j) * kSlice + ((g ^ row_swz(j)) << 4);
            at[1] = at[0] ^ 64;
        } else if constexpr (ES == 2) {
            const int k = 8 * g + j / 4;                      // + 4 for the second read
            at[0] = k * (X * 2) + (j % 4) * 8 + ((x0 / 16 ^ chunk_swz<X, ES>(k) >> 1) << 5);
            at[1] = at[0] + 32 * (X * 2);
        } else {
            const int k = 4 * g;                              // + 0 .. 3
            at[0] = k * (X * 4) + j * 4 + ((x0 / 16 ^ chunk_swz<X, ES>(k) >> 2) << 6);
            at[1] = at[0] + 16 * (X * 4);
        }
    }
    // (fragment i is unit x0 / 16 + i, permuted: a multiple of the wave's fragments plus i, and rows
    // are whole periods of the units, so its offset is that of fragment 0 with the bits of i flipped)
    // transposing reads: LDS offsets of fragments first .. first + N - 1, the offset of their
    // second halves, and the halves as one fragment
    static constexpr int kSecond = 4 * X * 2;
    template <int N>
    __device__ __forceinline__ void offsets(const uint8_t* lds, int half, int first, uint32_t (&from)[N]) const {
        const uint32_t base = uint32_t(reinterpret_cast<uintptr_t>((lds_void*)(lds + at[half])));
#pragma unroll
        for (int i = 0; i < N; ++i) from[i] = base ^ uint32_t(first + i) << 5;
    }
    template <int N, class V>
    static __device__ __forceinline__ void join(const s16x4 (&lo)[N], const s16x4 (&hi)[N], V (&v)[N]) {
        typedef __attribute__((ext_vector_type(8))) short s16x8;
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = __builtin_bit_cast(V, __builtin_shufflevector(lo[i], hi[i], 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // fragments first .. first + N - 1 of half-slice `half`
    template <int N, class V>
    __device__ __forceinline__ void read(const uint8_t* lds, int half, int first, V (&v)[N]) const {
        if constexpr (KC) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = *reinterpret_cast<const V*>(lds + at[half] + (first + i) * 16 * kSlice);
        } else if constexpr (ES == 2) {
            uint32_t from[N];
            s16x4 lo[N], hi[N];
            offsets(lds, half, first, from);
            read_transposed<kSecond>(from, lo, hi);
            join(lo, hi, v);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float* p = reinterpret_cast<const float*>(lds + (at[half] ^ uint32_t(first + i) << 6));
                v[i] = V{p[0], p[X], p[2 * X], p[3 * X]};
            }
        }
    }
};

// Counts of s_waitcnt: vector memory operations that may be in flight, LDS operations (15: any).
constexpr int wait_for(int vm, int lgkm) { return (vm & 15) | (7 << 4) | (lgkm << 8) | ((vm >> 4) << 14); }

// Barrier that hands loaded slices over: every wave waits for its own loads first.
__device__ __forceinline__ void barrier_loads() {
    __builtin_amdgcn_s_waitcnt(wait_for(0, 0));
    __syncthreads();
}

template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NW = WM * WN, kThreads = NW * kWave;
    static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16, FH = FM / 2;
    static constexpr int kFinishRow = TN * 4 + 16, kFinishBytes = NW * 2 * 16 * kFinishRow;
    static constexpr int STAGE = (BM + BN) * kSlice, kLdsBytes = 2 * STAGE;
    static_assert(kLdsBytes >= kFinishBytes && kLdsBytes <= 64 * 1024, "room for the results");
    static constexpr int kWavesPerSimd = NW * (160 * 1024 / kLdsBytes) / 4 < 2 ? 1 : 2;
    static_assert(FH * 32 == TM && FN * 16 == TN && FN % 2 == 0, "fragments");
};

// (row tile, column tile) of tile number `tile`: groups of kGroupM row tiles, columns slowest
__device__ __forceinline__ int2 tile_origin(int tile, int m_tiles, int n_tiles) {
    const int grp = tile / (kGroupM * n_tiles), in = tile % (kGroupM * n_tiles);
    const int gm = min(kGroupM, m_tiles - grp * kGroupM);
    return make_int2(grp * kGroupM + in % gm, in / gm);
}

// Between LDS writes and reads that pass values from lane to lane of one wave: the LDS takes a
// wave's operations in order, so only the compiler has to keep them so.
__device__ __forceinline__ void lanes_in_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// The sums of a wave's TM x TN tile, from its rows m0 and columns n0 on.  A lane holds pieces of
// four columns of 16 rows; written from there, every store instruction would touch 16 rows with
// 32 bytes each, which is slow.  So 16 rows at a time go through LDS (a wave's own part: no
// barrier; two places, the next rows are written before the last are read) and come back as W
// consecutive columns a lane (16 bytes of the result), whole lines of a few rows an instruction.
// Rows lie 4 banks apart.  Results of integer products are streamed (8192 x 24576 x 4096 took
// 690 us against 752: the results of all CUs, which leave at the same time, do not crowd the next
// tiles' operands out of L2); the block's are read by the next product.
// A wait for a load waits for every older store, so the loads of finishing are ahead: column
// scales and a row scale a lane at the start, gate and up values one pass ahead.  PARTIAL: fp32
// (or integer) sums to part, row by row.
template <int TYPE, int EPI, class C, bool PARTIAL, class Acc>
__device__ __forceinline__ void finish_tile(const Product& p, int64_t m0, int n0, const Acc (&acc)[C::FM][C::FN],
                                            uint8_t* lds, void* part, int64_t ld_part) {
    typedef typename Elem<TYPE>::Acc S;
    constexpr int ROW = C::kFinishRow;
    constexpr bool PAIR = kPaired<EPI> && !PARTIAL;
    constexpr int W = TYPE == kF32 || EPI == kGate8 || EPI == kScale32 || PARTIAL ? 4 : 8;
    constexpr int LPR = C::TN / (PAIR ? 2 * W : W);          // lanes a row
    constexpr int RPP = kWave / LPR < 16 ? kWave / LPR : 16; // rows a pass
    static_assert(16 % RPP == 0, "passes of whole rows");
    const int lane = threadIdx.x % kWave;
    uint8_t* st = lds + threadIdx.x / kWave * (2 * 16 * ROW);
    const int lr = lane / LPR, lc = lane % LPR;
    // this lane's first column in the tile: W lc, or the W lc-th gate column
    const int col = PAIR ? lc * W / 16 * 32 + lc * W % 16 : lc * W;
    const int n = n0 + col;
    const bool in = n < p.N && lr < RPP;
    constexpr int PASSES = 16 / RPP, ALL = C::FM * PASSES;
    auto row_of = [&](int k) { return k * RPP + lr % RPP; };    // in the wave's tile
    auto put_rows = [&](int i) {
        uint8_t* d = st + (i & 1) * (16 * ROW) + (lane % 16) * ROW + (lane / 16) * 16;
#pragma unroll
        for (int j = 0; j < C::FN; ++j) *reinterpret_cast<Acc*>(d + j * 64) = acc[i][j];
    };
    ColumnScales<EPI, W> cs;
    float scales = 0.0f;                                     // lane l: the scale of row l
    RowInputs<TYPE, EPI, W> ri[2];
    auto load_inputs = [&](int k) {
        if constexpr (EPI == kDGate && !PARTIAL) {
            const int64_t m = m0 + row_of(k);
            if (m < p.M && in) ri[k & 1].load(p, m, n);
        }
    };
    if constexpr (!PARTIAL) {
        cs.load(p, n < p.N ? n : 0);
        static_assert(C::TM <= kWave, "a row scale a lane");
        if (kScaled<EPI>) {
            const int64_t m = m0 + lane;
            scales = p.row_scale[m < p.M ? m : p.M - 1];
        }
        load_inputs(0);
    }
    put_rows(0);
#pragma unroll
    for (int k = 0; k < ALL; ++k) {
        if (k % PASSES == 0) {
            lanes_in_order();
            if (k / PASSES + 1 < C::FM) put_rows(k / PASSES + 1);
        }
        const uint8_t* row = st + (k / PASSES & 1) * (16 * ROW) + row_of(k) % 16 * ROW + col * 4;
        const int64_t m = m0 + row_of(k);
        S v[W], u[W];
#pragma unroll
        for (int e = 0; e < W / 4; ++e) {
            const Acc t = *reinterpret_cast<const Acc*>(row + e * 16);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[4 * e + q] = t[q];
            if constexpr (PAIR) {
                const Acc w = *reinterpret_cast<const Acc*>(row + 64 + e * 16);
#pragma unroll
                for (int q = 0; q < 4; ++q) u[4 * e + q] = w[q];
            }
        }
        if constexpr (!PARTIAL) {
            if (kScaled<EPI>) ri[k & 1].set_scale(__shfl(scales, row_of(k), kWave));
            if (k + 1 < ALL) load_inputs(k + 1);
        }
        if (m >= p.M || !in) continue;
        if constexpr (PARTIAL) {
            S* d = static_cast<S*>(part) + m * ld_part + n;
            *reinterpret_cast<Acc*>(d) = Acc{v[0], v[1], v[2], v[3]};
        } else {
            finish<TYPE, EPI, W, kScaled<EPI>>(p, m, n, v, u, cs, ri[k & 1]);
        }
    }
}

// 128 x 128 and 64 x 64 tiles: 4 waves, two LDS stages.  The one barrier of a slice stands before
// its last quarter, so the loads of a slice have a whole slice's time to land and the matrix
// instructions of the last quarter cover the first reads of the next slice.
template <int TYPE, int LAYOUT, int EPI, class C>
__device__ __forceinline__ void mma_tile(const Product& p, int block, int m_tiles, int n_tiles, int splits, uint8_t* lds) {
    typedef typename Frag<TYPE>::V V;
    typedef typename Frag<TYPE>::Acc Acc;
    constexpr int ES = Frag<TYPE>::ES, KS = kSlice / ES;
    constexpr bool AKC = LAYOUT != kTN, BKC = LAYOUT == kNT;
    // tile of this workgroup
    const int tiles = m_tiles * n_tiles, total = tiles * splits, per = (total + kXcds - 1) / kXcds;
    const int lid = block % kXcds * per + block / kXcds;
    if (block / kXcds >= per || lid >= total) return;
    const int split = lid / tiles, tile = lid % tiles;
    const int2 mn = tile_origin(tile, m_tiles, n_tiles);
    const int64_t m0 = int64_t(mn.x) * C::BM;
    const int n0 = mn.y * C::BN;
    // this workgroup's slices: [first, first + nk)
    const int all = (p.K + KS - 1) / KS, share = (all + splits - 1) / splits;
    const int first = split * share, nk = min(share, all - first);

    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int wm = wave / C::WN, wn = wave % C::WN;
    Side<C::BM, AKC, ES, C::NW> sa;
    Side<C::BN, BKC, ES, C::NW> sb;
    sa.init(p.a, p.lda, m0, p.M, first);
    sb.init(p.b, p.ldb, n0, p.N, first);
    Reader<C::BM, AKC, ES> ra;
    Reader<C::BN, BKC, ES> rb;
    ra.init(wm * C::TM);
    rb.init(wn * C::TN);

    Acc acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = Acc{0, 0, 0, 0};
    V fa[2][C::FH], fb[2][C::FN];

    // quarter s of a slice: half-slice s / 2 of K, half s % 2 of the wave's rows
    auto read = [&](const uint8_t* st, auto s_) {
        constexpr int s = decltype(s_)::value;
        ra.read(st, s / 2, (s % 2) * C::FH, fa[s % 2]);
        if constexpr (s % 2 == 0) rb.read(st + C::BM * kSlice, s / 2, 0, fb[s / 2]);
    };
    auto mul = [&](auto s_) {
        constexpr int s = decltype(s_)::value;
#pragma unroll
        for (int i = 0; i < C::FH; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                acc[(s % 2) * C::FH + i][j] = mma(fb[s / 2][j], fa[s % 2][i], acc[(s % 2) * C::FH + i][j]);
    };
    // matrix instructions of one quarter with the NR LDS reads of the next spread among them
    // (transposing reads wait for themselves)
    constexpr bool kHinted = (AKC && BKC) || ES != 2;
    auto sched = [&](auto nr_) {
        constexpr int NR = decltype(nr_)::value, NM = C::FH * C::FN * (TYPE == kF32 ? 4 : 1);
        constexpr int PAIRS = NR < NM ? NR : NM;
        if constexpr (!kHinted) return;
#pragma unroll
        for (int n = 0; n < PAIRS; ++n) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        if constexpr (NM > PAIRS) __builtin_amdgcn_sched_group_barrier(0x008, NM - PAIRS, 0);
    };
    typedef std::integral_constant<int, 0> Q0;
    typedef std::integral_constant<int, 1> Q1;
    typedef std::integral_constant<int, 2> Q2;
    typedef std::integral_constant<int, 3> Q3;
    constexpr int RA = C::FH * (AKC ? 1 : ES), RB = C::FN * (BKC ? 1 : ES);     // LDS reads
    typedef std::integral_constant<int, RA> NA;
    typedef std::integral_constant<int, RA + RB> NAB;

    int left = p.K - first * KS;                              // k from the next slice to request on
    auto issue = [&](int stage) {
        uint8_t* st = lds + stage * C::STAGE;
        sa.issue(st, left);
        sb.issue(st + C::BM * kSlice, left);
        left -= KS;
    };
    issue(0);
    barrier_loads();
    if (nk > 1) issue(1);
    read(lds, Q0{});
    for (int ks = 0; ks + 1 < nk; ++ks) {
        const uint8_t* st = lds + (ks & 1) * C::STAGE;
        read(st, Q1{});
        mul(Q0{});
        read(st, Q2{});
        mul(Q1{});
        read(st, Q3{});
        mul(Q2{});
        sched(NA{});
        sched(NAB{});
        sched(NA{});
        barrier_loads();       // slice ks is read by every wave, slice ks + 1 has landed
        if (ks + 2 < nk) issue(ks & 1);
        read(lds + ((ks + 1) & 1) * C::STAGE, Q0{});
        mul(Q3{});
        sched(NAB{});
    }
    {
        const uint8_t* st = lds + ((nk - 1) & 1) * C::STAGE;
        read(st, Q1{});
        mul(Q0{});
        read(st, Q2{});
        mul(Q1{});
        read(st, Q3{});
        mul(Q2{});
        mul(Q3{});
    }
    __syncthreads();                                         // the stages are read
    const int64_t mw = m0 + wm * C::TM;
    const int nw = n0 + wn * C::TN;
    const int64_t row_ld = part_ld(p.N);
    if (splits > 1)
        finish_tile<TYPE, EPI, C, true>(p, mw, nw, acc, lds,
                                        static_cast<typename Elem<TYPE>::Acc*>(p.part) + split * p.M * row_ld, row_ld);
    else
        finish_tile<TYPE, EPI, C, false>(p, mw, nw, acc, lds, nullptr, 0);
}
template <int TYPE, int LAYOUT, int EPI, class C>
__global__ void __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(C::kWavesPerSimd)))
k_mma(const Product p, int m_tiles, int n_tiles, int splits) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    mma_tile<TYPE, LAYOUT, EPI, C>(p, blockIdx.x, m_tiles, n_tiles, splits, lds);
}

// Two products of one kind and one K in a launch (the gradients of the two weights): the first
// `blocks` workgroups (a multiple of the XCDs) serve p, the others q.
struct Pair {
    Product p, q;
    int blocks, m_tiles[2], n_tiles[2];
};
template <int TYPE, int LAYOUT, int EPI, class C>
__global__ void __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(C::kWavesPerSimd)))
k_mma_pair(const Pair a, int splits) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int b = blockIdx.x;
    const bool q = b >= a.blocks;
    const Product p = q ? a.q : a.p;
    mma_tile<TYPE, LAYOUT, EPI, C>(p, q ? b - a.blocks : b, a.m_tiles[q], a.n_tiles[q], splits, lds);
}

__device__ __forceinline__ void fence_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The 256 x 256 tile: 8 waves, two on each SIMD, in two groups that take turns.  While one group
// runs the matrix instructions of half a slice (32 of them, 512 cycles of the matrix unit), the
// other reads its fragments of the next half from LDS; a barrier ends each turn, and the groups
// run half a period apart.  So the matrix units always have a wave whose operands are in
// registers: with loads left out this runs at the rate of the matrix instructions alone.
//
// What then decides is that a turn's loads do not outlast it: the CU's path from memory takes 512
// cycles for 32 KiB, so a slice's 64 KiB have to be spread over its four turns.  The operands lie
// in a ring of five 32 KiB places (all of the LDS), B and A of a slice by turns.  In its first
// reading turn of slice s a group requests its share of A of slice s + 1, in the second that of B
// of slice s + 2: the places are those of slice s - 1.  (Both in the first turn, two stages:
// 1.25 times the time of the loop.)
struct Turns {
    static constexpr int BM = 256, BN = 256, WM = 4, WN = 2, NW = 8, kThreads = 512;
    static constexpr int TM = 64, TN = 128, FM = 4, FN = 8;
    static constexpr int kFinishRow = TN * 4 + 16, kFinishBytes = NW * 2 * 16 * kFinishRow;
    static constexpr int PLACE = 256 * kSlice, kPlaces = 5, kLdsBytes = kPlaces * PLACE;
    static_assert(kLdsBytes >= kFinishBytes && kLdsBytes <= 160 * 1024, "LDS of a CU");
};

template <int TYPE, int LAYOUT, int EPI>
__device__ __forceinline__ void turns_tile(const Product& p, int block, int m_tiles, int n_tiles, uint8_t* lds) {
    typedef Turns C;
    typedef typename Frag<TYPE>::V V;
    typedef typename Frag<TYPE>::Acc Acc;
    constexpr int ES = Frag<TYPE>::ES, KS = kSlice / ES;
    constexpr bool AKC = LAYOUT != kTN, BKC = LAYOUT == kNT;
    const int tiles = m_tiles * n_tiles, per = (tiles + kXcds - 1) / kXcds;
    const int tile = block % kXcds * per + block / kXcds;
    if (block / kXcds >= per || tile >= tiles) return;
    const int2 mn = tile_origin(tile, m_tiles, n_tiles);
    const int64_t m0 = int64_t(mn.x) * C::BM;
    const int n0 = mn.y * C::BN;
    const int n = (p.K + KS - 1) / KS;                        // slices

    const int wave = threadIdx.x / kWave;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const bool second = __builtin_amdgcn_readfirstlane(wave) >= 4;    // (SIMD i has waves i and i + 4)
    Side<C::BM, AKC, ES, C::NW> sa;
    Side<C::BN, BKC, ES, C::NW> sb;
    sa.init(p.a, p.lda, m0, p.M, 0);
    sb.init(p.b, p.ldb, n0, p.N, 0);
    constexpr int kLoads = decltype(sb)::Q;                   // a wave's loads of B of a slice
    Reader<C::BM, AKC, ES> ra;
    Reader<C::BN, BKC, ES> rb;
    ra.init(wm * C::TM);
    rb.init(wn * C::TN);
    Acc acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = Acc{0, 0, 0, 0};

    int left_a = p.K, left_b = p.K;                           // k from the next slice to request on
    auto place = [&](int u) { return lds + (u >= C::kPlaces ? u - C::kPlaces : u) * C::PLACE; };
    auto issue_a = [&](int u) {
        sa.issue(place(u), left_a);
        left_a -= KS;
    };
    auto issue_b = [&](int u) {
        sb.issue(place(u), left_b);
        left_b -= KS;
    };
    // all but the newest B has landed: B of the slice after next, where there is one
    auto landed = [&](bool newest, auto lgkm_) {
        constexpr int lgkm = decltype(lgkm_)::value;
        if (newest) __builtin_amdgcn_s_waitcnt(wait_for(kLoads, lgkm));
        else __builtin_amdgcn_s_waitcnt(wait_for(0, lgkm));
    };
    typedef std::integral_constant<int, 0> AlsoLds;
    typedef std::integral_constant<int, 15> NotLds;
    issue_b(0);
    issue_a(1);
    if (n > 1) issue_b(2);
    landed(n > 1, NotLds{});
    fence_barrier();
    if (second) fence_barrier();                              // half a period behind
    int u = 0;                                                // B's place, A's is the next
    constexpr bool kLoadsInside = !BKC && ES == 2;            // loads issued among the transposing reads
    if constexpr (kLoadsInside) {
        if (left_a < KS) sa.end_of_k(left_a);
        if (left_b < KS) sb.end_of_k(left_b);
    }
    for (int j = 0; j < n; ++j) {
        const uint8_t *pb = place(u), *pa = place(u + 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            V fa[C::FM], fb[C::FN];
            if constexpr (kLoadsInside) {
                // (past the last slice the loads are out of range and write zeros to a free place)
                uint32_t tb[C::FN];
                s16x4 lb[C::FN], hb[C::FN];
                if (AKC) ra.read(pa, half, 0, fa);
                const SliceLoads ld = half == 0 ? sa.next(place(u + 3)) : sb.next(place(u + 4));
                rb.offsets(pb, half, 0, tb);
                if constexpr (AKC) {
                    read_transposed_and_load<decltype(rb)::kSecond>(tb, lb, hb, ld);
                } else {
                    uint32_t ta[C::FM];
                    s16x4 la[C::FM], ha[C::FM];
                    ra.offsets(pa, half, 0, ta);
                    read_transposed_and_load<decltype(rb)::kSecond, decltype(ra)::kSecond>(tb, lb, hb, ta, la, ha, ld);
                    ra.join(la, ha, fa);
                }
                rb.join(lb, hb, fb);
            } else {
                // (reads that the compiler waits for later, then loads)
                ra.read(pa, half, 0, fa);
                rb.read(pb, half, 0, fb);
                if (half == 0 && j + 1 < n) issue_a(u + 3);
                if (half == 1 && j + 2 < n) issue_b(u + 4);
            }
            // slice j + 1 has landed at the end of the slice's last turn: a reading turn of the
            // second group, a computing turn of the first
            if (half == 1 && second) landed(j + (kLoadsInside ? 1 : 2) < n, AlsoLds{});
            else __builtin_amdgcn_s_waitcnt(wait_for(63, 0));
            fence_barrier();
            if constexpr (kLoadsInside) {
                if (half == 0) {
                    left_a -= KS;
                    if (left_a < KS) sa.end_of_k(left_a);
                } else {
                    left_b -= KS;
                    if (left_b < KS) sb.end_of_k(left_b);
                }
            }
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int k = 0; k < C::FN; ++k) acc[i][k] = mma(fb[k], fa[i], acc[i][k]);
            __builtin_amdgcn_s_setprio(0);
            if (half == 1 && !second) landed(j + (kLoadsInside ? 1 : 2) < n, NotLds{});
            fence_barrier();
        }
        u = u + 2 >= C::kPlaces ? u + 2 - C::kPlaces : u + 2;
    }
    if (!second) fence_barrier();

    finish_tile<TYPE, EPI, C, false>(p, m0 + wm * C::TM, n0 + wn * C::TN, acc, lds, nullptr, 0);
}
template <int TYPE, int LAYOUT, int EPI>
__global__ void __launch_bounds__(Turns::kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
k_mma_turns(const Product p, int m_tiles, int n_tiles) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    turns_tile<TYPE, LAYOUT, EPI>(p, blockIdx.x, m_tiles, n_tiles, lds);
}
template <int TYPE, int LAYOUT, int EPI>
__global__ void __launch_bounds__(Turns::kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
k_mma_turns_pair(const Pair a) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int b = blockIdx.x;
    const bool q = b >= a.blocks;
    const Product p = q ? a.q : a.p;
    turns_tile<TYPE, LAYOUT, EPI>(p, q ? b - a.blocks : b, a.m_tiles[q], a.n_tiles[q], lds);
}

// Adds the splits' partial sums, in order, and finishes: 4 columns (or 4 pairs) of a row a thread.
template <int TYPE, int EPI>
__global__ void __launch_bounds__(256) k_join(const Product p, int splits) {
    typedef typename Elem<TYPE>::Acc S;
    typedef typename Frag<TYPE>::Acc V4;
    constexpr bool PAIR = kPaired<EPI>;
    const int64_t ld = part_ld(p.N), units = PAIR ? p.N / 8 : ld / 4, i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= p.M * units) return;
    const int64_t m = i / units;
    const int k = int(i % units), n = PAIR ? k / 4 * 32 + k % 4 * 4 : k * 4;
    if (n >= p.N) return;
    ColumnScales<EPI, 4> cs;
    cs.load(p, n);
    RowInputs<TYPE, EPI, 4> in;
    in.load(p, m, n);
    S v[4], u[4];
    auto add = [&](S (&t)[4], int col) {
        const S* part = static_cast<const S*>(p.part) + m * ld + col;
        V4 a = *reinterpret_cast<const V4*>(part);
#pragma unroll 8
        for (int s = 1; s < splits; ++s) {
            part += p.M * ld;
            a += *reinterpret_cast<const V4*>(part);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = a[e];
    };
    add(v, n);
    if constexpr (PAIR) add(u, n + 16);
    finish<TYPE, EPI, 4, false>(p, m, n, v, u, cs, in);
}

typedef Tile<128, 128, 2, 2> Mid;            // two workgroups a CU
typedef Tile<64, 64, 2, 2> Small;            // four

// Lets a kernel use more than 64 KiB of LDS, once on each device.
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

int64_t part_bytes(const Product& p, int splits) { return p.M * part_ld(p.N) * splits * 4; }

// LDS of a workgroup.  One slice needs one stage; twice the workgroups on a CU then hide each
// other's one trip to memory (gradients of the 4096 x 1536 block from 37 tokens 13.6 against 16.6 us).
template <class C>
int lds_bytes(const Product& p, int es) {
    if (int64_t(p.K) * es > kSlice) return C::kLdsBytes;
    return C::STAGE > C::kFinishBytes ? C::STAGE : C::kFinishBytes;
}

// The tiles of a product, and the workgroups of a launch for them (0: too many).
struct Tiles {
    int m, n;
    unsigned blocks;
};
template <class C>
Tiles tiles_of(const Product& p, int splits) {
    const int64_t mt = (p.M + C::BM - 1) / C::BM, nt = (p.N + C::BN - 1) / C::BN;
    const int64_t blocks = (mt * nt * splits + kXcds - 1) / kXcds * kXcds;
    if (mt * nt > 0x7FFFFFF0 / kXcds || blocks > 0x7FFFFFFF / C::kThreads) return Tiles{0, 0, 0};
    return Tiles{int(mt), int(nt), unsigned(blocks)};
}

template <int TYPE, int EPI>
hipError_t launch_join(const Product& p, int splits, hipStream_t s) {
    // (few results: more workgroups of one wave)
    const int64_t items = p.M * (kPaired<EPI> ? p.N / 8 : part_ld(p.N) / 4);
    const int threads = items < 256 * 1024 ? 64 : 256;
    hipLaunchKernelGGL((k_join<TYPE, EPI>), dim3(unsigned((items + threads - 1) / threads)), dim3(threads), 0, s, p, splits);
    return hipGetLastError();
}

template <int TYPE, int LAYOUT, int EPI, class C>
hipError_t launch(const Product& p, int splits, hipStream_t s) {
    const Tiles t = tiles_of<C>(p, splits);
    if (t.blocks == 0) return hipErrorInvalidValue;
    if (splits > 1 && part_bytes(p, splits) > p.part_bytes) return hipErrorInvalidValue;
    if constexpr (std::is_same<C, Turns>::value) {
        const auto kernel = &k_mma_turns<TYPE, LAYOUT, EPI>;
        static std::atomic<uint64_t> allowed{0};
        hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), C::kLdsBytes, allowed);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kernel, dim3(t.blocks), dim3(C::kThreads), C::kLdsBytes, s, p, t.m, t.n);
        return hipGetLastError();
    } else {
        hipLaunchKernelGGL((k_mma<TYPE, LAYOUT, EPI, C>), dim3(t.blocks), dim3(C::kThreads), lds_bytes<C>(p, Frag<TYPE>::ES), s,
                           p, t.m, t.n, splits);
    }
    hipError_t e = hipGetLastError();
    return e != hipSuccess || splits == 1 ? e : launch_join<TYPE, EPI>(p, splits, s);
}

template <int TYPE, int LAYOUT, int EPI, class C>
hipError_t launch_two(const Product& p, const Product& q, int splits, hipStream_t s) {
    const Tiles t = tiles_of<C>(p, splits), u = tiles_of<C>(q, splits);
    if (t.blocks == 0 || u.blocks == 0 || int64_t(t.blocks) + u.blocks > 0x7FFFFFFF / C::kThreads) return hipErrorInvalidValue;
    Pair a{p, q, int(t.blocks), {t.m, u.m}, {t.n, u.n}};
    const int64_t first = align256(part_bytes(p, splits));
    if (splits > 1 && first + part_bytes(q, splits) > p.part_bytes) return hipErrorInvalidValue;
    if (splits > 1) a.q.part = static_cast<uint8_t*>(p.part) + first;
    if constexpr (std::is_same<C, Turns>::value) {
        const auto kernel = &k_mma_turns_pair<TYPE, LAYOUT, EPI>;
        static std::atomic<uint64_t> allowed{0};
        hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), C::kLdsBytes, allowed);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kernel, dim3(t.blocks + u.blocks), dim3(C::kThreads), C::kLdsBytes, s, a);
        return hipGetLastError();
    } else {
        hipLaunchKernelGGL((k_mma_pair<TYPE, LAYOUT, EPI, C>), dim3(t.blocks + u.blocks), dim3(C::kThreads),
                           lds_bytes<C>(p, Frag<TYPE>::ES), s, a, splits);
    }
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && splits > 1) e = launch_join<TYPE, EPI>(a.p, splits, s);
    if (e == hipSuccess && splits > 1) e = launch_join<TYPE, EPI>(a.q, splits, s);
    return e;
}

template <int TYPE, int LAYOUT, int EPI>
hipError_t choose_two(const Product& p, const Product& q, hipStream_t s) {
    const Sizes second = q.sizes();
    const Tiling c = plan_tiles(p.sizes(), &second, Frag<TYPE>::ES, p.part_bytes, compute_units());
    if (c.tile == kTile256) return launch_two<TYPE, LAYOUT, EPI, Turns>(p, q, c.splits, s);
    if (c.tile == kTile128) return launch_two<TYPE, LAYOUT, EPI, Mid>(p, q, c.splits, s);
    return launch_two<TYPE, LAYOUT, EPI, Small>(p, q, c.splits, s);
}

template <int TYPE, int LAYOUT, int EPI>
hipError_t choose(const Product& p, hipStream_t s) {
    const Tiling c = plan_tiles(p.sizes(), nullptr, Frag<TYPE>::ES, p.part_bytes, compute_units());
    if (c.tile == kTile256) return launch<TYPE, LAYOUT, EPI, Turns>(p, c.splits, s);
    if (c.tile == kTile128) return launch<TYPE, LAYOUT, EPI, Mid>(p, c.splits, s);
    return launch<TYPE, LAYOUT, EPI, Small>(p, c.splits, s);
}

}  // namespace

hipError_t launch_product(int type, int layout, int epi, const Product& p, hipStream_t s) {
    if (p.M <= 0 || p.N <= 0) return hipSuccess;
    if (layout == kNT && few_tokens(p.sizes(), elem_bytes(type))) return launch_few(type, epi, p, s);
    if (type == kI8) {
        if (layout == kNT && epi == kScale) return choose<kI8, kNT, kScale>(p, s);
        if (layout == kNT && epi == kScale32) return choose<kI8, kNT, kScale32>(p, s);
        if (layout == kNT && epi == kGate8) return choose<kI8, kNT, kGate8>(p, s);
        return hipErrorInvalidValue;
    }
    const bool f32 = type == kF32;
    if (layout == kNT && epi == kStore) return f32 ? choose<kF32, kNT, kStore>(p, s) : choose<kBF16, kNT, kStore>(p, s);
    if (layout == kNT && epi == kGate) return f32 ? choose<kF32, kNT, kGate>(p, s) : choose<kBF16, kNT, kGate>(p, s);
    if (layout == kNN && epi == kStore) return f32 ? choose<kF32, kNN, kStore>(p, s) : choose<kBF16, kNN, kStore>(p, s);
    if (layout == kNN && epi == kDGate) return f32 ? choose<kF32, kNN, kDGate>(p, s) : choose<kBF16, kNN, kDGate>(p, s);
    return hipErrorInvalidValue;
}

hipError_t launch_gradients(int type, const Product& p, const Product& q, hipStream_t s) {
    return type == kF32 ? choose_two<kF32, kTN, kStore>(p, q, s) : choose_two<kBF16, kTN, kStore>(p, q, s);
}

}  // namespace dense
}  // namespace moe
