// Entry points of the dense operators: 8-bit integer products, and the dense gated block with
// its backward pass and its 8-bit form.  Contracts in include/moe.h; the kernels are in
// dense_quant.hip, dense_few.hip and dense_mma.hip.
#include <hip/hip_runtime.h>

#include "dense.h"

namespace moe {
namespace {

using namespace dense;

std::atomic<int> g_units[64];

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Workspace of moe_i8_matmul: codes and scales of x, and partial sums of calls with few tokens.
struct I8Work {
    int64_t codes = 0, scale = 0, part = 0, bytes = 0;
};
I8Work i8_work(int64_t T, int64_t K) {
    I8Work w;
    if (T < 1) T = 1;
    w.scale = align256(T * K);
    w.part = align256(w.scale + T * 4);
    w.bytes = w.part + i8_part_bytes(T);
    return w;
}

// Workspace of the block's calls: the forward pass without a save buffer keeps h, the backward
// pass dg and du; the 8-bit form the codes of x, h in fp32 and the codes of h.
struct BlockWork {
    int64_t xq = 0, xs = 0, h = 0, hq = 0, hs = 0, part = 0, bytes = 0;
};
BlockWork block_work(const moe_config& c, int64_t T) {
    BlockWork w;
    if (T < 1) T = 1;
    const int64_t H = c.hidden, I = c.inter, es = act_bytes(c);
    w.xs = align256(T * H);
    w.h = align256(w.xs + T * 4);
    w.hq = align256(w.h + T * I * 4);
    w.hs = align256(w.hq + T * I);
    const int64_t i8 = c.w_dtype == MOE_W_BF16 ? align256(w.hs + T * 4) : 0, dgu = align256(T * 2 * I * es);
    w.part = i8 > dgu ? i8 : dgu;
    w.bytes = w.part + kPartBytes;
    return w;
}

// What the forward pass saves: pre-activations [T][2I] (fp32, or for bf16 24 bits: the upper 16 in
// one array, the lower 8 in another), then h [T][I].
int64_t save_low_offset(const moe_config& c, int64_t T) { return align256(T * 2 * c.inter * act_bytes(c)); }
int64_t save_h_offset(const moe_config& c, int64_t T) {
    return align256(save_low_offset(c, T) + (c.w_dtype == MOE_W_F32 ? 0 : T * 2 * c.inter));
}

struct Blob8 {
    int64_t gu = 0, d = 0, gu_scale = 0, d_scale = 0, bytes = 0;
};
Blob8 blob8_layout(const moe_config& c) {
    const int64_t H = c.hidden, I = c.inter;
    Blob8 b;
    b.d = align256(2 * I * H);
    b.gu_scale = align256(b.d + H * I);
    b.d_scale = align256(b.gu_scale + 2 * I * 4);
    b.bytes = align256(b.d_scale + H * 4);
    return b;
}

constexpr int kMaxWidth = 1 << 20;    // H and I: row offsets inside a tile stay below 2 GiB
constexpr int kMaxCount = 1 << 24;    // tokens, outputs, columns: the threads of a launch fit 32 bits

// The configs that the block's calls take: their sizes and the packing refuse the others too.
int check_config(const moe_config& c, bool i8, const char** why) {
    if (i8 && c.w_dtype != MOE_W_BF16) {
        *why = "the 8-bit block is made from and for bf16 contexts";
        return MOE_EUNSUPPORTED;
    }
    if (c.w_dtype == MOE_W_MXFP4) {
        *why = "the dense block takes fp32 or bf16 weights";
        return MOE_EUNSUPPORTED;
    }
    if (i8 && (c.inter > kMaxKI8 || c.hidden > kMaxKI8)) {
        *why = "the 8-bit block takes H and I up to 131056";
        return MOE_ESHAPE;
    }
    if (c.hidden > kMaxWidth || c.inter > kMaxWidth) {
        *why = "the dense block takes H and I up to 2^20";
        return MOE_ESHAPE;
    }
    return MOE_OK;
}

int check_size(const moe_config* c, int32_t T, bool i8) {
    int st = validate_config(c, nullptr);
    if (st != MOE_OK) return st;
    if (T < 0) return MOE_EINVAL;
    const char* why;
    return check_config(*c, i8, &why);
}

int check_block(moe_ctx* ctx, int32_t T, bool i8) {
    if (T < 0) return fail(ctx, MOE_EINVAL, "T < 0");
    if (T > kMaxCount) return fail(ctx, MOE_ESHAPE, "T above 2^24");
    const char* why;
    const int st = check_config(ctx->cfg, i8, &why);
    return st == MOE_OK ? st : fail(ctx, st, why);
}

// Rows of numbers that start on 16 bytes each.
bool whole_rows(const void* x, int x_type, int64_t ld) {
    return aligned(x, 16) && ld * (x_type == MOE_A_F32 ? 4 : 2) % 16 == 0;
}

int type_of(const moe_config& c) { return c.w_dtype == MOE_W_F32 ? kF32 : kBF16; }

}  // namespace

int dense::compute_units() {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    n = g_units[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1) n = 256;
        g_units[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace moe

using namespace moe;
using namespace moe::dense;

extern "C" {

int64_t moe_i8_workspace_bytes(int32_t max_T, int32_t K) {
    if (max_T < 0) return MOE_EINVAL;
    if (K < 16 || K % 16 || K > kMaxKI8) return MOE_ESHAPE;
    // (fewer tokens may need more: the partial sums)
    const int64_t most = i8_work(max_T, K).bytes, few = i8_work(max_T < kSplitTokens ? max_T : kSplitTokens, K).bytes;
    return most > few ? most : few;
}

int moe_i8_quantize(moe_ctx* ctx, const void* d_x, int32_t x_type, int64_t ld_x, int32_t rows, int32_t cols,
                    int8_t* d_q, float* d_scale, hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    if (rows < 0) return fail(ctx, MOE_EINVAL, "rows < 0");
    if (x_type != MOE_A_F32 && x_type != MOE_A_BF16) return fail(ctx, MOE_EINVAL, "x must be fp32 or bf16");
    if (cols < 16 || cols % 16 || cols > kMaxCount)
        return fail(ctx, MOE_ESHAPE, "cols must be a multiple of 16 in 16..2^24");
    if (ld_x < cols) return fail(ctx, MOE_EINVAL, "ld_x < cols");
    if (rows == 0) return MOE_OK;
    if (!d_x || !d_q || !d_scale) return fail(ctx, MOE_EINVAL, "null buffer");
    if (!aligned(d_x, x_type == MOE_A_F32 ? 4 : 2) || !aligned(d_q, 16) || !aligned(d_scale, 4))
        return fail(ctx, MOE_EINVAL, "misaligned buffer");
    hipError_t e = launch_quantize(d_x, x_type, ld_x, rows, cols, d_q, d_scale, s);
    return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_i8_quantize launch");
}

int moe_i8_matmul(moe_ctx* ctx, const void* d_x, int32_t x_type, int64_t ld_x, const float* d_x_scale, int32_t T,
                  const int8_t* d_w, const float* d_w_scale, int32_t N, int32_t K, void* d_y, int32_t y_type,
                  int64_t ld_y, void* d_ws, hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    if (T < 0) return fail(ctx, MOE_EINVAL, "T < 0");
    if (x_type != MOE_A_F32 && x_type != MOE_A_BF16 && x_type != MOE_A_I8) return fail(ctx, MOE_EINVAL, "unknown x type");
    if (y_type != MOE_A_F32 && y_type != MOE_A_BF16) return fail(ctx, MOE_EINVAL, "y must be fp32 or bf16");
    if (K < 16 || K % 16 || K > kMaxKI8) return fail(ctx, MOE_ESHAPE, "K must be a multiple of 16 in 16..131056");
    if (N < 1 || N > kMaxCount || T > kMaxCount) return fail(ctx, MOE_ESHAPE, "N in 1..2^24, T up to 2^24");
    const bool codes = x_type == MOE_A_I8;
    if (ld_x < K || (codes && ld_x != K)) return fail(ctx, MOE_EINVAL, "ld_x: at least K, and K itself for codes");
    if (ld_y < N) return fail(ctx, MOE_EINVAL, "ld_y < N");
    if (T == 0) return MOE_OK;
    if (!d_x || !d_w || !d_w_scale || !d_y || !d_ws) return fail(ctx, MOE_EINVAL, "null buffer");
    if (codes != (d_x_scale != nullptr)) return fail(ctx, MOE_EINVAL, "x scales go with codes, and only with them");
    if (!aligned(d_x, codes ? 16 : x_type == MOE_A_F32 ? 4 : 2) || !aligned(d_w, 16) || !aligned(d_w_scale, 4) ||
        !aligned(d_x_scale, 4) || !aligned(d_y, y_type == MOE_A_F32 ? 4 : 2) || !aligned(d_ws, 256))
        return fail(ctx, MOE_EINVAL, "misaligned buffer");
    Product p{};
    p.a = d_x;
    p.lda = ld_x;
    p.row_scale = d_x_scale;
    const I8Work w = i8_work(T, K);
    p.part = static_cast<uint8_t*>(d_ws) + w.part;
    p.part_bytes = w.bytes - w.part;
    const bool on_the_way = !codes && quantise_inside(ld_x, whole_rows(d_x, x_type, ld_x), T, K, N);
    if (!codes && !on_the_way) {
        int8_t* q = static_cast<int8_t*>(d_ws) + w.codes;
        float* sc = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + w.scale);
        hipError_t e = launch_quantize(d_x, x_type, ld_x, T, K, q, sc, s);
        if (e != hipSuccess) return hip_fail(ctx, e, "moe_i8_matmul launch");
        p.a = q;
        p.lda = K;
        p.row_scale = sc;
    }
    p.b = d_w;
    p.ldb = K;
    p.M = T;
    p.N = N;
    p.K = K;
    p.out = d_y;
    p.ldo = ld_y;
    p.vec_out = y_type == MOE_A_F32 || (aligned(d_y, 4) && ld_y % 2 == 0);
    p.col_scale = d_w_scale;
    const int epi = y_type == MOE_A_F32 ? kScale32 : kScale;
    hipError_t e = on_the_way ? launch_few(kI8, epi, p, s, x_type, true) : launch_product(kI8, kNT, epi, p, s);
    return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_i8_matmul launch");
}

int64_t moe_dense_workspace_bytes(const moe_config* cfg, int32_t max_T) {
    const int st = check_size(cfg, max_T, false);
    if (st != MOE_OK) return st;
    return block_work(*cfg, max_T).bytes;
}

int64_t moe_dense_save_bytes(const moe_config* cfg, int32_t T) {
    const int st = check_size(cfg, T, false);
    if (st != MOE_OK) return st;
    return align256(save_h_offset(*cfg, T) + int64_t(T) * cfg->inter * act_bytes(*cfg));
}

int moe_dense_ffn(moe_ctx* ctx, const void* d_x, int32_t T, const void* d_blob, void* d_save, void* d_y, void* d_ws,
                  hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    int st = check_block(ctx, T, false);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!d_x || !d_blob || !d_y || !d_ws) return fail(ctx, MOE_EINVAL, "null buffer");
    if (!aligned(d_x, 16) || !aligned(d_blob, 16) || !aligned(d_y, 16) || !aligned(d_ws, 16) || !aligned(d_save, 16))
        return fail(ctx, MOE_EINVAL, "buffers must be 16-byte aligned");
    const moe_config& c = ctx->cfg;
    const int type = type_of(c);
    const uint8_t* blob = static_cast<const uint8_t*>(d_blob);
    uint8_t* h = d_save ? static_cast<uint8_t*>(d_save) + save_h_offset(c, T) : static_cast<uint8_t*>(d_ws);
    Product p{};
    p.part = static_cast<uint8_t*>(d_ws) + block_work(c, T).part;
    p.part_bytes = kPartBytes;
    p.a = d_x;
    p.b = blob + ctx->lay.gu;
    p.lda = p.ldb = c.hidden;
    p.M = T;
    p.N = 2 * c.inter;
    p.K = c.hidden;
    p.out = h;
    p.ldo = c.inter;
    p.gu = d_save;
    p.gu_low = d_save ? static_cast<uint8_t*>(d_save) + save_low_offset(c, T) : nullptr;
    hipError_t e = launch_product(type, kNT, kGate, p, s);
    if (e != hipSuccess) return hip_fail(ctx, e, "moe_dense_ffn launch");
    p.a = h;
    p.b = blob + ctx->lay.d;
    p.lda = p.ldb = c.inter;
    p.N = c.hidden;
    p.K = c.inter;
    p.out = d_y;
    p.ldo = c.hidden;
    p.gu = nullptr;
    e = launch_product(type, kNT, kStore, p, s);
    return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_dense_ffn launch");
}

int moe_dense_ffn_backward(moe_ctx* ctx, const void* d_dy, const void* d_x, int32_t T, const void* d_blob,
                           const void* d_save, void* d_dx, void* d_dblob, void* d_ws, hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    int st = check_block(ctx, T, false);
    if (st != MOE_OK) return st;
    const moe_config& c = ctx->cfg;
    const int64_t H = c.hidden, I = c.inter, es = act_bytes(c);
    uint8_t* dblob = static_cast<uint8_t*>(d_dblob);
    if (!aligned(d_dblob, 16)) return fail(ctx, MOE_EINVAL, "buffers must be 16-byte aligned");
    if (T == 0) {
        if (!dblob) return MOE_OK;
        hipError_t e = launch_zero(dblob + ctx->lay.gu, 2 * I * H * es / 16, s);
        if (e == hipSuccess) e = launch_zero(dblob + ctx->lay.d, H * I * es / 16, s);
        return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_dense_ffn_backward launch");
    }
    if (!d_dy || !d_x || !d_blob || !d_save || !d_ws) return fail(ctx, MOE_EINVAL, "null buffer");
    if (!aligned(d_dy, 16) || !aligned(d_x, 16) || !aligned(d_blob, 16) || !aligned(d_save, 16) || !aligned(d_dx, 16) ||
        !aligned(d_ws, 16))
        return fail(ctx, MOE_EINVAL, "buffers must be 16-byte aligned");
    if (!d_dx && !d_dblob) return MOE_OK;
    const int type = type_of(c);
    const uint8_t* blob = static_cast<const uint8_t*>(d_blob);
    const uint8_t* save = static_cast<const uint8_t*>(d_save);
    hipError_t e;
    // dg, du [T][2I] from dh = dy . Wd, which is never stored
    Product p{};
    p.part = static_cast<uint8_t*>(d_ws) + block_work(c, T).part;
    p.part_bytes = kPartBytes;
    p.a = d_dy;
    p.lda = H;
    p.b = blob + ctx->lay.d;
    p.ldb = I;
    p.M = T;
    p.N = int32_t(I);
    p.K = int32_t(H);
    p.out = d_ws;
    p.ldo = 2 * I;
    p.gu = const_cast<uint8_t*>(save);
    p.gu_low = const_cast<uint8_t*>(save) + save_low_offset(c, T);
    if ((e = launch_product(type, kNN, kDGate, p, s)) != hipSuccess) return hip_fail(ctx, e, "moe_dense_ffn_backward launch");
    if (dblob) {
        Product w{};                                   // dWgu = (dg, du)^T x
        w.part = p.part;
        w.part_bytes = p.part_bytes;
        w.a = d_ws;
        w.lda = 2 * I;
        w.b = d_x;
        w.ldb = H;
        w.M = 2 * I;
        w.N = int32_t(H);
        w.K = T;
        w.out = dblob + ctx->lay.gu;
        w.ldo = H;
        Product v = w;                                 // dWd = dy^T h
        v.a = d_dy;
        v.lda = H;
        v.b = save + save_h_offset(c, T);
        v.ldb = I;
        v.M = H;
        v.N = int32_t(I);
        v.out = dblob + ctx->lay.d;
        v.ldo = I;
        if ((e = launch_gradients(type, w, v, s)) != hipSuccess) return hip_fail(ctx, e, "moe_dense_ffn_backward launch");
    }
    if (d_dx) {
        Product q{};
        q.part = p.part;
        q.part_bytes = p.part_bytes;                   // dx = dg Wg + du Wu
        q.a = d_ws;
        q.lda = 2 * I;
        q.b = blob + ctx->lay.gu;
        q.ldb = H;
        q.M = T;
        q.N = int32_t(H);
        q.K = int32_t(2 * I);
        q.out = d_dx;
        q.ldo = H;
        if ((e = launch_product(type, kNN, kStore, q, s)) != hipSuccess)
            return hip_fail(ctx, e, "moe_dense_ffn_backward launch");
    }
    return MOE_OK;
}

int64_t moe_i8_blob_bytes(const moe_config* cfg) {
    const int st = check_size(cfg, 0, true);
    return st != MOE_OK ? st : blob8_layout(*cfg).bytes;
}

int moe_i8_pack(moe_ctx* ctx, const void* d_blob, void* d_blob8, hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    int st = check_block(ctx, 0, true);
    if (st != MOE_OK) return st;
    if (!d_blob || !d_blob8) return fail(ctx, MOE_EINVAL, "null buffer");
    if (!aligned(d_blob, 256) || !aligned(d_blob8, 256)) return fail(ctx, MOE_EINVAL, "blobs must be 256-byte aligned");
    const moe_config& c = ctx->cfg;
    const Blob8 b = blob8_layout(c);
    const uint8_t* src = static_cast<const uint8_t*>(d_blob);
    uint8_t* dst = static_cast<uint8_t*>(d_blob8);
    hipError_t e = launch_quantize(src + ctx->lay.gu, MOE_A_BF16, c.hidden, 2 * int64_t(c.inter), c.hidden,
                                   reinterpret_cast<int8_t*>(dst + b.gu), reinterpret_cast<float*>(dst + b.gu_scale), s);
    if (e == hipSuccess)
        e = launch_quantize(src + ctx->lay.d, MOE_A_BF16, c.inter, c.hidden, c.inter,
                            reinterpret_cast<int8_t*>(dst + b.d), reinterpret_cast<float*>(dst + b.d_scale), s);
    return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_i8_pack launch");
}

int moe_i8_ffn(moe_ctx* ctx, const void* d_x, int32_t T, const void* d_blob8, void* d_y, void* d_ws, hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    int st = check_block(ctx, T, true);
    if (st != MOE_OK) return st;
    const moe_config& c = ctx->cfg;
    if (T == 0) return MOE_OK;
    if (!d_x || !d_blob8 || !d_y || !d_ws) return fail(ctx, MOE_EINVAL, "null buffer");
    if (!aligned(d_x, 16) || !aligned(d_blob8, 256) || !aligned(d_y, 16) || !aligned(d_ws, 16))
        return fail(ctx, MOE_EINVAL, "misaligned buffer");
    const Blob8 b = blob8_layout(c);
    const BlockWork w = block_work(c, T);
    const uint8_t* blob = static_cast<const uint8_t*>(d_blob8);
    uint8_t* ws = static_cast<uint8_t*>(d_ws);
    int8_t* xq = reinterpret_cast<int8_t*>(ws + w.xq);
    int8_t* hq = reinterpret_cast<int8_t*>(ws + w.hq);
    float* xs = reinterpret_cast<float*>(ws + w.xs);
    float* hs = reinterpret_cast<float*>(ws + w.hs);
    hipError_t e = hipSuccess;
    const bool x_inside = quantise_inside(c.hidden, true, T, c.hidden, 2 * c.inter);
    const bool h_inside = quantise_inside(c.inter, true, T, c.inter, c.hidden);
    Product p{};
    p.part = ws + w.part;
    p.part_bytes = kPartBytes;
    if (!x_inside) e = launch_quantize(d_x, MOE_A_BF16, c.hidden, T, c.hidden, xq, xs, s);
    p.a = x_inside ? d_x : xq;
    p.b = blob + b.gu;
    p.lda = p.ldb = c.hidden;
    p.M = T;
    p.N = 2 * c.inter;
    p.K = c.hidden;
    p.out = ws + w.h;
    p.ldo = c.inter;
    p.row_scale = xs;
    p.col_scale = reinterpret_cast<const float*>(blob + b.gu_scale);
    if (e == hipSuccess)
        e = x_inside ? launch_few(kI8, kGate8, p, s, MOE_A_BF16, true) : launch_product(kI8, kNT, kGate8, p, s);
    if (e == hipSuccess && !h_inside) e = launch_quantize(ws + w.h, MOE_A_F32, c.inter, T, c.inter, hq, hs, s);
    p.a = h_inside ? ws + w.h : static_cast<const void*>(hq);
    p.b = blob + b.d;
    p.lda = p.ldb = c.inter;
    p.N = c.hidden;
    p.K = c.inter;
    p.out = d_y;
    p.ldo = c.hidden;
    p.vec_out = 1;
    p.row_scale = hs;
    p.col_scale = reinterpret_cast<const float*>(blob + b.d_scale);
    if (e == hipSuccess)
        e = h_inside ? launch_few(kI8, kScale, p, s, MOE_A_F32, true) : launch_product(kI8, kNT, kScale, p, s);
    return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_i8_ffn launch");
}

}  // extern "C"
