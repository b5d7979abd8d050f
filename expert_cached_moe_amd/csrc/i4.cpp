// Entry points of the products with 4-bit weights: quantisation, the dense product, and the experts
// of a layer.  Contracts in include/moe.h; the kernels are in i4_quant.hip, i4_few.hip,
// i4_mid.hip and i4_turns.hip.
#include <hip/hip_runtime.h>

#include "dense.h"
#include "i4.h"

namespace moe {
namespace {

using namespace i4;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool group_ok(int32_t g) { return g == 32 || g == 64 || g == 128; }
int shift_of(int32_t g) { return g == 32 ? 5 : g == 64 ? 6 : 7; }

// Blob of an expert: the parts of its interleaved gate and up rows, then those of its down rows.
struct Blob4 {
    int64_t gu = 0, gu_word = 0, gu_exp = 0, d = 0, d_word = 0, d_exp = 0, bytes = 0;
    int32_t gu_groups = 0, d_groups = 0;
};
Blob4 blob4_layout(const moe_config& c, int32_t group) {
    const int64_t H = c.hidden, I = c.inter;
    Blob4 b;
    b.gu_groups = int32_t((H + group - 1) / group);
    b.d_groups = int32_t((I + group - 1) / group);
    b.gu_word = align256(2 * I * (H / 2));
    b.gu_exp = align256(b.gu_word + 2 * I * b.gu_groups * 2);
    b.d = align256(b.gu_exp + 2 * I);
    b.d_word = align256(b.d + H * (I / 2));
    b.d_exp = align256(b.d_word + H * b.d_groups * 2);
    b.bytes = align256(b.d_exp + H);
    return b;
}

// Workspace of moe_i4_expert_ffn: the tile maps of the two products, and h in expert order.
int64_t map_bytes(int n, int64_t rows) { return align256(16 * (1 + map_tiles(n, rows, 32))); }
struct ExpertWork {
    int64_t h = 0, bytes = 0;
};
ExpertWork expert_work(const moe_config& c, int64_t T) {
    if (T < 1) T = 1;
    const int64_t rows = T * c.top_k + (c.n_shared ? T : 0);
    ExpertWork w;
    w.h = align256(2 * map_bytes(c.n_experts + 1, rows));
    w.bytes = align256(w.h + rows * c.inter * 2);
    return w;
}

hipError_t launch_dense(int what, const Product& p, hipStream_t s) {
    const int n_cu = dense::compute_units();
    if (few_dense(p.T, p.N, p.K, n_cu)) return launch_i4_few(what, p, nullptr, s);
    const int kind = plan_dense(p.T, p.N, p.K, p.planes, n_cu);
    return kind == kTurns ? launch_i4_turns(what, p, nullptr, nullptr, 0, s) : launch_i4_mid(what, kind, p, nullptr, nullptr, 0, s);
}

int check_config(const moe_config& c, const char** why) {
    if (c.w_dtype != MOE_W_BF16) {
        *why = "4-bit blobs are made from and for bf16 contexts";
        return MOE_EUNSUPPORTED;
    }
    if (c.hidden > kMaxK || c.inter > kMaxK) {
        *why = "4-bit blobs take H and I up to 2^20";
        return MOE_ESHAPE;
    }
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;
using namespace moe::i4;

extern "C" {

int moe_i4_quantize(moe_ctx* ctx, const void* d_x, int32_t x_type, int64_t ld_x, int32_t rows, int32_t cols, int32_t group,
                    int32_t zero_points, uint8_t* d_q, uint16_t* d_words, uint8_t* d_exps, hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    if (rows < 0) return fail(ctx, MOE_EINVAL, "rows < 0");
    if (x_type != MOE_A_F32 && x_type != MOE_A_BF16) return fail(ctx, MOE_EINVAL, "x must be fp32 or bf16");
    if (!group_ok(group)) return fail(ctx, MOE_EINVAL, "groups have 32, 64 or 128 weights");
    if (zero_points != 0 && zero_points != 1) return fail(ctx, MOE_EINVAL, "zero_points must be 0 or 1");
    if (cols < 32 || cols % 32 || cols > kMaxK || rows > kMaxCount)
        return fail(ctx, MOE_ESHAPE, "cols must be a multiple of 32 in 32..2^20, rows up to 2^23");
    if (ld_x < cols) return fail(ctx, MOE_EINVAL, "ld_x < cols");
    if (rows == 0) return MOE_OK;
    if (!d_x || !d_q || !d_words || !d_exps) return fail(ctx, MOE_EINVAL, "null buffer");
    if (!aligned(d_x, x_type == MOE_A_F32 ? 4 : 2) || !aligned(d_q, 16) || !aligned(d_words, 2))
        return fail(ctx, MOE_EINVAL, "misaligned buffer");
    hipError_t e = launch_i4_quantize(d_x, x_type, ld_x, rows, cols, group, zero_points, d_q, d_words, d_exps, s);
    return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_i4_quantize launch");
}

int64_t moe_i4_workspace_bytes(int32_t max_T, int32_t N, int32_t K) {
    if (max_T < 0) return MOE_EINVAL;
    if (K < 32 || K % 32 || K > kMaxK || N < 1 || N > kMaxCount || max_T > kMaxCount) return MOE_ESHAPE;
    return align256(int64_t(max_T < 1 ? 1 : max_T) * K * 6);
}

int moe_i4_matmul(moe_ctx* ctx, const void* d_x, int32_t x_type, int64_t ld_x, int32_t T, const uint8_t* d_w,
                  const uint16_t* d_words, const uint8_t* d_exps, int32_t N, int32_t K, int32_t group, void* d_y,
                  int32_t y_type, int64_t ld_y, void* d_ws, hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    if (T < 0) return fail(ctx, MOE_EINVAL, "T < 0");
    if (x_type != MOE_A_F32 && x_type != MOE_A_BF16) return fail(ctx, MOE_EINVAL, "x must be fp32 or bf16");
    if (y_type != MOE_A_F32 && y_type != MOE_A_BF16) return fail(ctx, MOE_EINVAL, "y must be fp32 or bf16");
    if (!group_ok(group)) return fail(ctx, MOE_EINVAL, "groups have 32, 64 or 128 weights");
    if (K < 32 || K % 32 || K > kMaxK) return fail(ctx, MOE_ESHAPE, "K must be a multiple of 32 in 32..2^20");
    if (N < 1 || N > kMaxCount || T > kMaxCount) return fail(ctx, MOE_ESHAPE, "N in 1..2^23, T up to 2^23");
    if (ld_x < K) return fail(ctx, MOE_EINVAL, "ld_x < K");
    if (ld_y < N) return fail(ctx, MOE_EINVAL, "ld_y < N");
    if (int64_t(T) * N > int64_t(1) << 36) return fail(ctx, MOE_ESHAPE, "T N above 2^36");
    if (T == 0) return MOE_OK;
    if (!d_x || !d_w || !d_words || !d_exps || !d_y || !d_ws) return fail(ctx, MOE_EINVAL, "null buffer");
    if (!aligned(d_x, x_type == MOE_A_F32 ? 4 : 2) || !aligned(d_w, 16) || !aligned(d_words, 2) ||
        !aligned(d_y, y_type == MOE_A_F32 ? 4 : 2) || !aligned(d_ws, 256))
        return fail(ctx, MOE_EINVAL, "misaligned buffer");
    Product p{};
    p.planes = 1;
    p.x = static_cast<const uint16_t*>(d_x);
    p.ldx = ld_x;
    p.T = T;
    // (rows that are read as they are start on 16 bytes each, and 128 of them lie within 4 GiB)
    if (x_type == MOE_A_F32 || !aligned(d_x, 16) || ld_x % 8 || ld_x >= (int64_t(1) << 24)) {
        hipError_t e = launch_i4_activations(d_x, x_type, ld_x, T, K, static_cast<uint16_t*>(d_ws), s);
        if (e != hipSuccess) return hip_fail(ctx, e, "moe_i4_matmul launch");
        p.x = static_cast<const uint16_t*>(d_ws);
        p.ldx = K;
        p.plane = int64_t(T) * K;
        p.planes = x_type == MOE_A_F32 ? 3 : 1;
    }
    p.N = N;
    p.K = K;
    p.w = Rows{d_w, d_words, d_exps, (K + group - 1) / group, shift_of(group)};
    p.out = d_y;
    p.ldo = ld_y;
    const int kind = y_type == MOE_A_F32 ? kOut32 : kOut16;
    hipError_t e = launch_dense(kind, p, s);
    return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_i4_matmul launch");
}

int64_t moe_i4_blob_bytes(const moe_config* cfg, int32_t group) {
    int st = validate_config(cfg, nullptr);
    const char* why;
    if (st == MOE_OK) st = check_config(*cfg, &why);
    if (st != MOE_OK) return st;
    if (!group_ok(group)) return MOE_EINVAL;
    return blob4_layout(*cfg, group).bytes;
}

int moe_i4_pack(moe_ctx* ctx, const void* d_blob, int32_t group, int32_t zero_points, void* d_blob4, hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    const moe_config& c = ctx->cfg;
    const char* why;
    const int st = check_config(c, &why);
    if (st != MOE_OK) return fail(ctx, st, why);
    if (!group_ok(group)) return fail(ctx, MOE_EINVAL, "groups have 32, 64 or 128 weights");
    if (zero_points != 0 && zero_points != 1) return fail(ctx, MOE_EINVAL, "zero_points must be 0 or 1");
    if (!d_blob || !d_blob4) return fail(ctx, MOE_EINVAL, "null buffer");
    if (!aligned(d_blob, 256) || !aligned(d_blob4, 256)) return fail(ctx, MOE_EINVAL, "blobs must be 256-byte aligned");
    const Blob4 b = blob4_layout(c, group);
    const uint8_t* src = static_cast<const uint8_t*>(d_blob);
    uint8_t* dst = static_cast<uint8_t*>(d_blob4);
    hipError_t e = launch_i4_quantize(src + ctx->lay.gu, MOE_A_BF16, c.hidden, 2 * int64_t(c.inter), c.hidden, group,
                                      zero_points, dst + b.gu, reinterpret_cast<uint16_t*>(dst + b.gu_word), dst + b.gu_exp, s);
    if (e == hipSuccess)
        e = launch_i4_quantize(src + ctx->lay.d, MOE_A_BF16, c.inter, c.hidden, c.inter, group, zero_points, dst + b.d,
                               reinterpret_cast<uint16_t*>(dst + b.d_word), dst + b.d_exp, s);
    return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_i4_pack launch");
}

int64_t moe_i4_expert_workspace_bytes(const moe_config* cfg, int32_t max_T) {
    int st = validate_config(cfg, nullptr);
    const char* why;
    if (st == MOE_OK) st = check_config(*cfg, &why);
    if (st != MOE_OK) return st;
    if (max_T < 0) return MOE_EINVAL;
    if (max_T > kMaxCount) return MOE_ESHAPE;
    return expert_work(*cfg, max_T).bytes;
}

int moe_i4_expert_ffn(moe_ctx* ctx, const void* d_x, int32_t T, const int32_t* d_offsets, const int32_t* d_perm,
                      const void* d_slot_base, const int32_t* h_experts, const int32_t* h_slots, int32_t n,
                      const void* d_shared, int32_t with_shared, int32_t group, void* d_o, void* d_ws, hipStream_t s) {
    if (!ctx) return MOE_EINVAL;
    const moe_config& c = ctx->cfg;
    const char* why;
    const int st = check_config(c, &why);
    if (st != MOE_OK) return fail(ctx, st, why);
    if (T < 0) return fail(ctx, MOE_EINVAL, "T < 0");
    if (T > kMaxCount) return fail(ctx, MOE_ESHAPE, "T above 2^23");
    if (n < 0 || n > c.n_experts) return fail(ctx, MOE_EINVAL, "n must be in 0..E");
    if (with_shared != 0 && with_shared != 1) return fail(ctx, MOE_EINVAL, "with_shared must be 0 or 1");
    if (with_shared && (!c.n_shared || !d_shared)) return fail(ctx, MOE_EINVAL, "no shared expert");
    if (!group_ok(group)) return fail(ctx, MOE_EINVAL, "groups have 32, 64 or 128 weights");
    if (n > 0 && (!h_experts || !h_slots)) return fail(ctx, MOE_EINVAL, "null expert list");
    ExpertList list;
    list.n = 0;
    uint32_t seen[kMaxExperts / 32] = {0};
    for (int i = 0; i < n; ++i) {
        const int e = h_experts[i], sl = h_slots[i];
        if (e < 0 || e >= c.n_experts || seen[e / 32] >> e % 32 & 1)
            return fail(ctx, MOE_EINVAL, "expert id out of range or repeated");
        if (sl < 0 || sl >= (1 << 21)) return fail(ctx, MOE_EINVAL, "slot out of range");
        seen[e / 32] |= 1u << e % 32;
        list.ent[list.n++] = e | (sl << 10);
    }
    if (with_shared) list.ent[list.n++] = kSharedTag;
    if (T == 0 || list.n == 0) return MOE_OK;
    if (!d_x || !d_o || !d_ws) return fail(ctx, MOE_EINVAL, "null buffer");
    if (n > 0 && (!d_offsets || !d_perm || !d_slot_base)) return fail(ctx, MOE_EINVAL, "null routed-expert argument");
    if (!aligned(d_x, 16) || !aligned(d_o, 16) || !aligned(d_ws, 256) || !aligned(d_slot_base, 256) || !aligned(d_shared, 256))
        return fail(ctx, MOE_EINVAL, "misaligned buffer");
    const Blob4 b = blob4_layout(c, group);
    const ExpertWork w = expert_work(c, T);
    uint8_t* ws = static_cast<uint8_t*>(d_ws);
    const uint8_t* base = static_cast<const uint8_t*>(n > 0 ? d_slot_base : d_shared);
    Product p{};
    p.planes = 1;
    p.T = T;
    p.offsets = d_offsets;
    p.perm = d_perm;
    p.top_k = c.top_k;
    p.stride = b.bytes;
    p.shared = with_shared ? static_cast<const uint8_t*>(d_shared) - base : 0;
    const int64_t pairs = int64_t(T) * c.top_k, rows = (n > 0 ? pairs : 0) + (with_shared ? T : 0);
    const int n_cu = dense::compute_units();
    const bool few = T <= kFewTokens;
    int built = 0;                                            // rows of the tiles that the map in the workspace lists
    auto product = [&](int what) {
        if (few) return launch_i4_few(what, p, &list, s);
        int kind = plan_experts(list.n, rows, p.N, p.K, n_cu);
        // (offsets of gathered rows have 32 bits on the smaller tiles)
        if (what == kGateUp && int64_t(T) * p.ldx * 2 > int64_t(0xFFFF0000)) kind = kTurns;
        uint8_t* map = ws + (what == kDown && built != kKind[kind].rows ? map_bytes(c.n_experts + 1, pairs + (c.n_shared ? T : 0)) : 0);
        if (built != kKind[kind].rows) {
            const hipError_t e = launch_i4_map(list, d_offsets, T, c.top_k, kKind[kind].rows, map, s);
            if (e != hipSuccess) return e;
            built = kKind[kind].rows;
        }
        const int64_t tiles = map_tiles(list.n, rows, kKind[kind].rows);
        return kind == kTurns ? launch_i4_turns(what, p, &list, map, tiles, s) : launch_i4_mid(what, kind, p, &list, map, tiles, s);
    };
    p.x = static_cast<const uint16_t*>(d_x);
    p.ldx = c.hidden;
    p.N = 2 * c.inter;
    p.K = c.hidden;
    p.w = Rows{base + b.gu, reinterpret_cast<const uint16_t*>(base + b.gu_word), base + b.gu_exp, b.gu_groups, shift_of(group)};
    p.out = ws + w.h;
    p.ldo = c.inter;
    hipError_t e = product(kGateUp);
    if (e != hipSuccess) return hip_fail(ctx, e, "moe_i4_expert_ffn launch");
    p.x = reinterpret_cast<const uint16_t*>(ws + w.h);
    p.ldx = c.inter;
    p.N = c.hidden;
    p.K = c.inter;
    p.w = Rows{base + b.d, reinterpret_cast<const uint16_t*>(base + b.d_word), base + b.d_exp, b.d_groups, shift_of(group)};
    p.out = d_o;
    p.ldo = c.hidden;
    e = product(kDown);
    return e == hipSuccess ? MOE_OK : hip_fail(ctx, e, "moe_i4_expert_ffn launch");
}

}  // extern "C"
