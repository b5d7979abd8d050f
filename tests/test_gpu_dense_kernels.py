"""Sizes chosen by the kernel they take: every kernel of the dense operators, K whole and split,
against the fp64 forms.  test_dense_coverage_cpu.py checks that these lists (with SHAPES and BLOCKS)
leave no compiled kernel out.

Few-token sizes walk: more groups of weight rows than workgroups, the last one ragged, and K of two
and three passes where the kernel takes several.
"""
import numpy as np
import pytest
import torch

from oracle import dense_oracle as D
from test_gpu_dense import (BF16, F32, I8, NAME, TORCH, Ctx, Guarded, _blob, _check, _matmul, _views, f64, normal,
                            same_bits)
from test_gpu_dense import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

# (rows, cols): 256 threads a row and 1024, each with 1, 2 and 4 vectors of 8 held, and beyond
ROWS = [(5, 4112), (2, 9008), (3, 17008), (600, 1040), (600, 2064), (600, 4112), (520, 8208), (7, 40000)]
# T, N, K of the 8-bit product
FEW_PRODUCTS = [(1, 643, 11072), (1, 5003, 4080), (2, 5001, 9008), (3, 1030, 5120), (6, 2003, 4144), (7, 4099, 4080),
                (8, 8209, 4080), (1, 16403, 2064), (3, 24593, 8208), (5, 24593, 4112), (12, 8209, 2064), (16, 513, 2048),
                (10, 16427, 4112), (13, 24593, 8208), (25, 1003, 1040), (25, 8003, 4144)]
TILE_PRODUCTS = [(565, 14648, 144), (66, 8469, 5376), (814, 10720, 1232), (2000, 1003, 4096), (300, 777, 1040)]
# T, H, I of the block, few tokens (forward pass)
FEW_BLOCKS = {
    F32: [(1, 4160, 1056), (2, 4160, 800), (3, 1024, 4160), (3, 2112, 12320), (3, 8256, 992), (5, 24640, 1056),
          (10, 1024, 4160), (10, 8256, 992), (11, 24640, 1056), (12, 2112, 8224), (9, 16448, 1056), (14, 1088, 12320),
          (20, 1088, 1056), (27, 1024, 1024)],
    BF16: [(1, 4096, 12288), (2, 4160, 800), (2, 4160, 2080), (3, 2048, 4160), (3, 2112, 12320), (3, 8256, 992),
           (5, 24640, 2080), (10, 2048, 4160), (10, 8256, 992), (11, 24640, 2080), (12, 2112, 8224), (9, 16448, 2080),
           (14, 2112, 12320), (20, 2112, 2080), (27, 1024, 1024)],
}
# T, H, I of the block, forward and backward pass
TILE_BLOCKS = {
    F32: [(206, 448, 9664), (2302, 2176, 256), (3023, 256, 4128), (4123, 256, 1568), (4585, 2752, 224), (760, 1600, 3648),
          (2048, 2048, 4096)],
    BF16: [(194, 4288, 4288), (4790, 896, 448), (4096, 2048, 768), (2839, 2752, 1344), (75, 6080, 11520)],
}
# T, H, I of the 8-bit block
BLOCKS8 = [(1, 4096, 12288), (2, 7872, 416), (8, 2368, 800), (11, 1024, 800), (8, 4096, 4128), (8, 4160, 800), (5, 4160, 12320),
           (12, 2112, 4160), (14, 4160, 12320), (9, 4160, 8224), (20, 4160, 800), (30, 2112, 800), (34, 1728, 160),
           (2148, 8192, 288), (4108, 256, 512), (194, 7296, 3104)]


def _on_gpu(seed, shape, dtype, scale):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(TORCH[dtype])


def _weights(seed, H, I, w):
    return (_on_gpu(seed, (I, H), w, 2 * H ** -0.5), _on_gpu(seed + 1, (I, H), w, H ** -0.5),
            _on_gpu(seed + 2, (H, I), w, I ** -0.5))


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("x", [F32, BF16])
@pytest.mark.parametrize("off", [0, 1])
def test_rows(B, rows, cols, x, off):
    rng = np.random.default_rng(rows + cols)
    flat = normal(rng, rows * cols + off, x)
    q, s = Guarded(rows * cols, torch.int8), Guarded(rows, torch.float32)
    with Ctx(B) as c:
        B.moe_i8_quantize(c.p, flat[off:], x, cols, rows, cols, q.t, s.t)
        torch.cuda.synchronize()
    rq, rs = D.quantize_rows(f64(flat[off:]).reshape(rows, cols))
    assert np.array_equal(s.t.cpu().numpy(), rs)
    assert np.array_equal(q.t.cpu().numpy().reshape(rows, cols), rq)
    q.check(), s.check()


@pytest.mark.parametrize("T,N,K", FEW_PRODUCTS + TILE_PRODUCTS)
@pytest.mark.parametrize("x_type,y_type", [(BF16, BF16), (F32, F32), (I8, BF16), (BF16, F32), (F32, BF16)])
def test_products(B, T, N, K, x_type, y_type):
    """Every result: the sums are whole numbers below 2^53, exact in a 64-bit product."""
    print(f"[products] T={T} N={N} K={K} x={x_type} y={y_type}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(T * 7 + N * 3 + K)
    wq = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=gen)
    ws = torch.rand(N, device="cuda", generator=gen) * 0.01 + 1e-4
    with Ctx(B) as c:
        if x_type == I8:
            x = torch.randint(-128, 128, (T, K), dtype=torch.int8, device="cuda", generator=gen)
            xs = torch.rand(T, device="cuda", generator=gen) * 0.1 + 1e-3
            codes, given = x.double(), xs
        else:
            x, given = _on_gpu(T + K, (T, K), x_type, 1.0), None
            q, s = D.quantize_rows(f64(x))
            codes, xs = torch.from_numpy(q).cuda().double(), torch.from_numpy(s).cuda()
        got = _matmul(B, c, x, x_type, K, given, T, wq, ws, N, K, y_type, N)
        again = _matmul(B, c, x, x_type, K, given, T, wq, ws, N, K, y_type, N)
    assert same_bits(got, again)
    ref = torch.mm(codes, wq.double().t()) * xs.double()[:, None] * ws.double()
    _check("y", f64(got), f64(ref), D.i8_bound(f64(ref), NAME[y_type]))


def _saved(save, T, I, w):
    """Pre-activations (gate, up) and h as the forward pass kept them, in fp64."""
    n = T * 2 * I
    if w == F32:
        gu = f64(save[: 4 * n].view(torch.float32))
        end = 4 * n
    else:
        hi = save[: 2 * n].view(torch.int16).cpu().numpy().astype(np.int64) & 0xFFFF
        low = (2 * n + 255) // 256 * 256
        lo = save[low: low + n].cpu().numpy().astype(np.int64)
        gu = (hi << 16 | lo << 8).astype(np.uint32).view(np.float32).astype(np.float64)
        end = low + n
    at = (end + 255) // 256 * 256
    h = f64(save[at: at + T * I * (4 if w == F32 else 2)].view(TORCH[w])).reshape(T, I)
    gu = gu.reshape(T, I // 16, 2, 16)
    return gu[:, :, 0].reshape(T, I), gu[:, :, 1].reshape(T, I), h


@pytest.mark.parametrize("w,T,H,I", [(w, *s) for w in (F32, BF16) for s in FEW_BLOCKS[w]])
def test_few_tokens_block(B, w, T, H, I):
    print(f"[few_tokens_block] w={w} T={T} H={H} I={I}", flush=True)
    x = _on_gpu(T + H, (T, H), w, 1.0)
    wg, wu, wd = _weights(T * 5 + I, H, I, w)
    with Ctx(B, H, I, w) as c:
        blob = _blob(B, c, wg, wu, wd)
        work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        y, y2 = Guarded(T * H, TORCH[w]), Guarded(T * H, TORCH[w])
        save = Guarded(B.moe_dense_save_bytes(c.cfg, T), torch.uint8)
        B.moe_dense_ffn(c.p, x, T, blob, None, y2.t, work)
        B.moe_dense_ffn(c.p, x, T, blob, save.t, y.t, work)
        torch.cuda.synchronize()
        for g in (y, y2, save):
            g.check()
    assert same_bits(y.t, y2.t)
    args = [f64(t) for t in (x, wg, wu, wd)]
    ref, (g, u, _, _) = D.block(*args)
    _check("y", f64(y.t).reshape(T, H), ref, D.block_bounds(None, *args, NAME[w])["y"])
    kg, ku, kh = _saved(save.t, T, I, w)
    for name, got, want, m in (("gate", kg, g, args[1]), ("up", ku, u, args[2])):
        e = H * 1.01 * D.F32_HALF * (np.abs(args[0]) @ np.abs(m).T)
        _check(name, got, want, e + (np.abs(want) + e) * D.KEPT[NAME[w]])
    # h against the kept values, which are those it came from less a cut of KEPT of each (silu' is 1.1
    # at most, so either cut moves h by 1.1 |gate up| KEPT), then the sigmoid's error and one rounding
    kept, want = D.KEPT[NAME[w]], kg * D.sigmoid(kg) * ku
    e = np.abs(kg * ku) * (2.2 * kept + D.SIGMOID_REL)
    _check("h", kh, want, e + (np.abs(want) + e) * (D.HALF[NAME[w]] + 4 * D.F32_HALF))


@pytest.mark.parametrize("w,T,H,I", [(w, *s) for w in (F32, BF16) for s in TILE_BLOCKS[w]])
def test_tiled_block(B, w, T, H, I):
    """48 rows of y and dx and the gradients of 48 inner indices, elementwise; all results finite,
    nothing beside them written."""
    print(f"[tiled_block] w={w} T={T} H={H} I={I}", flush=True)
    rng = np.random.default_rng(T)
    x, dy = _on_gpu(T, (T, H), w, 1.0), _on_gpu(T + 1, (T, H), w, 0.1)
    wg, wu, wd = _weights(T + 2, H, I, w)
    with Ctx(B, H, I, w) as c:
        blob = _blob(B, c, wg, wu, wd)
        work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        y, dx, grad = Guarded(T * H, TORCH[w]), Guarded(T * H, TORCH[w]), Guarded(blob.numel(), torch.uint8)
        save = Guarded(B.moe_dense_save_bytes(c.cfg, T), torch.uint8)
        B.moe_dense_ffn(c.p, x, T, blob, save.t, y.t, work)
        B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save.t, dx.t, grad.t, work)
        torch.cuda.synchronize()
        for g in (y, dx, grad, save):
            g.check()
        gu, d = _views(grad.t, H, I, TORCH[w])
        for t in (y.t, dx.t, gu, d):
            assert torch.isfinite(t.float()).all()
        first = [t.clone() for t in (dx.t, gu, d)]
        B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save.t, dx.t, grad.t, work)
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(first, (dx.t, gu.contiguous(), d.contiguous()))), "runs differ"
    rows = np.unique(np.minimum(np.r_[0, 63, 64, 127, 128, 255, 256, T - 1, rng.integers(0, T, 40)], T - 1))
    r = torch.from_numpy(rows).cuda()
    args = [f64(t) for t in (x[r], wg, wu, wd)]
    bounds = D.block_bounds(f64(dy[r]), *args, NAME[w])
    _check("y", f64(y.t.view(T, H)[r]), D.block(*args)[0], bounds["y"])
    _check("dx", f64(dx.t.view(T, H)[r]), D.block_backward(f64(dy[r]), *args)[0], bounds["dx"])
    inner = np.unique(np.minimum(np.r_[0, 31, 32, 63, 64, 127, 128, I - 1, rng.integers(0, I, 40)], I - 1))
    k = torch.from_numpy(inner).cuda()
    args = [f64(t) for t in (x, wg[k], wu[k], wd[:, k].contiguous())]
    bounds = D.block_bounds(f64(dy), *args, NAME[w])
    _, rg, ru, rd = D.block_backward(f64(dy), *args)
    at = k // 16 * 32 + k % 16
    _check("dwg", f64(gu[at]), rg, bounds["dwg"])
    _check("dwu", f64(gu[at + 16]), ru, bounds["dwu"])
    _check("dwd", f64(d[:, k]), rd, bounds["dwd"])


@pytest.mark.parametrize("T,H,I", BLOCKS8)
def test_i8_blocks(B, T, H, I):
    """Elementwise, up to 64 rows: h is within 2^-17 of its size, so a code moves by one where its
    quotient lies within 127 * 2^-16 of a border and each term by 2^-16 with its scale; the rest is
    the result's rounding."""
    print(f"[i8_blocks] T={T} H={H} I={I}", flush=True)
    x = _on_gpu(T + H, (T, H), BF16, 1.0)
    wg, wu, wd = _weights(T * 5 + I, H, I, BF16)
    with Ctx(B, H, I) as c:
        b8 = torch.empty(B.moe_i8_blob_bytes(c.cfg), dtype=torch.uint8, device="cuda")
        B.moe_i8_pack(c.p, _blob(B, c, wg, wu, wd), b8)
        work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        y, y2 = Guarded(T * H, torch.bfloat16), Guarded(T * H, torch.bfloat16)
        B.moe_i8_ffn(c.p, x, T, b8, y.t, work)
        B.moe_i8_ffn(c.p, x, T, b8, y2.t, work)
        torch.cuda.synchronize()
        y.check(), y2.check()
    assert same_bits(y.t, y2.t)
    rows = np.arange(T) if T <= 64 else np.unique(np.r_[0, 127, 128, T - 1, np.random.default_rng(T).integers(0, T, 60)])
    q = [v for m in (wg, wu, wd) for v in D.quantize_rows(f64(m))]
    ref, (h, hs) = D.i8_block(f64(x)[rows], *q)
    step = hs.astype(np.float64)[:, None]
    quot = h / np.where(step > 0, step, 1)
    near = (np.abs(quot - np.floor(quot) - 0.5) <= 127 * 2.0 ** -16) * step
    wdeq = np.abs(q[4].astype(np.float64)) * q[5].astype(np.float64)[:, None]
    bound = near @ wdeq.T + np.abs(ref) * (2.0 ** -16 + 2.0 ** -8) + 2.0 ** -16 * (step * 0.5 * wdeq.sum(1))
    _check("y", f64(y.t).reshape(T, H)[rows], ref, bound)
