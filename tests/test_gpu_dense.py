"""GPU parity of the dense operators against their fp64 forms: 8-bit quantisation and products,
the gated block with its backward pass, the 8-bit block, and the three used together.

Every output is held elementwise to a worst-case bound of the documented arithmetic, computed
from the data (oracle.dense_oracle).  Outputs lie between guard values that must survive.
"""
import numpy as np
import pytest
import torch

from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu

F32, BF16, I8 = 0, 1, 2
TORCH = {F32: torch.float32, BF16: torch.bfloat16, I8: torch.int8}
NAME = {F32: "f32", BF16: "bf16"}
GUARD = 64


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from expert_cached_moe_amd import binding
    return binding


class Ctx:
    def __init__(self, B, H=64, I=32, w=BF16):
        self.B, self.cfg = B, B.make_config(H, I, 1, 1, w_dtype=w)
        self.p = B.moe_create(self.cfg)

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.B.moe_destroy(self.p)


class Guarded:
    """A buffer of n elements between two runs of guard values (NaN, or -77 for integers)."""

    def __init__(self, n, dtype):
        self.pad = 256 // torch.empty((), dtype=dtype).element_size()
        self.fill = float("nan") if dtype.is_floating_point else (77 if dtype == torch.uint8 else -77)
        self.all = torch.full((n + 2 * self.pad,), self.fill, dtype=dtype, device="cuda")
        self.t = self.all[self.pad: self.pad + n]

    def check(self):
        for g in (self.all[: self.pad], self.all[-self.pad:]):
            ok = torch.isnan(g) if g.dtype.is_floating_point else g == self.fill
            assert ok.all(), "written outside the buffer"


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(TORCH[dtype]).cuda()


def same_bits(a, b):
    return torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols,ld,off", [(1, 16, 16, 0), (3, 48, 48, 0), (7, 2048, 2048, 0), (5, 2064, 2071, 0),
                                              (4, 2048, 2064, 3), (2, 16384, 16384, 0), (2, 40000, 40008, 8),
                                              (1500, 64, 64, 0)])
def test_quantize(B, dtype, rows, cols, ld, off):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = normal(rng, rows * ld + off, dtype)
    x[::977] *= 30
    view = x[off:].as_strided((rows, cols), (ld, 1))
    q, s = Guarded(rows * cols, torch.int8), Guarded(rows, torch.float32)
    with Ctx(B) as c:
        B.moe_i8_quantize(c.p, x[off:], dtype, ld, rows, cols, q.t, s.t)
        torch.cuda.synchronize()
    rq, rs = D.quantize_rows(f64(view))
    assert np.array_equal(s.t.cpu().numpy(), rs)
    assert np.array_equal(q.t.cpu().numpy().reshape(rows, cols), rq)
    q.check(), s.check()


def test_quantize_half_way_and_special_rows(B):
    """Exact half-way quotients, quotients one step of fp32 beside them, zeros, numbers whose
    scale is too small for fp32, infinities and NaNs."""
    rng = np.random.default_rng(3)
    rows = []
    for top in (127.0, 254.0, 127.0 * 2.0 ** -60, 3.0, 1e30, 7e-30, 3.3e38, 1.6e-36):
        s = np.float32(float(np.float32(top)) / 127.0)
        half = (np.float64(s) * (rng.integers(-127, 127, 60) + 0.5)).astype(np.float32)
        rows.append(np.concatenate([[np.float32(top)], half, np.nextafter(half, np.float32(np.inf)),
                                    np.nextafter(half, -np.float32(np.inf)), np.zeros(11, np.float32)]))
        rows[-1] = np.clip(rows[-1], -np.float32(top), np.float32(top))
    z = np.zeros((6, 192), np.float32)
    z[1, 7], z[2, 100], z[3, 0], z[4, 191] = np.inf, -np.inf, np.nan, 1e-40
    z[1:4, 50] = 4.0
    z[5, 3] = -5.0
    x = np.concatenate([np.stack(rows), z]).astype(np.float32)
    d = torch.from_numpy(x).cuda()
    q, s = Guarded(x.size, torch.int8), Guarded(len(x), torch.float32)
    with Ctx(B) as c:
        B.moe_i8_quantize(c.p, d, F32, 192, len(x), 192, q.t, s.t)
        torch.cuda.synchronize()
    rq, rs = D.quantize_rows(x)
    assert np.array_equal(s.t.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.t.cpu().numpy().reshape(x.shape), rq)


# ---------------------------------------------------------------- 8-bit product

def _matmul(B, c, x, x_type, ldx, xs, T, wq, ws, N, K, y_type, ldy, stream=None):
    y = Guarded((T - 1) * ldy + N, TORCH[y_type])
    work = torch.full((B.moe_i8_workspace_bytes(T, K),), 0xA5, dtype=torch.uint8, device="cuda")
    B.moe_i8_matmul(c.p, x, x_type, ldx, xs, T, wq, ws, N, K, y.t, y_type, ldy, work, stream)
    torch.cuda.synchronize()
    y.check()
    out = torch.full((T * ldy,), float("nan"), dtype=TORCH[y_type], device="cuda")
    out[: y.t.numel()] = y.t
    out = out.view(T, ldy)
    assert torch.isnan(out[:, N:]).all(), "written between the rows"
    return out[:, :N]


SHAPES = [(1, 64, 16), (1, 2048, 2048), (1, 1, 16), (2, 17, 48), (3, 2051, 1552), (5, 33, 4096), (8, 4099, 4096),
          (8, 16, 131056), (9, 100, 80), (15, 129, 1040), (16, 513, 2048), (17, 300, 336), (31, 64, 64), (33, 1000, 2064),
          (64, 2048, 768), (65, 255, 144), (100, 257, 400), (128, 128, 128), (129, 131, 272), (255, 1025, 112),
          (257, 513, 1552), (300, 70, 16400), (777, 2051, 1552), (1024, 1536, 2048), (2048, 256, 64)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("x_type,y_type,pad", [(BF16, BF16, 0), (F32, F32, 3), (I8, F32, 0), (BF16, F32, 16)])
def test_i8_matmul(B, T, N, K, x_type, y_type, pad):
    print(f"[i8_matmul] T={T} N={N} K={K} x={x_type} y={y_type} pad={pad}", flush=True)
    rng = np.random.default_rng(T * 7 + N * 3 + K)
    wq = rng.integers(-128, 128, (N, K), dtype=np.int8)
    ws = (rng.random(N) * 0.01 + 1e-4).astype(np.float32)
    dw, dws = torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda()
    with Ctx(B) as c:
        if x_type == I8:
            xq = rng.integers(-128, 128, (T, K), dtype=np.int8)
            xs = (rng.random(T) * 0.1 + 1e-3).astype(np.float32)
            x, dxs, ldx = torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), K
        else:
            ldx, dxs = K + pad, None
            x = normal(rng, (T, ldx), x_type)
            xq, xs = D.quantize_rows(f64(x[:, :K]))
        got = _matmul(B, c, x, x_type, ldx, dxs, T, dw, dws, N, K, y_type, N + pad)
        again = _matmul(B, c, x, x_type, ldx, dxs, T, dw, dws, N, K, y_type, N + pad)
    assert same_bits(got.contiguous(), again.contiguous())
    ref = D.i8_matmul(xq, xs, wq, ws)
    err = np.abs(f64(got) - ref)
    bound = D.i8_bound(ref, NAME[y_type])
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:4])


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_i8_matmul_extreme_codes(B, T):
    """All codes -128: the sums reach 128 * 128 * K = 2^31 - 2^18."""
    K, N = 131056, 35
    xq = np.full((T, K), -128, np.int8)
    wq = np.full((N, K), -128, np.int8)
    wq[1::2] = 127
    with Ctx(B) as c:
        got = _matmul(B, c, torch.from_numpy(xq).cuda(), I8, K, torch.ones(T, device="cuda"), T,
                      torch.from_numpy(wq).cuda(), torch.ones(N, device="cuda"), N, K, F32, N)
    ref = D.i8_matmul(xq, np.ones(T, np.float32), wq, np.ones(N, np.float32))
    assert (np.abs(f64(got) - ref) <= D.i8_bound(ref, "f32")).all()


@pytest.mark.parametrize("T", [1, 6, 20, 200])
def test_i8_matmul_special_rows(B, T):
    """Rows with NaN or infinity give NaN rows, zero rows zeros; the others are unchanged."""
    rng = np.random.default_rng(T)
    K, N = 272, 45
    x = normal(rng, (T, K), F32)
    x[T // 2] = 0
    if T > 3:
        x[1, 5], x[3, 270] = float("nan"), float("-inf")
    wq = rng.integers(-127, 128, (N, K), dtype=np.int8)
    ws = np.full(N, 0.01, np.float32)
    with Ctx(B) as c:
        got = f64(_matmul(B, c, x, F32, K, None, T, torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda(), N, K, F32, N))
    xq, xs = D.quantize_rows(f64(x))
    ref = D.i8_matmul(xq, xs, wq, ws)
    bad = np.isnan(xs)
    assert np.isnan(got[bad]).all()
    assert (np.abs(got[~bad] - ref[~bad]) <= D.i8_bound(ref[~bad], "f32")).all()
    assert not got[xs == 0].any()


@pytest.mark.parametrize("T", [1, 6, 20, 200, 2100])
def test_i8_matmul_far_scales(B, T):
    """Scales of x up to 2.4e36 with scales of W near 1e-31, and small ones with large ones: sum *
    scale leaves fp32 where sum * scale * scale does not."""
    rng = np.random.default_rng(T)
    K, N = 1040, 133
    for far, near in ((3e38, 1e-31), (1e30, 1e-24), (1e-34, 1e20)):
        x = normal(rng, (T, K), F32)
        x *= far / x.abs().amax(1, keepdim=True)
        wq = rng.integers(-127, 128, (N, K), dtype=np.int8)
        ws = ((rng.random(N) + 0.5) * near).astype(np.float32)
        with Ctx(B) as c:
            got = f64(_matmul(B, c, x, F32, K, None, T, torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda(), N, K,
                              F32, N))
        xq, xs = D.quantize_rows(f64(x))
        ref = D.i8_matmul(xq, xs, wq, ws)
        assert (np.abs(got - ref) <= D.i8_bound(ref, "f32")).all()


@pytest.mark.parametrize("T", [1, 40])
def test_i8_matmul_offsets_past_32_bits(B, T):
    """Weights of 4.6 GB, and rows of x and y more than 2^31 elements apart (T = 2)."""
    N, K = 140001, 32768
    gen = torch.Generator(device="cuda").manual_seed(T)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=gen)
    ws = torch.full((N,), 0.01, device="cuda")
    x = torch.randn((T, K), device="cuda", generator=gen)
    with Ctx(B) as c:
        got = f64(_matmul(B, c, x, F32, K, None, T, w, ws, N, K, F32, N))
    xq, xs = D.quantize_rows(f64(x))
    rows = np.r_[0:50, 65530:65550, 131060:131080, N - 50:N]
    ref = D.i8_matmul(xq, xs, w[torch.from_numpy(rows).cuda()].cpu().numpy(), np.full(len(rows), 0.01, np.float32))
    assert (np.abs(got[:, rows] - ref) <= D.i8_bound(ref, "f32")).all()


@pytest.mark.parametrize("T", [2, 11])
def test_i8_matmul_far_rows(B, T):
    far = (1 << 31) // (T - 1) + 64
    K, N = 64, 20
    rng = np.random.default_rng(1)
    x = torch.zeros(far * (T - 1) + K, dtype=torch.bfloat16, device="cuda")
    xv = x.as_strided((T, K), (far, 1))
    xv.copy_(normal(rng, (T, K), BF16))
    y = torch.zeros(far * (T - 1) + N, dtype=torch.bfloat16, device="cuda")
    wq = rng.integers(-127, 128, (N, K), dtype=np.int8)
    ws = np.full(N, 0.01, np.float32)
    work = torch.empty(B.moe_i8_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
    with Ctx(B) as c:
        B.moe_i8_matmul(c.p, x, BF16, far, None, T, torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda(), N, K, y,
                        BF16, far, work)
        torch.cuda.synchronize()
    xq, xs = D.quantize_rows(f64(xv))
    ref = D.i8_matmul(xq, xs, wq, ws)
    assert (np.abs(f64(y.as_strided((T, N), (far, 1))) - ref) <= D.i8_bound(ref, "bf16")).all()


# ---------------------------------------------------------------- gated block

def _blob(B, c, wg, wu, wd):
    """Device blob from natural-layout device weights, padding bytes 0xFF."""
    I, H = wg.shape
    es = wg.element_size()
    blob = torch.full((B.moe_expert_bytes(c.cfg),), 0xFF, dtype=torch.uint8, device="cuda")
    gu, d = _views(blob, H, I, wg.dtype)
    gu.copy_(torch.stack([wg.view(I // 16, 16, H), wu.view(I // 16, 16, H)], 1).reshape(2 * I, H))
    d.copy_(wd)
    return blob


def _views(blob, H, I, dtype):
    flat = blob.view(dtype)
    es = flat.element_size()
    d0 = (2 * I * H * es + 255) // 256 * 256 // es
    return flat[: 2 * I * H].view(2 * I, H), flat[d0: d0 + H * I].view(H, I)


def _block_inputs(rng, T, H, I, w):
    x, dy = normal(rng, (T, H), w), normal(rng, (T, H), w, 0.1)
    s = 1.0 / np.sqrt(H)
    return x, dy, normal(rng, (I, H), w, 2 * s), normal(rng, (I, H), w, s), normal(rng, (H, I), w, 1 / np.sqrt(I))


def _check(name, got, ref, bound):
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), name
    assert (err <= bound).all(), (name, float((err / bound).max()), np.argwhere(err > bound)[:4])


BLOCKS = [(1, 64, 32), (1, 128, 4096), (2, 192, 96), (3, 1024, 800), (7, 576, 1120), (8, 2048, 768), (9, 256, 160),
          (16, 64, 544), (17, 512, 256), (31, 320, 64), (33, 128, 128), (64, 256, 288), (65, 1088, 96), (100, 512, 800),
          (128, 256, 128), (129, 320, 416), (255, 64, 64), (256, 512, 512), (300, 576, 1120), (515, 1024, 736),
          (1000, 256, 352)]


@pytest.mark.parametrize("T,H,I", BLOCKS)
@pytest.mark.parametrize("w", [BF16, F32])
def test_block(B, T, H, I, w):
    print(f"[block] T={T} H={H} I={I} w={w}", flush=True)
    rng = np.random.default_rng(T + H + I)
    x, dy, wg, wu, wd = _block_inputs(rng, T, H, I, w)
    with Ctx(B, H, I, w) as c:
        blob = _blob(B, c, wg, wu, wd)
        work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        y, y2, dx = (Guarded(T * H, TORCH[w]) for _ in range(3))
        save = Guarded(B.moe_dense_save_bytes(c.cfg, T), torch.uint8)
        grad = Guarded(blob.numel(), torch.uint8)
        B.moe_dense_ffn(c.p, x, T, blob, None, y2.t, work)
        B.moe_dense_ffn(c.p, x, T, blob, save.t, y.t, work)
        B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save.t, dx.t, grad.t, work)
        torch.cuda.synchronize()
        for g in (y, y2, dx, save, grad):
            g.check()
        assert same_bits(y.t, y2.t), "y depends on the save buffer"
        dgu, dd = _views(grad.t, H, I, TORCH[w])
        pad = torch.full_like(grad.t, 0xFF)
        for v, p in zip((dgu, dd), _views(pad, H, I, TORCH[w])):
            p.copy_(v)
        first = grad.t.clone()
        gap = slice(2 * I * H * x.element_size(), (2 * I * H * x.element_size() + 255) // 256 * 256)
        assert (grad.t[gap] == 77).all(), "padding of the gradient blob written"
        dx1 = dx.t.clone()
        B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save.t, dx.t, grad.t, work)
        torch.cuda.synchronize()
        assert same_bits(dx1, dx.t) and same_bits(first, grad.t), "runs differ"
    args = [f64(t) for t in (x, wg, wu, wd)]
    bounds = D.block_bounds(f64(dy), *args, NAME[w])
    ref_dx, ref_dg, ref_du, ref_dd = D.block_backward(f64(dy), *args)
    _check("y", f64(y.t).reshape(T, H), D.block(*args)[0], bounds["y"])
    _check("dx", f64(dx.t).reshape(T, H), ref_dx, bounds["dx"])
    g, u = D.deinterleave(f64(dgu))
    _check("dwg", g, ref_dg, bounds["dwg"])
    _check("dwu", u, ref_du, bounds["dwu"])
    _check("dwd", f64(dd), ref_dd, bounds["dwd"])


# (the last three: products of one to three K slices on the largest tiles)
@pytest.mark.parametrize("T,H,I", [(4100, 4160, 4128), (2600, 8192, 2080), (40, 4096, 2560), (130, 4096, 4128), (8192, 64, 4096)])
def test_block_large(B, T, H, I):
    """Sizes that fill the chip with the largest tiles, with edges in each dimension: 48 rows of y
    and dx, and the gradients of 48 inner indices, against the formulas."""
    rng = np.random.default_rng(T)
    x, dy, wg, wu, wd = _block_inputs(rng, T, H, I, BF16)
    with Ctx(B, H, I, BF16) as c:
        blob = _blob(B, c, wg, wu, wd)
        work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        save = torch.full((B.moe_dense_save_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        y, dx = Guarded(T * H, torch.bfloat16), Guarded(T * H, torch.bfloat16)
        grad = Guarded(blob.numel(), torch.uint8)
        B.moe_dense_ffn(c.p, x, T, blob, save, y.t, work)
        B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save, dx.t, grad.t, work)
        torch.cuda.synchronize()
        for g in (y, dx, grad):
            g.check()
        assert torch.isfinite(y.t.float()).all() and torch.isfinite(dx.t.float()).all()
        gu, d = _views(grad.t, H, I, torch.bfloat16)
        assert torch.isfinite(gu.float()).all() and torch.isfinite(d.float()).all()
    rows = np.unique(np.minimum(np.r_[0, 255, 256, T - 1, rng.integers(0, T, 44)], T - 1))
    r = torch.from_numpy(rows).cuda()
    args = [f64(t) for t in (x[r], wg, wu, wd)]
    bounds = D.block_bounds(f64(dy[r]), *args, "bf16")
    _check("y", f64(y.t.view(T, H)[r]), D.block(*args)[0], bounds["y"])
    _check("dx", f64(dx.t.view(T, H)[r]), D.block_backward(f64(dy[r]), *args)[0], bounds["dx"])
    inner = np.unique(np.r_[0, 127, 128, I - 1, rng.integers(0, I, 44)])
    k = torch.from_numpy(inner).cuda()
    args = [f64(t) for t in (x, wg[k], wu[k], wd[:, k].contiguous())]
    bounds = D.block_bounds(f64(dy), *args, "bf16")
    _, rg, ru, rd = D.block_backward(f64(dy), *args)
    at = k // 16 * 32 + k % 16
    _check("dwg", f64(gu[at]), rg, bounds["dwg"])
    _check("dwu", f64(gu[at + 16]), ru, bounds["dwu"])
    _check("dwd", f64(d[:, k]), rd, bounds["dwd"])


@pytest.mark.parametrize("T,N,K,y_type", [(4100, 4099, 4112, BF16), (4097, 8195, 144, F32), (8200, 2056, 1040, BF16)])
def test_i8_matmul_large(B, T, N, K, y_type):
    rng = np.random.default_rng(T + N)
    x = normal(rng, (T, K), BF16)
    wq = rng.integers(-128, 128, (N, K), dtype=np.int8)
    ws = (rng.random(N) * 0.01 + 1e-4).astype(np.float32)
    with Ctx(B) as c:
        got = f64(_matmul(B, c, x, BF16, K, None, T, torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda(), N, K, y_type, N))
    rows = np.unique(np.r_[0, 255, 256, T - 1, rng.integers(0, T, 60)])
    ref = D.i8_matmul(*D.quantize_rows(f64(x)[rows]), wq, ws)
    _check("y", got[rows], ref, D.i8_bound(ref, NAME[y_type]))
    cols = np.unique(np.r_[0, 255, 256, N - 1, rng.integers(0, N, 30)])
    ref = D.i8_matmul(*D.quantize_rows(f64(x)), wq[cols], ws[cols])
    _check("y", got[:, cols], ref, D.i8_bound(ref, NAME[y_type]))


def test_i8_block_large(B):
    """Every row of the 8-bit block at sizes of the largest tiles: relative error in the 2-norm.
    The result's rounding is 2^-8 of each value at most; codes that differ are few (h's quotient
    within 2^-10 of a border) and move a row by less than 2^-8 of its norm."""
    T, H, I = 4100, 2112, 4128
    rng = np.random.default_rng(6)
    x, _, wg, wu, wd = _block_inputs(rng, T, H, I, BF16)
    with Ctx(B, H, I) as c:
        b8 = torch.empty(B.moe_i8_blob_bytes(c.cfg), dtype=torch.uint8, device="cuda")
        B.moe_i8_pack(c.p, _blob(B, c, wg, wu, wd), b8)
        work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        y = Guarded(T * H, torch.bfloat16)
        B.moe_i8_ffn(c.p, x, T, b8, y.t, work)
        torch.cuda.synchronize()
        y.check()
    rows = np.unique(np.r_[0, 255, 256, T - 1, rng.integers(0, T, 120)])
    ref, _ = D.i8_block(f64(x)[rows], *[v for w in (wg, wu, wd) for v in D.quantize_rows(f64(w))])
    err = np.linalg.norm(f64(y.t).reshape(T, H)[rows] - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert (err <= 2.0 ** -7).all(), err.max()


@pytest.mark.parametrize("w", [BF16, F32])
def test_block_backward_partial_outputs(B, w):
    """dx alone, the weights' gradient alone: the same bits as both together, and nothing else
    written; T = 0 gives a zero gradient and leaves the padding."""
    T, H, I = 70, 192, 96
    rng = np.random.default_rng(2)
    x, dy, wg, wu, wd = _block_inputs(rng, T, H, I, w)
    with Ctx(B, H, I, w) as c:
        blob = _blob(B, c, wg, wu, wd)
        work = torch.empty(B.moe_dense_workspace_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
        save = torch.empty(B.moe_dense_save_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
        y = torch.empty_like(x)
        B.moe_dense_ffn(c.p, x, T, blob, save, y, work)
        out = []
        for with_dx, with_dw in ((1, 1), (1, 0), (0, 1)):
            dx, g = Guarded(T * H, TORCH[w]), Guarded(blob.numel(), torch.uint8)
            B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save, dx.t if with_dx else None, g.t if with_dw else None, work)
            torch.cuda.synchronize()
            dx.check(), g.check()
            out.append((dx.t, g.t))
        assert same_bits(out[0][0], out[1][0]) and same_bits(out[0][1], out[2][1])
        assert torch.isnan(out[2][0]).all() and (out[1][1] == 77).all()
        g = Guarded(blob.numel(), torch.uint8)
        B.moe_dense_ffn_backward(c.p, None, None, 0, None, None, None, g.t, None)
        torch.cuda.synchronize()
        g.check()
        es = x.element_size()
        end = 2 * I * H * es
        assert not g.t[:end].any() and not g.t[(end + 255) // 256 * 256:][: H * I * es].any()


def test_block_gradient_against_differences(B):
    """fp32: the loss sum(y * dy) moves as the gradients say.  The step 2^-6 along a random
    direction of unit entries leaves a third-order term; both sides' own error is bounded by
    the elementwise bounds summed."""
    T, H, I = 20, 128, 64
    rng = np.random.default_rng(9)
    x, dy, wg, wu, wd = _block_inputs(rng, T, H, I, F32)
    with Ctx(B, H, I, F32) as c:
        work = torch.empty(B.moe_dense_workspace_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
        save = torch.empty(B.moe_dense_save_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
        y, dx = torch.empty_like(x), torch.empty_like(x)
        blob = _blob(B, c, wg, wu, wd)
        grad = torch.empty_like(blob)
        B.moe_dense_ffn(c.p, x, T, blob, save, y, work)
        B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save, dx, grad, work)

        def loss(px, pblob):
            B.moe_dense_ffn(c.p, px, T, pblob, None, y, work)
            torch.cuda.synchronize()
            return float((y.double() * dy.double()).sum())

        bounds = D.block_bounds(f64(dy), *(f64(t) for t in (x, wg, wu, wd)), "f32")
        noise = float((bounds["y"] * np.abs(f64(dy))).sum())
        for k in range(4):
            step = 2.0 ** -10
            ws = [wg, wu, wd]
            d = torch.randn_like(x if k == 0 else ws[k - 1])
            if k == 0:
                up, dn = loss(x + step * d, blob), loss(x - step * d, blob)
                want = float((dx.double() * d.double()).sum())
            else:
                v = []
                for sgn in (1, -1):
                    m = [t.clone() for t in ws]
                    m[k - 1] += sgn * step * d
                    v.append(loss(x, _blob(B, c, *m)))
                up, dn = v
                gu, dd = _views(grad, H, I, torch.float32)
                gg = gu.view(I // 16, 2, 16, H)
                g = [gg[:, 0].reshape(I, H), gg[:, 1].reshape(I, H), dd][k - 1]
                want = float((g.double() * d.double()).sum())
            # central difference in fp64 of the formulas gives the third-order term exactly
            args = [f64(t) for t in (x, wg, wu, wd)]
            dd64 = f64(d)
            ref = []
            for sgn in (1, -1):
                b = [a.copy() for a in args]
                b[k] = f64(torch.from_numpy(args[k]).float() + sgn * step * d.cpu())
                ref.append(float((D.block(*b)[0] * f64(dy)).sum()))
            third = abs((ref[0] - ref[1]) / (2 * step) - float((D.block_backward(f64(dy), *args)[k] * dd64).sum()))
            key = ["dx", "dwg", "dwu", "dwd"][k]
            tol = third + noise / step * 1.5 + float((bounds[key] * np.abs(dd64)).sum())
            assert abs((up - dn) / (2 * step) - want) <= tol, (k, up, dn, want, tol)


# ---------------------------------------------------------------- 8-bit block

def _blob8_parts(B, blob8, H, I):
    d = (2 * I * H + 255) // 256 * 256
    gs = (d + H * I + 255) // 256 * 256
    ds = (gs + 8 * I + 255) // 256 * 256
    return (blob8[: 2 * I * H].view(torch.int8).view(2 * I, H), blob8[d: d + H * I].view(torch.int8).view(H, I),
            blob8[gs: gs + 8 * I].view(torch.float32), blob8[ds: ds + 4 * H].view(torch.float32))


def test_i8_pack(B):
    H, I = 192, 160
    rng = np.random.default_rng(4)
    _, _, wg, wu, wd = _block_inputs(rng, 1, H, I, BF16)
    with Ctx(B, H, I) as c:
        blob = _blob(B, c, wg, wu, wd)
        b8 = Guarded(B.moe_i8_blob_bytes(c.cfg), torch.uint8)
        B.moe_i8_pack(c.p, blob, b8.t)
        torch.cuda.synchronize()
        b8.check()
        gu, d, gs, ds = _blob8_parts(B, b8.t, H, I)
    for codes, scale, ref in ((gu, gs, D.interleave(f64(wg), f64(wu))), (d, ds, f64(wd))):
        q, s = D.quantize_rows(ref)
        assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(scale.cpu().numpy(), s)


@pytest.mark.parametrize("T,H,I", [(1, 64, 32), (1, 4096, 1536), (2, 192, 96), (5, 2048, 768), (8, 1088, 8192),
                                   (9, 256, 160), (16, 576, 1120), (17, 320, 64), (40, 512, 544), (64, 64, 1024),
                                   (130, 192, 416), (300, 576, 1120), (600, 1024, 768)])
def test_i8_block(B, T, H, I):
    print(f"[i8_block] T={T} H={H} I={I}", flush=True)
    rng = np.random.default_rng(T + H + I)
    x, _, wg, wu, wd = _block_inputs(rng, T, H, I, BF16)
    with Ctx(B, H, I) as c:
        blob = _blob(B, c, wg, wu, wd)
        b8 = torch.empty(B.moe_i8_blob_bytes(c.cfg), dtype=torch.uint8, device="cuda")
        B.moe_i8_pack(c.p, blob, b8)
        work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        y, y2 = Guarded(T * H, torch.bfloat16), Guarded(T * H, torch.bfloat16)
        B.moe_i8_ffn(c.p, x, T, b8, y.t, work)
        B.moe_i8_ffn(c.p, x, T, b8, y2.t, work)
        torch.cuda.synchronize()
        y.check(), y2.check()
        assert same_bits(y.t, y2.t)
    q = [v for w in (wg, wu, wd) for v in D.quantize_rows(f64(w))]
    ref, (h, hs) = D.i8_block(f64(x), *q)
    # h is within about 2^-17 of its size, so its scale moves by that and a code by one at most;
    # codes move where the quotient lies within 127 * 2^-16 of a border, and half of the rest of
    # the bound is the result's own rounding
    step = hs.astype(np.float64)[:, None]
    frac = np.abs(h / np.where(step > 0, step, 1) - np.floor(h / np.where(step > 0, step, 1)) - 0.5)
    near = (frac <= 127 * 2.0 ** -16) * step
    wdeq = np.abs(q[4].astype(np.float64)) * q[5].astype(np.float64)[:, None]
    # every term's scale moves by 2^-17 with h's largest magnitude
    bound = near @ wdeq.T + np.abs(ref) * (2.0 ** -16 + 2.0 ** -8) + 2.0 ** -16 * (step * 0.5 * wdeq.sum(1))
    _check("y", f64(y.t).reshape(T, H), ref, bound)


# ---------------------------------------------------------------- used together

def test_train_then_serve_in_8_bits(B):
    """A block's forward and backward pass, one descent step on its blob, the new blob packed to
    8 bits, and a batch through the 8-bit block into an 8-bit head, on a stream of its own: each
    stage against the fp64 forms on the stage's own inputs."""
    T, H, I, N = 96, 256, 128, 1003
    rng = np.random.default_rng(12)
    x, dy, wg, wu, wd = _block_inputs(rng, T, H, I, BF16)
    head = normal(rng, (N, H), BF16, 0.05)
    st = torch.cuda.Stream()
    with Ctx(B, H, I) as c, torch.cuda.stream(st):
        st.wait_stream(torch.cuda.default_stream())
        blob = _blob(B, c, wg, wu, wd)
        work = torch.empty(B.moe_dense_workspace_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
        save = torch.empty(B.moe_dense_save_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
        grad, y, dx = torch.zeros_like(blob), torch.empty_like(x), torch.empty_like(x)
        B.moe_dense_ffn(c.p, x, T, blob, save, y, work, st)
        B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save, dx, grad, work, st)
        for v, g in zip(_views(blob, H, I, torch.bfloat16), _views(grad, H, I, torch.bfloat16)):
            v.sub_(0.01 * g)
        b8 = torch.empty(B.moe_i8_blob_bytes(c.cfg), dtype=torch.uint8, device="cuda")
        B.moe_i8_pack(c.p, blob, b8, st)
        B.moe_i8_ffn(c.p, x, T, b8, y, work, st)
        hq, hs = torch.empty((N, H), dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
        B.moe_i8_quantize(c.p, head, BF16, H, N, H, hq, hs, st)
        logits = torch.empty((T, N), device="cuda")
        hw = torch.empty(B.moe_i8_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
        B.moe_i8_matmul(c.p, y, BF16, H, None, T, hq, hs, N, H, logits, F32, N, hw, st)
        st.synchronize()
        gu, d = _views(blob, H, I, torch.bfloat16)
        g2, u2 = D.deinterleave(f64(gu))
        old = D.block_backward(f64(dy), *(f64(t) for t in (x, wg, wu, wd)))
        # the step moved the weights along the gradient (both roundings: half a bf16 step each)
        for new, was, step in ((g2, f64(wg), old[1]), (u2, f64(wu), old[2]), (f64(d), f64(wd), old[3])):
            assert np.abs(new - (was - 0.01 * step)).max() <= 2.0 ** -8 * np.abs(was).max() + 0.01 * 2.0 ** -4 * np.abs(step).max()
        q = [v for w in (g2, u2, f64(d)) for v in D.quantize_rows(w)]
        ref, _ = D.i8_block(f64(x), *q)
        assert np.linalg.norm(f64(y) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
        xq, xs = D.quantize_rows(f64(y))
        wq, ws = D.quantize_rows(f64(head))
        want = D.i8_matmul(xq, xs, wq, ws)
        _check("logits", f64(logits), want, D.i8_bound(want, "f32"))


@pytest.mark.parametrize("T", [1, 8, 40, 200])
def test_graph_replays(B, T):
    """The whole chain captured once and replayed with new inputs between replays, eager work and
    synchronisations in between; two graphs with workspaces of their own."""
    H, I, N = 256, 160, 530
    rng = np.random.default_rng(T)
    x0, dy0, wg, wu, wd = _block_inputs(rng, T, H, I, BF16)
    with Ctx(B, H, I) as c:
        blob = _blob(B, c, wg, wu, wd)
        b8 = torch.empty(B.moe_i8_blob_bytes(c.cfg), dtype=torch.uint8, device="cuda")
        B.moe_i8_pack(c.p, blob, b8)
        wq = torch.randint(-127, 128, (N, H), dtype=torch.int8, device="cuda")
        ws = torch.rand(N, device="cuda")

        class Chain:
            def __init__(self):
                self.x, self.dy = x0.clone(), dy0.clone()
                self.y, self.dx, self.y8 = (torch.empty_like(x0) for _ in range(3))
                self.save = torch.empty(B.moe_dense_save_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
                self.grad = torch.zeros_like(blob)
                self.work = torch.empty(B.moe_dense_workspace_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
                self.hwork = torch.empty(B.moe_i8_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
                self.logits = torch.empty((T, N), device="cuda")

            def go(self, s):
                B.moe_dense_ffn(c.p, self.x, T, blob, self.save, self.y, self.work, s)
                B.moe_dense_ffn_backward(c.p, self.dy, self.x, T, blob, self.save, self.dx, self.grad, self.work, s)
                B.moe_i8_ffn(c.p, self.x, T, b8, self.y8, self.work, s)
                B.moe_i8_matmul(c.p, self.y8, BF16, H, None, T, wq, ws, N, H, self.logits, F32, N, self.hwork, s)

            def outs(self):
                return [t.clone() for t in (self.y, self.dx, self.grad, self.y8, self.logits)]

        chains, graphs = [Chain(), Chain()], []
        for ch in chains:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                ch.go(s)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                ch.go(s)
            graphs.append(g)
        eager = Chain()
        for k in range(4):
            for ch, g in zip(chains, graphs):
                ch.x.copy_(normal(rng, (T, H), BF16))
                ch.dy.copy_(normal(rng, (T, H), BF16, 0.1))
                eager.x.copy_(ch.x), eager.dy.copy_(ch.dy)
                torch.cuda.synchronize()
                g.replay()
                torch.cuda.synchronize()
                got = ch.outs()
                eager.go(torch.cuda.current_stream())
                torch.cuda.synchronize()
                for a, b in zip(got, eager.outs()):
                    assert same_bits(a, b), k


def test_large_workspace_few_tokens(B):
    """Calls with fewer tokens than their workspace was sized for (they split K and keep partial
    sums there) give what an exact workspace gives, and stay inside it."""
    K, N, H, I = 4096, 264, 1024, 160
    rng = np.random.default_rng(21)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    ws = torch.rand(N, device="cuda")
    with Ctx(B, H, I) as c:
        for T in (20, 64, 300):
            x = normal(rng, (T, K), BF16)
            want = _matmul(B, c, x, BF16, K, None, T, w, ws, N, K, F32, N)
            work = Guarded(B.moe_i8_workspace_bytes(1100, K), torch.uint8)
            y = torch.empty((T, N), device="cuda")
            B.moe_i8_matmul(c.p, x, BF16, K, None, T, w, ws, N, K, y, F32, N, work.t)
            torch.cuda.synchronize()
            work.check()
            assert same_bits(y, want.contiguous())
            bx, bdy, wg, wu, wd = _block_inputs(rng, T, H, I, BF16)
            blob = _blob(B, c, wg, wu, wd)
            save = torch.empty(B.moe_dense_save_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
            outs = []
            for n in (T, 1100):
                work = Guarded(B.moe_dense_workspace_bytes(c.cfg, n), torch.uint8)
                by, dx, grad = torch.empty_like(bx), torch.empty_like(bx), torch.zeros_like(blob)
                B.moe_dense_ffn(c.p, bx, T, blob, save, by, work.t)
                B.moe_dense_ffn_backward(c.p, bdy, bx, T, blob, save, dx, grad, work.t)
                torch.cuda.synchronize()
                work.check()
                outs.append((by, dx, grad))
            assert all(same_bits(p, q) for p, q in zip(*outs))


def test_large_tiles_in_a_graph(B):
    """Calls of the largest tiles captured before they ever ran eagerly (they set an attribute of
    their kernels), then replayed."""
    T, N, K = 4096, 4096 + 32, 320
    rng = np.random.default_rng(22)
    x = normal(rng, (T, K), F32)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    ws = torch.rand(N, device="cuda")
    with Ctx(B) as c:
        work = torch.empty(B.moe_i8_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
        y = torch.zeros((T, N), device="cuda")
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            B.moe_i8_matmul(c.p, x, F32, K, None, T, w, ws, N, K, y, F32, N, work, s)
        for _ in range(3):
            x.copy_(normal(rng, (T, K), F32))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert same_bits(y, _matmul(B, c, x, F32, K, None, T, w, ws, N, K, F32, N).contiguous())


def test_two_streams_at_once(B):
    """Two calls in flight on two streams, each with a workspace and a context of its own."""
    T, K, N = 300, 1040, 777
    rng = np.random.default_rng(8)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    ws = torch.rand(N, device="cuda")
    xs = [normal(rng, (T, K), BF16) for _ in range(2)]
    outs = []
    with Ctx(B) as c0, Ctx(B) as c1:
        alone = [_matmul(B, c0, x, BF16, K, None, T, w, ws, N, K, F32, N).clone() for x in xs]
        works = [torch.empty(B.moe_i8_workspace_bytes(T, K), dtype=torch.uint8, device="cuda") for _ in range(2)]
        outs = [torch.empty((T, N), device="cuda") for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(10):
            for i, c in enumerate((c0, c1)):
                B.moe_i8_matmul(c.p, xs[i], BF16, K, None, T, w, ws, N, K, outs[i], F32, N, works[i], streams[i])
        torch.cuda.synchronize()
    for a, b in zip(alone, outs):
        assert same_bits(a.contiguous(), b)


def test_no_tokens(B):
    """T = 0 (and no rows) writes nothing."""
    with Ctx(B, 64, 32) as c:
        y = torch.full((64,), 3.0, dtype=torch.bfloat16, device="cuda")
        e = torch.empty(256, dtype=torch.uint8, device="cuda")
        B.moe_dense_ffn(c.p, y, 0, e, e, y, e)
        B.moe_i8_ffn(c.p, y, 0, e, y, e)
        B.moe_i8_matmul(c.p, y, BF16, 64, None, 0, e, e, 4, 64, y, BF16, 4, e)
        B.moe_i8_quantize(c.p, y, BF16, 64, 0, 64, y, y)
        torch.cuda.synchronize()
        assert (y == 3).all()
