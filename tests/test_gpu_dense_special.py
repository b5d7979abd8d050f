"""Dense operators on values far out: gates near the end of fp32, shut gates with large gradients
behind them, and tokens or weight rows with infinities and NaNs beside ordinary ones."""
import numpy as np
import pytest
import torch

from oracle import dense_oracle as D
from test_gpu_dense import (BF16, F32, NAME, TORCH, Ctx, Guarded, _blob, _block_inputs, _check, _matmul, _views, f64,
                            normal, same_bits)
from test_gpu_dense import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def _i8_ffn(B, c, x, b8):
    T, H = x.shape
    work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
    y = Guarded(T * H, torch.bfloat16)
    B.moe_i8_ffn(c.p, x, T, b8, y.t, work)
    torch.cuda.synchronize()
    y.check()
    return y.t.view(T, H)


def _pack8(B, c, wg, wu, wd):
    b8 = torch.empty(B.moe_i8_blob_bytes(c.cfg), dtype=torch.uint8, device="cuda")
    B.moe_i8_pack(c.p, _blob(B, c, wg, wu, wd), b8)
    return b8


@pytest.mark.parametrize("T,I", [(1, 32), (1, 8192), (7, 96), (12, 64), (40, 160), (300, 256)])
def test_i8_block_far_gates(B, T, I):
    """Gates up to 3.3e38 of either sign, with |up| < 1: h = silu(gate) up and y are finite.

    One channel of x is not 0, so gate and up are single products: each of the three roundings of
    2^-24 once, silu's four steps of 2^-23 and the product's rounding put h within 2^-20, and half
    of the argument's error times its size for gates that are neither small nor far (|gate| <= 8:
    3 * 8 * 2^-24); 2^-17 of h covers both.  From there on as for ordinary values."""
    H = 64
    rng = np.random.default_rng(T + I)
    x = np.zeros((T, H))
    x[:, 5] = 2.0 ** 63 * rng.choice([1.0, 0.75, 2.0 ** -64, 2.0 ** -70], T)
    x[0, 5] = 2.0 ** 63
    wg, wu, wd = np.zeros((I, H)), np.zeros((I, H)), rng.standard_normal((H, I)) * 2.0 ** -100
    # gates over 2^127 (1.7e38): 1.5 and 1.9375 of it; ordinary ones (up to 8); their negatives
    wg[:, 5] = rng.choice([1.5, 1.9375, 1.0, 2.0 ** -127, 2.0 ** -124, 2.0 ** -60], I) * rng.choice([-1, 1], I) * 2.0 ** 64
    wg[:4, 5] = np.array([1.5, 1.9375, -1.9375, 2.0 ** -126]) * 2.0 ** 64
    wu[:, 5] = (rng.random(I) * 0.5 + 0.25) * rng.choice([-1, 1], I) * 2.0 ** -63
    x, wg, wu, wd = (torch.from_numpy(a.astype(np.float32)).bfloat16().cuda() for a in (x, wg, wu, wd))
    with Ctx(B, H, I) as c:
        y = _i8_ffn(B, c, x, _pack8(B, c, wg, wu, wd))
    q = [v for w in (wg, wu, wd) for v in D.quantize_rows(f64(w))]
    ref, (h, hs) = D.i8_block(f64(x), *q)
    assert np.abs(h[0]).max() > 1e37 and np.isfinite(ref).all()
    step = hs.astype(np.float64)[:, None]
    quot = h / np.where(step > 0, step, 1)
    near = (np.abs(quot - np.floor(quot) - 0.5) <= 127 * 2.0 ** -16) * step
    wdeq = np.abs(q[4].astype(np.float64)) * q[5].astype(np.float64)[:, None]
    bound = near @ wdeq.T + np.abs(ref) * (2.0 ** -16 + 2.0 ** -8) + 2.0 ** -16 * (step * 0.5 * wdeq.sum(1))
    _check("y", f64(y), ref, bound)


@pytest.mark.parametrize("T", [1, 5, 40, 300])
@pytest.mark.parametrize("w", [BF16, F32])
def test_block_backward_shut_gates(B, T, w):
    """Gates at -2^80 beside ordinary ones, with dh near 2^60: dh g leaves fp32, and so does dh u
    where u is large, but silu and its derivative are 0 there, so dg and du are.

    One channel of x is not 0 and holds a power of two, so gates and up are exact (bounds with
    exact pre-activations)."""
    H, I = 64, 96
    rng = np.random.default_rng(T)
    xs = np.zeros((T, H))
    xs[:, 9] = 2.0 ** 40 * rng.choice([1.0, 0.5, 0.25], T)
    gate, up = rng.standard_normal((I, H)), rng.standard_normal((I, H))
    gate[:, 9] *= 2.0 ** -40
    up[:, 9] *= 2.0 ** -40
    gate[::3, 9] = -2.0 ** 40 * (1 + rng.random(len(gate[::3])))
    up[::6, 9] *= 2.0 ** 75
    x, dy, wg, wu, wd = (torch.from_numpy(a.astype(np.float32)).to(TORCH[w]).cuda()
                         for a in (xs, rng.standard_normal((T, H)) * 2.0 ** 57, gate, up, rng.standard_normal((H, I))))
    with Ctx(B, H, I, w) as c:
        blob = _blob(B, c, wg, wu, wd)
        work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        save = torch.full((B.moe_dense_save_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        y, dx, grad = Guarded(T * H, TORCH[w]), Guarded(T * H, TORCH[w]), Guarded(blob.numel(), torch.uint8)
        B.moe_dense_ffn(c.p, x, T, blob, save, y.t, work)
        B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save, dx.t, grad.t, work)
        torch.cuda.synchronize()
        for g in (y, dx, grad):
            g.check()
        gu, dd = _views(grad.t, H, I, TORCH[w])
    args = [f64(t) for t in (x, wg, wu, wd)]
    g64 = args[0] @ args[1].T
    assert (np.abs(f64(dy) @ args[3])[:, ::3] * np.abs(g64)[:, ::3]).max() > 3.5e38
    bounds = D.block_bounds(f64(dy), *args, NAME[w], exact=True)
    ref = D.block_backward(f64(dy), *args)
    _check("y", f64(y.t).reshape(T, H), D.block(*args)[0], bounds["y"])
    _check("dx", f64(dx.t).reshape(T, H), ref[0], bounds["dx"])
    dwg, dwu = D.deinterleave(f64(gu))
    _check("dwg", dwg, ref[1], bounds["dwg"])
    _check("dwu", dwu, ref[2], bounds["dwu"])
    _check("dwd", f64(dd), ref[3], bounds["dwd"])


TOKENS = [(3, 64, 64), (12, 320, 96), (40, 192, 544), (300, 576, 160), (2100, 1088, 2080)]


def _step(B, c, x, dy, blob, w):
    T, H = x.shape
    work = torch.full((B.moe_dense_workspace_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
    save = torch.full((B.moe_dense_save_bytes(c.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
    y, dx, grad = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(blob)
    B.moe_dense_ffn(c.p, x, T, blob, save, y, work)
    B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save, dx, grad, work)
    torch.cuda.synchronize()
    gu, dd = _views(grad, H, c.cfg.inter, TORCH[w])
    return y, dx, gu.clone(), dd.clone()


@pytest.mark.parametrize("T,H,I", TOKENS)
@pytest.mark.parametrize("w", [BF16, F32])
def test_block_keeps_tokens_apart(B, w, T, H, I):
    """A token with a NaN, an infinity or numbers whose products overflow leaves y and dx of the
    others as they are, bit for bit; so does one in dy, which reaches one row of dWd."""
    rng = np.random.default_rng(T)
    x, dy, wg, wu, wd = _block_inputs(rng, T, H, I, w)
    at, others = T // 2, [t for t in range(T) if t != T // 2]
    with Ctx(B, H, I, w) as c:
        blob = _blob(B, c, wg, wu, wd)
        y, dx, gu, dd = _step(B, c, x, dy, blob, w)
        for bad in (float("nan"), float("inf"), 3e38):
            x2 = x.clone()
            x2[at, 7 if bad != 3e38 else slice(None)] = bad
            y2, dx2, _, _ = _step(B, c, x2, dy, blob, w)
            assert same_bits(y2[others], y[others]) and same_bits(dx2[others], dx[others])
            if bad != bad:
                assert torch.isnan(y2[at]).all() and torch.isnan(dx2[at]).all()
            dy2 = dy.clone()
            dy2[at, 5] = bad
            y2, dx2, gu2, dd2 = _step(B, c, x, dy2, blob, w)
            rest = [h for h in range(H) if h != 5]
            assert same_bits(y2, y) and same_bits(dx2[others], dx[others]) and same_bits(dd2[rest], dd[rest])
            if bad != bad:
                assert torch.isnan(dx2[at]).all() and torch.isnan(dd2[5]).all() and torch.isnan(gu2).all()


@pytest.mark.parametrize("T,H,I", [(1, 64, 64)] + TOKENS)
def test_i8_block_keeps_tokens_apart(B, T, H, I):
    rng = np.random.default_rng(T)
    x, _, wg, wu, wd = _block_inputs(rng, T, H, I, BF16)
    at, others = T // 2, [t for t in range(T) if t != T // 2]
    with Ctx(B, H, I) as c:
        b8 = _pack8(B, c, wg, wu, wd)
        y = _i8_ffn(B, c, x, b8)
        assert torch.isfinite(y.float()).all()
        for bad in (float("nan"), float("inf"), -float("inf")):
            x2 = x.clone()
            x2[at, 7] = bad
            y2 = _i8_ffn(B, c, x2, b8)
            assert torch.isnan(y2[at]).all() and same_bits(y2[others], y[others])
        x2 = x.clone()
        x2[at] = 0
        y2 = _i8_ffn(B, c, x2, b8)
        assert not y2[at].any() and same_bits(y2[others], y[others])


@pytest.mark.parametrize("T", [1, 5, 12, 40, 300, 2100])
def test_i8_matmul_special_weight_rows(B, T):
    """Weight rows with a NaN or an infinity make their column NaN, zero rows zeros; the others are
    unchanged."""
    K, N = 272, 163
    rng = np.random.default_rng(T)
    x, w = normal(rng, (T, K), BF16), normal(rng, (N, K), F32)
    with Ctx(B) as c:
        def run(w):
            q, s = torch.empty((N, K), dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
            B.moe_i8_quantize(c.p, w, F32, K, N, K, q, s)
            return _matmul(B, c, x, BF16, K, None, T, q, s, N, K, F32, N)
        y = run(w)
        w2 = w.clone()
        w2[3, 9], w2[100, 0], w2[162, 271], w2[64] = float("nan"), float("inf"), -float("inf"), 0
        y2 = run(w2)
    others = [n for n in range(N) if n not in (3, 64, 100, 162)]
    assert torch.isnan(y2[:, [3, 100, 162]]).all() and not y2[:, 64].any()
    assert same_bits(y2[:, others], y[:, others])
