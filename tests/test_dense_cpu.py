"""CPU checks of the dense operators: the fp64 forms against differences and whole-number
arithmetic, buffer sizes, and every refusal (arguments are checked before any GPU work)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import dense_oracle as D

B = pytest.importorskip("expert_cached_moe_amd.binding")

P = 1 << 20            # a plausible, aligned address; refused calls never follow it


@pytest.fixture
def ctx():
    c = B.moe_create(B.make_config(128, 64, 1, 1, w_dtype=B.MOE_W_BF16))
    yield c
    B.moe_destroy(c)


def test_quantize_rows_against_fractions():
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((6, 48)) * 10.0 ** rng.integers(-20, 20, (6, 1))).astype(np.float32)
    x[1] = np.arange(-24, 24)                              # max 24
    x[2, :] = 0
    x[3, :16] = 127.0
    x[3, 16:] = np.arange(32) + 0.5                        # scale 1: exact half-way points
    q, s = D.quantize_rows(x)
    for r in range(6):
        if not x[r].any():
            assert s[r] == 0 and not q[r].any()
            continue
        assert s[r] == np.float32(float(np.abs(x[r]).max()) / 127.0)
        for v, c in zip(x[r], q[r]):
            d = Fraction(float(v)) / Fraction(float(s[r]))
            assert abs(d - int(c)) <= Fraction(1, 2)
            if abs(d - int(c)) == Fraction(1, 2):
                assert c % 2 == 0


def test_quantize_rows_special():
    x = np.zeros((4, 16), np.float32)
    x[0, 3] = np.inf
    x[1, 0], x[1, 1] = 5.0, np.nan
    x[2, 5] = 1e-44
    x[3, 2] = -3.0e38
    q, s = D.quantize_rows(x)
    assert np.isnan(s[:2]).all() and not q[:3].any() and s[2] == 0 and q[3, 2] == -127


def test_block_gradient_against_differences():
    rng = np.random.default_rng(7)
    T, H, I = 3, 8, 16
    x, dy = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    w = [rng.standard_normal(s) * 0.5 for s in ((I, H), (I, H), (H, I))]
    got = D.block_backward(dy, x, *w)
    args = [x, *w]
    e = 1e-5
    for k, grad in enumerate(got):
        for _ in range(25):
            i = tuple(rng.integers(0, n) for n in args[k].shape)
            v = []
            for d in (e, -e):
                b = [a.copy() for a in args]
                b[k][i] += d
                v.append((D.block(*b)[0] * dy).sum())
            assert abs((v[0] - v[1]) / (2 * e) - grad[i]) <= 1e-7 * (1 + abs(grad[i]))


def test_interleave_matches_pack_layout():
    cfg = B.make_config(64, 32, 1, 1, w_dtype=B.MOE_W_F32)
    rng = np.random.default_rng(1)
    wg, wu = rng.standard_normal((2, 32, 64)).astype(np.float32)
    wd = rng.standard_normal((64, 32)).astype(np.float32)
    blob = np.zeros(B.moe_expert_bytes(cfg), np.uint8)
    B.moe_pack_expert(cfg, wg, wu, wd, None, None, None, blob)
    gu = D.interleave(wg, wu)
    assert np.array_equal(blob.view(np.float32)[: 64 * 64].reshape(64, 64), gu)
    assert all(np.array_equal(a, b) for a, b in zip(D.deinterleave(gu), (wg, wu)))


def test_sizes():
    cfg = B.make_config(128, 64, 1, 1, w_dtype=B.MOE_W_BF16)
    assert B.moe_i8_workspace_bytes(3, 64) >= 3 * 64 + 3 * 4
    assert B.moe_i8_workspace_bytes(0, 16) > 0
    assert B.moe_i8_workspace_bytes(2 ** 31 - 1, 131056) > 2 ** 31 * 131056 * 0.99
    assert B.moe_dense_save_bytes(cfg, 5) >= 5 * (2 * 64 * 3 + 64 * 2)
    assert B.moe_dense_workspace_bytes(cfg, 5) >= 5 * (128 + 64 * 4 + 64 + 8)
    assert B.moe_i8_blob_bytes(cfg) >= 3 * 128 * 64 + 4 * (2 * 64 + 128)
    for K in (0, 8, 24, -16, 131072):
        with pytest.raises(B.MoeError) as e:
            B.moe_i8_workspace_bytes(4, K)
        assert e.value.status == B.MOE_ESHAPE
    for f in (lambda: B.moe_i8_workspace_bytes(-1, 64), lambda: B.moe_dense_workspace_bytes(cfg, -1),
              lambda: B.moe_dense_save_bytes(cfg, -1)):
        with pytest.raises(B.MoeError) as e:
            f()
        assert e.value.status == B.MOE_EINVAL


def test_workspace_serves_fewer_tokens():
    """A workspace for max_T tokens is enough for every T below it (calls with fewer tokens split
    K and add partial sums)."""
    for K in (16, 64, 4096, 131056):
        sizes = [B.moe_i8_workspace_bytes(T, K) for T in (0, 1, 17, 64, 1023, 1024, 1025, 2048, 8192, 100000)]
        assert sizes == sorted(sizes)
    for cfg in (B.make_config(128, 64, 1, 1, w_dtype=w) for w in (B.MOE_W_BF16, B.MOE_W_F32)):
        sizes = [B.moe_dense_workspace_bytes(cfg, T) for T in (0, 1, 17, 1024, 1025, 100000)]
        assert sizes == sorted(sizes)


def _refused(ctx, status, f, *args):
    with pytest.raises(B.MoeError) as e:
        f(ctx, *args)
    assert e.value.status == status
    assert B.moe_last_error(ctx)


def test_quantize_refusals(ctx):
    ok = dict(x=P, t=B.MOE_A_BF16, ld=64, rows=4, cols=64, q=P, s=P)
    for status, bad in [(B.MOE_EINVAL, dict(rows=-1)), (B.MOE_EINVAL, dict(t=B.MOE_A_I8)), (B.MOE_EINVAL, dict(t=9)),
                        (B.MOE_ESHAPE, dict(cols=0)), (B.MOE_ESHAPE, dict(cols=40)), (B.MOE_EINVAL, dict(ld=63)),
                        (B.MOE_EINVAL, dict(x=None)), (B.MOE_EINVAL, dict(q=None)), (B.MOE_EINVAL, dict(s=None)),
                        (B.MOE_EINVAL, dict(x=P + 1)), (B.MOE_EINVAL, dict(q=P + 8)), (B.MOE_EINVAL, dict(s=P + 2))]:
        a = {**ok, **bad}
        _refused(ctx, status, B.moe_i8_quantize, a["x"], a["t"], a["ld"], a["rows"], a["cols"], a["q"], a["s"])
    B.moe_i8_quantize(ctx, None, B.MOE_A_F32, 64, 0, 64, None, None)          # no rows: no-op
    assert B._lib.moe_i8_quantize(None, P, 0, 64, 1, 64, P, P, None) == B.MOE_EINVAL


def test_matmul_refusals(ctx):
    ok = dict(x=P, t=B.MOE_A_BF16, ld=64, xs=None, T=4, w=P, ws=P, N=5, K=64, y=P, yt=B.MOE_A_F32, ldy=5, work=P)
    for status, bad in [(B.MOE_EINVAL, dict(T=-1)), (B.MOE_EINVAL, dict(t=3)), (B.MOE_EINVAL, dict(yt=B.MOE_A_I8)),
                        (B.MOE_ESHAPE, dict(K=8)), (B.MOE_ESHAPE, dict(K=72)), (B.MOE_ESHAPE, dict(K=131072, ld=131072)),
                        (B.MOE_ESHAPE, dict(N=0)), (B.MOE_EINVAL, dict(ld=48)), (B.MOE_EINVAL, dict(ldy=4)),
                        (B.MOE_EINVAL, dict(xs=P)), (B.MOE_EINVAL, dict(t=B.MOE_A_I8)),
                        (B.MOE_EINVAL, dict(t=B.MOE_A_I8, xs=P, ld=80)), (B.MOE_EINVAL, dict(x=None)),
                        (B.MOE_EINVAL, dict(w=None)), (B.MOE_EINVAL, dict(ws=None)), (B.MOE_EINVAL, dict(y=None)),
                        (B.MOE_EINVAL, dict(work=None)), (B.MOE_EINVAL, dict(x=P + 1)), (B.MOE_EINVAL, dict(w=P + 8)),
                        (B.MOE_EINVAL, dict(y=P + 2)), (B.MOE_EINVAL, dict(work=P + 16)),
                        (B.MOE_EINVAL, dict(t=B.MOE_A_I8, xs=P, x=P + 8))]:
        a = {**ok, **bad}
        _refused(ctx, status, B.moe_i8_matmul, a["x"], a["t"], a["ld"], a["xs"], a["T"], a["w"], a["ws"], a["N"],
                 a["K"], a["y"], a["yt"], a["ldy"], a["work"])
    B.moe_i8_matmul(ctx, None, B.MOE_A_F32, 64, None, 0, None, None, 5, 64, None, B.MOE_A_F32, 5, None)


@pytest.mark.parametrize("w_dtype", [B.MOE_W_F32, B.MOE_W_BF16])
def test_block_refusals(w_dtype):
    ctx = B.moe_create(B.make_config(128, 64, 1, 1, w_dtype=w_dtype))
    for bad in range(4):
        a = [P, P, P, P]                                   # x, blob, y, ws
        for v in (None, P + 8):
            a[bad] = v
            _refused(ctx, B.MOE_EINVAL, B.moe_dense_ffn, a[0], 3, a[1], None, a[2], a[3])
    _refused(ctx, B.MOE_EINVAL, B.moe_dense_ffn, P, 3, P, P + 2, P, P)
    _refused(ctx, B.MOE_EINVAL, B.moe_dense_ffn, P, -1, P, None, P, P)
    for bad in range(5):
        a = [P, P, P, P, P]                                # dy, x, blob, save, ws
        for v in (None, P + 8):
            a[bad] = v
            _refused(ctx, B.MOE_EINVAL, B.moe_dense_ffn_backward, a[0], a[1], 3, a[2], a[3], P, P, a[4])
    _refused(ctx, B.MOE_EINVAL, B.moe_dense_ffn_backward, P, P, 3, P, P, P + 4, P, P)
    _refused(ctx, B.MOE_EINVAL, B.moe_dense_ffn_backward, P, P, 3, P, P, P, P + 4, P)
    _refused(ctx, B.MOE_EINVAL, B.moe_dense_ffn_backward, P, P, -2, P, P, P, P, P)
    B.moe_dense_ffn(ctx, None, 0, None, None, None, None)
    B.moe_dense_ffn_backward(ctx, None, None, 0, None, None, None, None, None)
    if w_dtype == B.MOE_W_F32:
        _refused(ctx, B.MOE_EUNSUPPORTED, B.moe_i8_ffn, P, 3, P, P, P)
        _refused(ctx, B.MOE_EUNSUPPORTED, B.moe_i8_pack, P, P)
    else:
        for bad in range(4):
            a = [P, P, P, P]                               # x, blob8, y, ws
            for v in (None, P + 8):
                a[bad] = v
                _refused(ctx, B.MOE_EINVAL, B.moe_i8_ffn, a[0], 3, a[1], a[2], a[3])
        _refused(ctx, B.MOE_EINVAL, B.moe_i8_ffn, P, -1, P, P, P)
        _refused(ctx, B.MOE_EINVAL, B.moe_i8_pack, None, P)
        _refused(ctx, B.MOE_EINVAL, B.moe_i8_pack, P, None)
        _refused(ctx, B.MOE_EINVAL, B.moe_i8_pack, P + 16, P)
        _refused(ctx, B.MOE_EINVAL, B.moe_i8_pack, P, P + 16)
        B.moe_i8_ffn(ctx, None, 0, None, None, None)
    B.moe_destroy(ctx)


def test_mxfp4_context_refused():
    ctx = B.moe_create(B.make_config(256, 64, 1, 1, w_dtype=B.MOE_W_MXFP4))
    _refused(ctx, B.MOE_EUNSUPPORTED, B.moe_dense_ffn, P, 3, P, None, P, P)
    _refused(ctx, B.MOE_EUNSUPPORTED, B.moe_dense_ffn_backward, P, P, 3, P, P, P, P, P)
    _refused(ctx, B.MOE_EUNSUPPORTED, B.moe_i8_ffn, P, 3, P, P, P)
    _refused(ctx, B.MOE_EUNSUPPORTED, B.moe_i8_pack, P, P)
    B.moe_destroy(ctx)


def test_counts_past_the_limits(ctx):
    big = 2 ** 24 + 16
    _refused(ctx, B.MOE_ESHAPE, B.moe_i8_quantize, P, B.MOE_A_F32, big, 1, big, P, P)
    for T, N in ((1, big), (big, 1)):
        _refused(ctx, B.MOE_ESHAPE, B.moe_i8_matmul, P, B.MOE_A_BF16, 64, None, T, P, P, N, 64, P, B.MOE_A_F32, N, P)
    _refused(ctx, B.MOE_ESHAPE, B.moe_dense_ffn, P, big, P, None, P, P)
    _refused(ctx, B.MOE_ESHAPE, B.moe_dense_ffn_backward, P, P, big, P, P, P, P, P)
    _refused(ctx, B.MOE_ESHAPE, B.moe_i8_ffn, P, big, P, P, P)
