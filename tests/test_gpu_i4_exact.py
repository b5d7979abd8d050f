"""Products with 4-bit weights whose results are exact: every part of an fp32 number on every kind of tiles, numbers
near the ends of fp32, and rows of x near the limits of the tiles' offsets."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
B = pytest.importorskip("expert_cached_moe_amd.binding")
from oracle import i4_oracle as Q  # noqa: E402
from test_gpu_i4 import BF16, F32, TORCH, Layer, Weights, check, ctx, numbers, product  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def powers(N, K, group, seed):
    """Weights that are powers of two, of either sign, or zero."""
    r = np.random.default_rng(seed)
    n = -(-K // group)
    z = r.integers(4, 12, (N, n))
    step = np.array([-4, -2, -1, 0, 1, 2, 4])[r.integers(0, 7, (N, K))]
    codes = (np.repeat(z, group, 1)[:, :K] + step).astype(np.uint8)
    words = (r.integers(1, 15, (N, n)) << 3 | z << 8).astype(np.uint16)
    return Weights(N, K, group, 0, quantised=(codes, words, r.integers(110, 116, N).astype(np.uint8)))


# tokens, rows, K: every kind of tiles with fp32 rows of x (tests/test_i4_exact_coverage_cpu.py)
TILES_F32 = [(17, 96, 544), (129, 1000, 736), (40, 4230, 416), (33, 4150, 4128), (90, 4230, 160), (70, 4100, 1120),
             (130, 4100, 2080), (68, 8202, 256), (70, 8202, 288), (40, 20028, 96), (70, 61128, 416), (214, 61128, 288)]


@pytest.mark.parametrize("T,N,K", TILES_F32)
def test_all_24_bits_of_fp32_numbers_on_every_kind_of_tiles(ctx, T, N, K):  # noqa: F811
    """Tokens of one number of 24 significant bits, at every slice of 32 k: each result is that number times a
    power of two, so a part of it that is left out or taken from elsewhere shows in the lowest bits."""
    group = 32 << N % 3
    w = powers(N, K, group, T + N)
    dw, v = w.upload(), Q.weights(*w.parts, group)
    r = np.random.default_rng(K)
    slices = K // 32
    for turn in range(-(-slices // T)):
        hot = (np.arange(T) + turn * T) % slices * 32 + r.integers(0, 32, T)
        x = np.zeros((T, K), np.float32)
        # (odd integers of 24 bits whose middle and last 8 bits are not zero)
        x[np.arange(T), hot] = (r.integers(128, 256, T) << 16 | r.integers(1, 256, T) << 8 | r.integers(0, 128, T) * 2 + 1)
        got = product(ctx, torch.from_numpy(x).cuda(), F32, K, T, w, dw, F32)
        assert np.array_equal(got, x[np.arange(T), hot].astype(np.float64)[:, None] * v[:, hot].T)


@pytest.mark.parametrize("T,N,K", [(1, 70, 288), (4, 70, 9248), (6, 70, 288), (8, 300, 4128), (20, 70, 1056), (70, 4100, 1120)])
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("power,exps", [(-116, 170), (-100, 200), (100, 30), (120, 40), (-124, 200), (-126, 200)])
def test_numbers_near_the_ends_of_fp32(ctx, T, N, K, xt, power, exps):  # noqa: F811
    """One power of two a token, against rows of weights as large as x is small: ordinary results, each exact."""
    group = 64
    w = Weights(N, K, group, 5)
    w.exps = (w.exps.astype(np.int64) - 113 + exps).astype(np.uint8)
    w.parts = (w.codes, w.words, w.exps)
    hot = np.random.default_rng(T).integers(0, K, T)
    x = torch.zeros((T, K), dtype=TORCH[xt])
    x[torch.arange(T), torch.from_numpy(hot)] = 2.0 ** power
    got = product(ctx, x.cuda(), xt, K, T, w, w.upload(), F32)
    assert np.array_equal(got, 2.0 ** power * Q.weights(*w.parts, group)[:, hot].T)


# tokens, rows, K: 128 rows of x a tile, split and wide, and 64
FAR = [(128, 4230, 160), (128, 8202, 256), (128, 61128, 416), (128, 40003, 96)]


@pytest.mark.parametrize("T,N,K", FAR)
def test_rows_of_x_almost_2_24_elements_apart(ctx, T, N, K):  # noqa: F811
    """Rows that are read in place, the last one almost 4 GiB behind the first (2 GiB on tiles of 64 rows)."""
    ld = (1 << 24) - 8
    w = Weights(N, K, 32, N)
    x = torch.zeros((T - 1) * ld + K, dtype=torch.bfloat16, device="cuda")
    some, ref = numbers((T, K), 8, BF16)
    x.as_strided((T, K), (ld, 1)).copy_(some)
    got = product(ctx, x, BF16, ld, T, w, w.upload(), F32)
    check(got, *Q.matmul_bound(ref, *w.parts, 32, "f32"))


FAR_EXPERTS = [(4096, 64, 2, 1, 0, 64, (1 << 19) - 16)]


@pytest.mark.parametrize("H,I,E,k,shared,group,T", FAR_EXPERTS)
def test_tokens_of_experts_that_end_just_below_4_gib(H, I, E, k, shared, group, T):
    """Gathered rows by 32-bit offsets up to their limit; rows at the ends and in the middle are checked."""
    layer = Layer(H, I, E, k, shared, group, 1)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    rows = np.array([0, 1, 255, 262143, 262144, 400001, T - 129, T - 2, T - 1])
    at = torch.from_numpy(rows).cuda()
    some, ref = numbers((len(rows), H), 3, BF16)
    x[at] = some
    ids = np.random.default_rng(1).integers(0, E, (T, 1)).astype(np.int32)
    o = layer.run(x, ids)
    got = o[at].double().cpu().numpy()
    for e in range(E):
        mine = ids[rows, 0] == e
        check(got[mine], *Q.expert_bound(ref[mine], *layer.parts[e], group))
    assert (o[T] == -7).all()
    o[at] = 0
    assert not bool(o[:T].any())
