"""Operators on 4-bit weights on the GPU: quantisation bit for bit, products and experts elementwise
within derived bounds of the 64-bit form."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
B = pytest.importorskip("expert_cached_moe_amd.binding")
from oracle import i4_oracle as Q, scored_oracle as S  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = 0, 1
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
NAME = {F32: "f32", BF16: "bf16"}


@pytest.fixture(scope="module")
def ctx():
    c = B.moe_create(B.make_config(64, 32, 1, 1))
    yield c
    B.moe_destroy(c)


def u8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def numbers(shape, seed, t, scale=1.0):
    """Numbers of a type as a tensor on the GPU and in fp64."""
    x = torch.from_numpy((np.random.default_rng(seed).normal(size=shape) * scale).astype(np.float32)).to(TORCH[t])
    return x.cuda(), x.double().numpy()


class Weights:
    """Rows of random codes with words and exponents of ordinary weights, or rows quantised by the oracle."""

    def __init__(self, N, K, group, seed, zero=True, quantised=None):
        r = np.random.default_rng(seed)
        n = -(-K // group)
        self.N, self.K, self.group = N, K, group
        if quantised is None:
            self.codes = r.integers(0, 16, (N, K)).astype(np.uint8)
            z = r.integers(0, 16, (N, n)) if zero else np.full((N, n), 8)
            self.words = (r.integers(0x08, 0x7F, (N, n)) | z << 8).astype(np.uint16)
            self.exps = r.integers(110, 116, N).astype(np.uint8)
        else:
            self.codes, self.words, self.exps = quantised
        self.parts = (self.codes, self.words, self.exps)

    def upload(self):
        return u8(Q.pack(self.codes)), u8(Q.lay_words(self.words).view(np.int16)), u8(self.exps)


# ------------------------------------------------------------------ quantisation

def quantize(ctx, x, t, ld, rows, cols, group, zero):
    n = -(-cols // group)
    q = torch.full((rows * cols // 2 + 16,), 0x5A, dtype=torch.uint8, device="cuda")
    w = torch.full((rows * n + 4,), 0x5A5A, dtype=torch.int16, device="cuda")
    e = torch.full((rows + 4,), 0x5A, dtype=torch.uint8, device="cuda")
    B.moe_i4_quantize(ctx, x, t, ld, rows, cols, group, zero, q, w, e)
    torch.cuda.synchronize()
    assert (q[rows * cols // 2:] == 0x5A).all() and (w[rows * n:] == 0x5A5A).all() and (e[rows:] == 0x5A).all()
    return (Q.unpack(q[:rows * cols // 2].cpu().numpy().reshape(rows, -1)),
            Q.unlay_words(w[:rows * n].cpu().numpy().view(np.uint16), rows, n), e[:rows].cpu().numpy())


def same(a, b):
    return all(np.array_equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("zero", [0, 1])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,cols,pad,off", [(1, 32, 0, 0), (3, 96, 0, 0), (17, 416, 5, 1), (5, 1568, 8, 0), (64, 2048, 0, 0),
                                              (2, 8224, 3, 3), (3, 20000, 0, 0)])
def test_quantize_bit_for_bit(ctx, rows, cols, pad, off, group, zero, t):
    x, ref = numbers((rows * (cols + pad) + off,), rows + cols, t, 0.02)
    x = x[off:]
    ref = ref[off:].reshape(rows, cols + pad)[:, :cols]
    assert same(quantize(ctx, x, t, cols + pad, rows, cols, group, zero), Q.quantize(ref, group, zero))


@pytest.mark.parametrize("zero", [0, 1])
@pytest.mark.parametrize("group", [32, 128])
def test_quantize_special_rows(ctx, group, zero):
    r = np.random.default_rng(3)
    K = 288
    x = r.normal(size=(24, K)).astype(np.float32)
    x[0] = 0
    x[1] = -0.0
    x[2] = 1e-45
    x[3] *= np.float32(2.0 ** -95)
    x[4] *= np.float32(2.0 ** -88)
    x[5, 40] = np.inf
    x[6, 287] = np.nan
    x[7, 0] = -np.inf
    x[8, 5] = 2.0 ** 120
    x[9, 5] = np.float32(2.0 ** 120) * (1 - 2.0 ** -24)
    x[10] = 3.0
    x[11] = -3.0
    x[12] = np.abs(x[12])
    x[13] = -np.abs(x[13])
    x[14, 100] = 1e6
    x[15, :32] = 0
    x[16] = 0
    x[16, 200] = 7 * 448 * 2.0 ** -3
    x[17] = 0
    x[17, 31] = 15 * 448.0
    x[18] = np.arange(K) % 15 - 7
    x[19] = (np.arange(K) % 16 - 7.5)
    x[20] = np.float32(2.0 ** -60)
    x[21, ::2] = 1e-6
    x[22] *= 1e30
    for t in (F32, BF16):
        d = torch.from_numpy(x).to(TORCH[t])
        assert same(quantize(ctx, d.cuda(), t, K, 24, K, group, zero), Q.quantize(d.double().numpy(), group, zero))


def test_quantize_rows_past_2_gib(ctx):
    """Rows 2^25 elements apart, 100 of them: offsets past 2^32 bytes."""
    ld, K = 1 << 25, 64
    x = torch.zeros(99 * ld + K, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn((100, K), device="cuda").to(torch.bfloat16)
    x.as_strided((100, K), (ld, 1)).copy_(rows)
    assert same(quantize(ctx, x, BF16, ld, 100, K, 32, 1), Q.quantize(rows.double().cpu().numpy(), 32, 1))


# ------------------------------------------------------------------ products

def product(ctx, x, xt, ld, T, w, dw, yt, pad=0, off=0, ws=None, s=None):
    ldy = w.N + pad
    y = torch.full((T * ldy + off + 8,), -7.0, dtype=TORCH[yt], device="cuda")
    if ws is None:
        ws = torch.empty(B.moe_i4_workspace_bytes(T, w.N, w.K), dtype=torch.uint8, device="cuda")
    B.moe_i4_matmul(ctx, x, xt, ld, T, *dw, w.N, w.K, w.group, y[off:], yt, ldy, ws, s)
    torch.cuda.synchronize()
    assert (y[:off] == -7).all() and (y[off + T * ldy:] == -7).all()
    v = y[off:off + T * ldy].view(T, ldy)
    assert (v[:, w.N:] == -7).all()
    return v[:, :w.N].double().cpu().numpy()


def check(got, ref, bound):
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (np.argwhere(bad)[:5], (np.abs(got - ref) / bound).max())


# tokens, rows, K: one token and up, every count of 4-token blocks, tiles' edges; K of one group and less,
# of several passes, of odd numbers of halves
SHAPES = [(1, 1, 32), (1, 33, 64), (1, 2048, 2048), (2, 100, 96), (3, 515, 416), (4, 64, 4096), (5, 31, 1568),
          (7, 130, 160), (8, 1000, 1536), (9, 257, 768), (12, 48, 8192), (13, 300, 4128), (16, 2051, 1024),
          (17, 96, 544), (31, 200, 2048), (33, 129, 96), (64, 512, 512), (65, 640, 1120), (100, 77, 12288),
          (127, 128, 64), (129, 1000, 736), (260, 515, 2080), (513, 384, 1024)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("xt,yt,pad,off", [(BF16, BF16, 0, 0), (BF16, F32, 8, 8), (F32, F32, 3, 1), (F32, BF16, 0, 2),
                                           (BF16, BF16, 1, 1)])
def test_matmul(ctx, T, N, K, group, xt, yt, pad, off):
    w = Weights(N, K, group, T + N + K)
    x, ref = numbers((T * (K + pad) + off,), T * N, xt)
    x, ref = x[off:], ref[off:].reshape(T, K + pad)[:, :K]
    got = product(ctx, x, xt, K + pad, T, w, w.upload(), yt, pad, off)
    check(got, *Q.matmul_bound(ref, *w.parts, group, NAME[yt], 3 if xt == F32 else 1))


# (each kind of tiles: tests/test_i4_coverage_cpu.py)
TILES = [(40, 4230, 416), (90, 4230, 160), (9, 8202, 160), (70, 8202, 288), (68, 8202, 256), (40, 20028, 96), (70, 61128, 416), (214, 61128, 288),
         (300, 40003, 352), (333, 61003, 96), (70, 61003, 96), (33, 4150, 4128), (70, 4100, 1120), (130, 4100, 2080)]


@pytest.mark.parametrize("T,N,K", TILES)
@pytest.mark.parametrize("xt,yt,pad,off", [(BF16, BF16, 0, 0), (BF16, F32, 8, 8), (F32, F32, 0, 0), (F32, BF16, 3, 1)])
def test_matmul_on_every_kind_of_tiles(ctx, T, N, K, xt, yt, pad, off):
    group = 32 << T % 3
    w = Weights(N, K, group, T + N + K)
    x, ref = numbers((T * (K + pad) + off,), T * N, xt)
    x, ref = x[off:], ref[off:].reshape(T, K + pad)[:, :K]
    got = product(ctx, x, xt, K + pad, T, w, w.upload(), yt, pad, off)
    check(got, *Q.matmul_bound(ref, *w.parts, group, NAME[yt], 3 if xt == F32 else 1))


@pytest.mark.parametrize("T", [1, 6, 16, 40, 200])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_matmul_is_as_good_as_fp32(ctx, T, xt):
    """Results in fp32 lie within a few fp32 steps of the exact ones, measured against the size of the
    sums: 40 steps of 2^-24 of the root of the sum of squares (errors of 128 groups' sums that add up
    at random, each up to 4 steps of sums up to 2.5 times the weights' size)."""
    N, K = 300, 4096
    r = np.random.default_rng(4)
    w = Weights(N, K, 64, 0, quantised=Q.quantize((r.normal(size=(N, K)) * 0.02).astype(np.float32), 64, 1))
    x, ref = numbers((T, K), 6, xt)
    got = product(ctx, x, xt, K, T, w, w.upload(), F32)
    v = Q.weights(*w.parts, 64)
    size = np.sqrt((ref ** 2) @ (v ** 2).T)
    assert (np.abs(got - ref @ v.T) <= 40 * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("T", [1, 5, 16, 20, 130])
def test_one_hot_tokens_return_the_weights(ctx, T):
    """Each result is one weight, exactly (both output types: eight significant bits)."""
    N, K, group = 70, 288, 32
    w = Weights(N, K, group, 5)
    hot = np.random.default_rng(T).integers(0, K, T)
    for xt in (F32, BF16):
        x = torch.zeros((T, K), dtype=TORCH[xt])
        x[torch.arange(T), torch.from_numpy(hot)] = 1
        for yt in (F32, BF16):
            got = product(ctx, x.cuda(), xt, K, T, w, w.upload(), yt)
            assert np.array_equal(got, Q.weights(*w.parts, group)[:, hot].T)


@pytest.mark.parametrize("T", [3, 16, 50, 300])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_tokens_with_infinities_and_nans_keep_to_themselves(ctx, T, xt):
    N, K, group = 60, 224, 64
    w = Weights(N, K, group, 2)
    x, ref = numbers((T, K), 3, xt)
    x[1, 5], x[T - 1, 223], x[T // 2, 100] = np.nan, np.inf, -np.inf
    bad = [1, T // 2, T - 1]
    good = [t for t in range(T) if t not in bad]
    got = product(ctx, x, xt, K, T, w, w.upload(), F32)
    bound = Q.matmul_bound(ref, *w.parts, group, "f32", 3)
    check(got[good], bound[0][good], bound[1][good])
    assert not np.isfinite(got[bad]).any()


@pytest.mark.parametrize("T", [2, 50])
def test_rows_of_nan_weights_and_of_every_word(ctx, T):
    """Exponent 255, the e4m3 NaN and negative scales; other rows are as they would be."""
    N, K, group = 300, 64, 32
    w = Weights(N, K, group, 1)
    w.words[:256, 0] = np.arange(256) | 9 << 8
    w.exps[260] = 255
    w.exps[261] = 1
    w.exps[262] = 250
    w.words[262] = 0x0801
    x, ref = numbers((T, K), 3, BF16)
    got = product(ctx, x, BF16, K, T, w, w.upload(), F32)
    nan = [0x7F, 0xFF, 260]
    assert np.isnan(got[:, nan]).all()
    rest = [n for n in range(N) if n not in nan]
    parts = tuple(p[rest] for p in w.parts)
    ref, bound = Q.matmul_bound(ref, *parts, group, "f32")
    check(got[:, rest], ref, bound)


@pytest.mark.parametrize("T", [4, 64])
def test_fp32_numbers_of_all_sizes(ctx, T):
    """The three parts of an fp32 number add up to it from 2^-100 to the end of the range."""
    N, K, group = 40, 96, 32
    w = Weights(N, K, group, 1, quantised=Q.quantize(np.random.default_rng(0).normal(size=(N, K)).astype(np.float32) * 1e-3, group, 0))
    r = np.random.default_rng(1)
    x = (r.normal(size=(T, K)) * np.exp2(r.integers(-90, 120, (T, 1)))).astype(np.float32)
    x[0] = np.float32(3.4028235e38) * np.where(r.random(K) < 0.5, 1, -1)
    x[1] = np.float32(1.1754944e-38) * 2.0 ** 20 * r.normal(size=K).astype(np.float32)
    got = product(ctx, torch.from_numpy(x).cuda(), F32, K, T, w, w.upload(), F32)
    ref, bound = Q.matmul_bound(x, *w.parts, group, "f32", 3)
    inside = np.abs(ref) < 3e38
    # (parts below 2^-126 may be lost: 96 of them)
    assert (np.abs(got - ref) <= bound + 96 * 2.0 ** -126 * np.abs(Q.weights(*w.parts, group)).max())[inside].all()


def test_offsets_past_2_gib_and_4_gib(ctx):
    """Codes past 2^32 bytes; rows of x and of y whose offsets pass 2^32 bytes."""
    N, K, group = 66000, 131072, 128
    q = torch.randint(0, 256, (N * (K // 2),), dtype=torch.uint8, device="cuda")
    words = torch.randint(0x30, 0x50, (N, K // group), dtype=torch.int16, device="cuda") | (7 << 8)
    exps = torch.full((N,), 112, dtype=torch.uint8, device="cuda")
    w = Weights(1, 32, 32, 0)
    w.N, w.K, w.group = N, K, group
    rows = [0, 1, 32767, 32768, 65535, 65536, 65999]
    at = torch.tensor(rows, device="cuda")
    words_of = words.view(N // 16, K // group, 16)[at // 16, :, at % 16]
    parts = (Q.unpack(q.view(N, K // 2)[at].cpu().numpy()), words_of.cpu().numpy().view(np.uint16), exps[at].cpu().numpy())
    for T in (1, 20):
        x, ref = numbers((T, K), 3, BF16)
        got = product(ctx, x, BF16, K, T, w, (q, words, exps), F32)
        check(got[:, rows], *Q.matmul_bound(ref, *parts, group, "f32"))
    del q, words, exps
    w = Weights(40, 64, 32, 1)
    for T in (9, 70):
        ld = (1 << 32) // (T - 2)
        ld -= ld % 8
        x = torch.zeros((T - 1) * ld + 64, dtype=torch.bfloat16, device="cuda")
        some, ref = numbers((T, 64), 8, BF16)
        x.as_strided((T, 64), (ld, 1)).copy_(some)
        y = torch.full(((T - 1) * ld + 41,), -7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(B.moe_i4_workspace_bytes(T, 40, 64), dtype=torch.uint8, device="cuda")
        B.moe_i4_matmul(ctx, x, BF16, ld, T, *w.upload(), 40, 64, 32, y, BF16, ld, ws)
        got = y.as_strided((T, 40), (ld, 1)).double().cpu().numpy()
        check(got, *Q.matmul_bound(ref, *w.parts, 32, "bf16"))
        assert y[40] == -7 and y[-1] == -7
        del x, y


def test_most_rows(ctx):
    """2^23 rows of weights, of x and of both kinds of results; rows at the ends and in the middle are checked."""
    N, K = 1 << 23, 32
    rows = np.array([0, 1, 4095, 4194303, 4194304, N - 17, N - 2, N - 1])
    at = torch.from_numpy(rows).cuda()
    g = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randn((N, K), generator=g, device="cuda", dtype=torch.bfloat16)
    q = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    words = torch.empty(N, dtype=torch.int16, device="cuda")
    exps = torch.empty(N, dtype=torch.uint8, device="cuda")
    B.moe_i4_quantize(ctx, w, BF16, K, N, K, 32, 1, q, words, exps)
    torch.cuda.synchronize()
    want = Q.quantize(w[at].double().cpu().numpy(), 32, 1)
    parts = (Q.unpack(q[at].cpu().numpy()), words[at].cpu().numpy().view(np.uint16)[:, None], exps[at].cpu().numpy())
    for have, ref in zip(parts, want):
        assert np.array_equal(have, ref)
    for T in (2, 9):
        x, ref = numbers((T, K), T, BF16)
        y = torch.full((T * N + 1,), -7.0, device="cuda")
        ws = torch.empty(B.moe_i4_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
        B.moe_i4_matmul(ctx, x, BF16, K, T, q, words, exps, N, K, 32, y, F32, N, ws)
        torch.cuda.synchronize()
        check(y[:T * N].view(T, N)[:, at].double().cpu().numpy(), *Q.matmul_bound(ref, *parts, 32, "f32"))
        assert y[T * N] == -7
    few = Weights(3, K, 32, 5)
    y = torch.full((N * 3 + 1,), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.moe_i4_workspace_bytes(N, 3, K), dtype=torch.uint8, device="cuda")
    B.moe_i4_matmul(ctx, w, BF16, K, N, *few.upload(), 3, K, 32, y, BF16, 3, ws)
    torch.cuda.synchronize()
    check(y[:N * 3].view(N, 3)[at].double().cpu().numpy(), *Q.matmul_bound(w[at].double().cpu().numpy(), *few.parts, 32, "bf16"))
    assert y[N * 3] == -7


@pytest.mark.parametrize("T", [3, 16, 40, 300])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_matmul_in_a_graph_on_another_stream_with_a_larger_workspace(ctx, T, xt):
    N, K, group = 200, 512, 64
    w = Weights(N, K, group, 7)
    dw = w.upload()
    ws = torch.full((B.moe_i4_workspace_bytes(8192, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
    x, ref = numbers((T, K), 1, xt)
    y = torch.empty((T, N), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.moe_i4_matmul(ctx, x, xt, K, T, *dw, N, K, group, y, F32, N, ws, side)
    for seed in range(2, 6):
        new, ref = numbers((T, K), seed, xt)
        x.copy_(new)
        y.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        first = y.cpu().numpy()
        check(first.astype(np.float64), *Q.matmul_bound(ref, *w.parts, group, "f32", 3))
        again = product(ctx, x, xt, K, T, w, dw, F32)
        assert np.array_equal(first, again)                    # the same sums in the same order


@pytest.mark.parametrize("T", [2, 40, 600])
def test_two_calls_at_once(ctx, T):
    """Two streams, each with its own workspace and results, the weights shared."""
    N, K, group = 1000, 1024, 64
    w = Weights(N, K, group, 7)
    dw = w.upload()
    xs = [numbers((T, K), seed, F32) for seed in (1, 2)]
    alone = [product(ctx, x, F32, K, T, w, dw, F32) for x, _ in xs]
    ys = [torch.empty((T, N), device="cuda") for _ in xs]
    ws = [torch.empty(B.moe_i4_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda") for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(10):
        for (x, _), y, work, s in zip(xs, ys, ws, streams):
            B.moe_i4_matmul(ctx, x, F32, K, T, *dw, N, K, group, y, F32, N, work, s)
    torch.cuda.synchronize()
    for y, one in zip(ys, alone):
        assert np.array_equal(y.double().cpu().numpy(), one)


# ------------------------------------------------------------------ experts

class Layer:
    """Experts of random weights, quantised by the library from bf16 blobs; the oracle's parts of each."""

    def __init__(self, H, I, E, k, shared, group, zero, seed=0, spare=1):
        self.H, self.I, self.E, self.k, self.n_shared, self.group = H, I, E, k, shared, group
        self.cfg = B.make_config(H, I, E, k, shared)
        self.ctx = B.moe_create(self.cfg)
        size = B.moe_i4_blob_bytes(self.cfg, group)
        self.pool = torch.full(((E + shared + spare) * size,), 0xFF, dtype=torch.uint8, device="cuda")
        r = np.random.default_rng(seed)
        self.slots = r.permutation(E + spare)[:E].tolist() if spare else list(range(E))
        self.parts = []
        for e in range(E + shared):
            w = [torch.from_numpy((r.normal(size=s) * 0.05).astype(np.float32)).to(torch.bfloat16)
                 for s in ((I, H), (I, H), (H, I))]
            bits = [t.view(torch.int16).numpy().view(np.uint16) for t in w]
            blob = np.empty(B.moe_expert_bytes(self.cfg), np.uint8)
            B.moe_pack_expert(self.cfg, *bits, None, None, None, blob)
            d = torch.from_numpy(blob).cuda()
            at = self.slots[e] if e < E else E + spare
            B.moe_i4_pack(self.ctx, d, group, zero, self.pool[at * size:])
            self.parts.append([Q.quantize(t.double().numpy(), group, zero) for t in w])
        self.shared = self.pool[(E + spare) * size:] if shared else None
        torch.cuda.synchronize()

    def __del__(self):
        B.moe_destroy(self.ctx)

    def run(self, x, ids, listed=None, with_shared=None, ws=None, s=None, o=None):
        T = x.shape[0]
        listed = list(range(self.E)) if listed is None else listed
        with_shared = self.n_shared if with_shared is None else with_shared
        _, offsets, perm, _ = S.group_pairs(ids, self.E)
        off, pm = u8(offsets.astype(np.int32)), u8(perm.astype(np.int32))
        if o is None:
            o = torch.full((T * self.k + T * self.n_shared + 1, self.H), -7.0, dtype=torch.bfloat16, device="cuda")
        if ws is None:
            ws = torch.full((B.moe_i4_expert_workspace_bytes(self.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        B.moe_i4_expert_ffn(self.ctx, x, T, off, pm, self.pool, listed, [self.slots[e] for e in listed], len(listed),
                            self.shared, with_shared, self.group, o, ws, s)
        torch.cuda.synchronize()
        return o

    def check(self, o, x, ids, listed=None, with_shared=None):
        """Every listed pair within its bound, everything else untouched."""
        T = len(x)
        listed = range(self.E) if listed is None else listed
        with_shared = self.n_shared if with_shared is None else with_shared
        got = o.double().cpu().numpy()
        left = np.ones(len(got), bool)
        flat = ids.ravel()
        for e in listed:
            at = np.nonzero(flat == e)[0]
            if len(at):
                check(got[at], *Q.expert_bound(x[at // self.k], *self.parts[e], self.group))
                left[at] = False
        if with_shared:
            at = T * self.k + np.arange(T)
            check(got[at], *Q.expert_bound(x, *self.parts[-1], self.group))
            left[at] = False
        assert (got[left] == -7).all()


def some_ids(T, E, k, seed, popular=0.0):
    r = np.random.default_rng(seed)
    return np.argsort(-(r.normal(size=(T, E)) + popular * r.normal(size=(1, E))), axis=1)[:, :k].astype(np.int32)


LAYERS = [(64, 32, 4, 2, 0, 32), (128, 96, 6, 3, 1, 64), (256, 160, 5, 1, 1, 128), (448, 416, 8, 4, 0, 128), (1024, 544, 4, 2, 1, 32)]
TOKENS = [1, 2, 4, 5, 8, 11, 16, 17, 40, 130, 300]


@pytest.mark.parametrize("zero", [0, 1])
@pytest.mark.parametrize("H,I,E,k,shared,group", LAYERS)
@pytest.mark.parametrize("T", TOKENS)
def test_experts(T, H, I, E, k, shared, group, zero):
    layer = Layer(H, I, E, k, shared, group, zero, seed=H)
    x, ref = numbers((T, H), T, BF16)
    ids = some_ids(T, E, k, T, 1.0)
    layer.check(layer.run(x, ids), ref, ids)


# (each kind of tiles for either product)
LARGE = [(384, 64, 2, 2, 0, 32, 1031), (128, 352, 2, 2, 0, 64, 1031), (192, 64, 2, 2, 0, 128, 1031), (128, 192, 2, 2, 0, 32, 1031),
         (192, 128, 2, 2, 0, 64, 2016), (256, 192, 2, 2, 0, 64, 2016), (128, 96, 8, 4, 1, 128, 1612), (192, 96, 8, 4, 1, 32, 1612),
         (64, 64, 8, 4, 1, 64, 1612), (384, 352, 4, 4, 1, 128, 1612), (704, 352, 4, 4, 1, 32, 1612), (256, 928, 2, 2, 1, 64, 2521),
         (1856, 256, 2, 2, 1, 128, 2521)]


@pytest.mark.parametrize("H,I,E,k,shared,group,T", LARGE)
def test_experts_on_every_kind_of_tiles(H, I, E, k, shared, group, T):
    layer = Layer(H, I, E, k, shared, group, T % 2, seed=H)
    x, ref = numbers((T, H), T, BF16)
    ids = some_ids(T, E, k, T, 1.0)
    layer.check(layer.run(x, ids), ref, ids)


@pytest.mark.parametrize("H,I,E,k,shared,group,T", LARGE)
def test_experts_on_every_kind_of_tiles(H, I, E, k, shared, group, T):
    layer = Layer(H, I, E, k, shared, group, T % 2, seed=H)
    x, ref = numbers((T, H), T, BF16)
    ids = some_ids(T, E, k, T, 1.0)
    layer.check(layer.run(x, ids), ref, ids)


def test_experts_of_tokens_past_4_gib():
    """x and o of 4 GiB and more; the last rows are checked."""
    H, I, T = 4096, 64, (1 << 19) + 300
    layer = Layer(H, I, 2, 1, 0, 64, 1)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    rows = np.array([0, 1, 255, 262143, 262144, 524287, 524288, T - 2, T - 1])
    some, ref = numbers((len(rows), H), 3, BF16)
    x[torch.from_numpy(rows).cuda()] = some
    ids = np.random.default_rng(1).integers(0, 2, (T, 1)).astype(np.int32)
    o = layer.run(x, ids)
    got = o[torch.from_numpy(rows).cuda()].double().cpu().numpy()
    for e in range(2):
        at = ids[rows, 0] == e
        check(got[at], *Q.expert_bound(ref[at], *layer.parts[e], layer.group))
    assert (o[T] == -7).all()
    few = torch.ones(T, dtype=torch.bool)
    few[rows] = False
    assert not bool(o[:T].any(dim=1).cpu()[few].any())


@pytest.mark.parametrize("T", [1, 6, 16, 64, 200])
def test_experts_not_listed_are_left_alone(T):
    layer = Layer(128, 96, 12, 3, 1, 64, 1)
    x, ref = numbers((T, 128), T, BF16)
    ids = some_ids(T, 12, 3, T)
    for listed, with_shared in (([3, 0, 11], 0), ([5], 1), ([], 1), (list(range(11, -1, -1)), 1)):
        layer.check(layer.run(x, ids, listed, with_shared), ref, ids, listed, with_shared)


@pytest.mark.parametrize("T", [9, 16, 90, 400])
def test_all_tokens_to_one_expert_and_experts_without_any(T):
    layer = Layer(192, 64, 300, 2, 0, 32, 0, spare=0)
    x, ref = numbers((T, 192), T, BF16)
    ids = np.tile(np.int32([[299, 7]]), (T, 1))
    layer.check(layer.run(x, ids), ref, ids)


def test_shared_expert_without_routed_ones():
    layer = Layer(128, 96, 4, 2, 1, 128, 1)
    for T in (1, 16, 50):
        x, ref = numbers((T, 128), T, BF16)
        o = torch.full((T * 3 + 1, 128), -7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(B.moe_i4_expert_workspace_bytes(layer.cfg, T), dtype=torch.uint8, device="cuda")
        B.moe_i4_expert_ffn(layer.ctx, x, T, None, None, None, None if T == 1 else [], None if T == 1 else [], 0, layer.shared, 1,
                            128, o, ws)
        torch.cuda.synchronize()
        layer.check(o, ref, np.zeros((T, 2), np.int32), [], 1)


@pytest.mark.parametrize("T", [4, 40])
def test_tokens_with_nans_keep_to_themselves(T):
    layer = Layer(128, 96, 6, 2, 1, 64, 1)
    x, ref = numbers((T, 128), 5, BF16)
    ids = some_ids(T, 6, 2, 3)
    x[2, 7], x[3, 100] = np.nan, np.inf
    o = layer.run(x, ids)
    bad = [p for p in range(T * 3) if (p // 2 if p < T * 2 else p - T * 2) in (2, 3)]
    assert not torch.isfinite(o[bad].float()).all(1).any()
    good = torch.ones(len(o), dtype=torch.bool)
    good[bad] = False
    clean = ref.copy()
    clean[2:4] = 0
    zeros = layer.run(torch.from_numpy(clean).to(torch.bfloat16).cuda(), ids)
    assert torch.equal(o[good], zeros[good])


@pytest.mark.parametrize("T", [3, 16, 70, 300])
def test_experts_in_a_graph_on_another_stream(T):
    """One graph for every routing: the tokens' experts are read on the device."""
    layer = Layer(256, 96, 10, 2, 1, 32, 1)
    off, pm = u8(np.zeros(11, np.int32)), u8(np.zeros(T * 2, np.int32))
    x, _ = numbers((T, 256), 0, BF16)
    o = torch.empty((T * 3 + 1, 256), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.moe_i4_expert_workspace_bytes(layer.cfg, 1000), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.moe_i4_expert_ffn(layer.ctx, x, T, off, pm, layer.pool, range(10), layer.slots, 10, layer.shared, 1, 32, o, ws, side)
    for seed in range(1, 5):
        new, ref = numbers((T, 256), seed, BF16)
        ids = some_ids(T, 10, 2, seed, 2.0)
        _, offsets, perm, _ = S.group_pairs(ids, 10)
        x.copy_(new)
        off.copy_(u8(offsets.astype(np.int32)))
        pm.copy_(u8(perm.astype(np.int32)))
        o.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        layer.check(o, ref, ids)
        assert torch.equal(layer.run(x, ids), o)


def test_same_numbers_as_the_layer_on_the_weights_that_the_codes_stand_for():
    """The 4-bit weights are exact in bf16, so moe_expert_ffn on a blob of them computes the same values
    within both calls' roundings."""
    H, I, E, k, group, T = 256, 128, 6, 2, 64, 50
    layer = Layer(H, I, E, k, 0, group, 1, spare=0)
    blobs = []
    for e in range(E):
        bits = [torch.from_numpy(Q.weights(*p, group)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
                for p in layer.parts[e]]
        blob = np.empty(B.moe_expert_bytes(layer.cfg), np.uint8)
        B.moe_pack_expert(layer.cfg, *bits, None, None, None, blob)
        blobs.append(blob)
    pool = torch.from_numpy(np.concatenate(blobs)).cuda()
    x, ref = numbers((T, H), 1, BF16)
    ids = some_ids(T, E, k, 2)
    o = layer.run(x, ids)
    _, offsets, perm, _ = S.group_pairs(ids, E)
    other = torch.empty_like(o)
    ws = torch.empty(B.moe_workspace_bytes(layer.cfg, T), dtype=torch.uint8, device="cuda")
    B.moe_expert_ffn(layer.ctx, x, T, None, u8(offsets.astype(np.int32)), u8(perm.astype(np.int32)), pool, range(E), range(E),
                     E, None, 0, other, ws)
    torch.cuda.synchronize()
    a, b = o[:T * k].double().cpu().numpy(), other[:T * k].double().cpu().numpy()
    bound = np.empty_like(a)
    for e in range(E):
        at = np.nonzero(ids.ravel() == e)[0]
        bound[at] = Q.expert_bound(ref[at // k], *layer.parts[e], group)[1]
    assert (np.abs(a - b) <= 2 * bound).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("T", [1, 4, 16, 90])
def test_a_layer_step_from_logits_to_the_head(T):
    """Router logits, router by scores, 4-bit experts with the shared one, merge, 4-bit output head: one
    stream, no host copy, captured and replayed; against the 64-bit form of each step on its own inputs."""
    H, I, E, k, group, N = 256, 96, 16, 4, 64, 333
    layer = Layer(H, I, E, k, 1, group, 1, seed=9)
    head = Weights(N, H, 32, 4)
    dh = head.upload()
    r = np.random.default_rng(1)
    wr, bias = (r.normal(size=(E, H)) * 0.1).astype(np.float32), (r.normal(size=E) * 0.1).astype(np.float32)
    dwr, db = u8(wr), u8(bias)
    rule = B.make_route_rule(B.MOE_SCORE_SIGMOID, 4, 2, 2, 1, 2.5)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    logits, w = torch.empty((T, E), device="cuda"), torch.empty((T, k), device="cuda")
    ids, perm, inv = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(3))
    counts, offsets = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    o = torch.full((T * (k + 1) + 1, H), -7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((T, N), device="cuda")
    ws = torch.empty(max(B.moe_workspace_bytes(layer.cfg, T), B.moe_i4_expert_workspace_bytes(layer.cfg, T),
                         B.moe_i4_workspace_bytes(T, N, H)), dtype=torch.uint8, device="cuda")

    def step(s):
        B.moe_router_logits(layer.ctx, x, T, dwr, logits, s)
        B.moe_route_scored(layer.ctx, logits, db, T, rule, ids, w, counts, offsets, perm, inv, ws, s)
        B.moe_i4_expert_ffn(layer.ctx, x, T, offsets, perm, layer.pool, range(E), layer.slots, E, layer.shared, 1, group, o,
                            ws, s)
        B.moe_merge_partial(layer.ctx, o, ids, w, range(E), E, 1, None, T, out, s)
        B.moe_i4_matmul(layer.ctx, out, BF16, H, T, *dh, N, H, 32, y, F32, N, ws, s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for seed in range(3):
        new, ref = numbers((T, H), seed, BF16)
        x.copy_(new)
        if seed < 2:
            graph.replay()
        else:
            step(None)
        torch.cuda.synchronize()
        got = logits.cpu().numpy()
        assert np.abs(got - ref @ wr.T.astype(np.float64)).max() <= Q.gamma(H) * (np.abs(ref) @ np.abs(wr).T).max()
        s, want = S.choose(got, bias, k, "sigmoid", 4, 2, 2)
        gates = S.gates(s, want, 1, 2.5)
        i = ids.cpu().numpy().reshape(T, k)
        assert np.array_equal(i, want)
        layer.check(o, ref, want)
        ob = o.double().cpu().numpy()
        pairs, shared = ob[:T * k].reshape(T, k, H), ob[T * k:T * (k + 1)]
        merged = (gates[:, :, None] * pairs).sum(1) + shared
        terms = (np.abs(gates[:, :, None] * pairs)).sum(1) + np.abs(shared)
        a = out.double().cpu().numpy()
        assert (np.abs(a - merged) <= np.abs(merged) * 2.0 ** -8 + 2 * (k + 2) * 2.0 ** -24 * terms).all()
        check(y.double().cpu().numpy(), *Q.matmul_bound(a, *head.parts, 32, "f32"))
