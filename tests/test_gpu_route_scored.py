"""The router by scores and its gradient on the GPU against the 64-bit form."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
B = pytest.importorskip("expert_cached_moe_amd.binding")
from oracle import scored_oracle as S  # noqa: E402

pytestmark = pytest.mark.gpu

KIND = {"softmax": 0, "sigmoid": 1}
POISON = -77


class Router:
    def __init__(self, E, k, T, kind, groups=1, keep=1, top=1, renorm=1, scale=1.0):
        self.cfg = B.make_config(64, 32, E, k)
        self.ctx = B.moe_create(self.cfg)
        self.E, self.k, self.kind, self.groups, self.keep, self.top = E, k, kind, groups, keep, top
        self.renorm, self.scale = renorm, float(np.float32(scale))
        self.rule = B.make_route_rule(KIND[kind], groups, keep, top, renorm, scale)
        self.T = T
        n = T * k

        def whole(m):
            return torch.full((m + 8,), POISON, dtype=torch.int32, device="cuda")
        self.ids, self.counts, self.offsets, self.perm, self.inv = whole(n), whole(E), whole(E + 1), whole(n), whole(n)
        self.w = torch.full((n + 8,), float(POISON), device="cuda")
        self.d = torch.full((T * E + 8,), float(POISON), device="cuda")
        self.ws = torch.empty(B.moe_workspace_bytes(self.cfg, T), dtype=torch.uint8, device="cuda")

    def __del__(self):
        B.moe_destroy(self.ctx)

    def forward(self, logits, bias, s=None):
        B.moe_route_scored(self.ctx, logits, bias, self.T, self.rule, self.ids, self.w, self.counts, self.offsets,
                           self.perm, self.inv, self.ws, s)

    def backward(self, logits, dw, s=None):
        B.moe_route_scored_backward(self.ctx, logits, self.T, self.rule, self.ids, dw, self.d, s)

    def results(self):
        torch.cuda.synchronize()
        n = self.T * self.k
        for t, m in ((self.ids, n), (self.counts, self.E), (self.offsets, self.E + 1), (self.perm, n), (self.inv, n),
                     (self.w, n)):
            assert (t[m:] == POISON).all()                    # nothing behind the outputs
        return (self.ids[:n].cpu().numpy().reshape(self.T, self.k), self.w[:n].cpu().numpy().reshape(self.T, self.k))

    def check(self, logits, bias):
        """ids and grouping equal; gates within one rounding to fp32 of the 64-bit form."""
        ids, w = self.results()
        s, ref = S.choose(logits, bias, self.k, self.kind, self.groups, self.keep, self.top)
        assert np.array_equal(ids, ref)
        g = S.gates(s, ref, self.renorm, self.scale)
        # (the 64-bit arithmetic: some 40 operations of 2^-53; results below 2^-126 by half of 2^-149)
        assert (np.abs(w - g) <= np.abs(g) * (2.0 ** -24 + 2.0 ** -46) + 2.0 ** -149).all()
        counts, offsets, perm, inv = S.group_pairs(ref, self.E)
        n = self.T * self.k
        assert np.array_equal(self.counts[:self.E].cpu(), counts) and np.array_equal(self.offsets[:self.E + 1].cpu(), offsets)
        assert np.array_equal(self.perm[:n].cpu(), perm) and np.array_equal(self.inv[:n].cpu(), inv)
        return ref

    def check_gradient(self, logits, ids, dw):
        torch.cuda.synchronize()
        assert (self.d[self.T * self.E:] == POISON).all()
        d = self.d[:self.T * self.E].cpu().numpy().reshape(self.T, self.E)
        ref = S.backward(logits, ids, dw, self.kind, self.renorm, self.scale)
        # cancelling terms: sums of up to 16 products of scale * dw and factors below 1 (over the
        # chosen scores' sum where they are renormalised, times p: below 1 again)
        size = np.abs(self.scale * dw).sum(1, keepdims=True)
        assert (np.abs(d - ref) <= np.abs(ref) * 2.0 ** -24 + size * 2.0 ** -46 + 2.0 ** -149).all()


def draw(T, E, seed, biased=True, k=1):
    r = np.random.default_rng(seed)
    return (r.normal(size=(T, E)).astype(np.float32) * 2, (r.normal(size=E) * 0.1).astype(np.float32) if biased else None,
            r.normal(size=(T, k)).astype(np.float32))


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


# T, E, k, groups, keep, top: every number of experts a lane, of waves (1, 2, 4, 8, 16), of 16 lanes (4, 8, 12, 16) and of 32
# (above 2,048 tokens), with and without groups; one workgroup (16 tokens and 64 pairs) and several, of 4, 8 and more
# than 64 tokens; E that fill no wave; whole groups of one expert
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 8, 2, 1, 1, 1), (4, 256, 8, 8, 4, 2), (3, 512, 16, 1, 1, 1), (1, 512, 16, 1, 1, 2),
          (64, 64, 1, 64, 33, 2), (5, 495, 12, 33, 20, 2), (30, 500, 10, 5, 2, 2), (63, 141, 6, 3, 1, 1),
          (129, 160, 8, 8, 3, 2), (700, 128, 8, 1, 1, 1), (515, 256, 8, 8, 4, 2), (1021, 141, 6, 1, 1, 1),
          (333, 510, 7, 17, 9, 1), (200, 65, 3, 13, 13, 2), (97, 12, 4, 2, 1, 2), (640, 7, 7, 7, 7, 1),
          (6, 100, 3, 1, 1, 1), (100, 512, 4, 1, 1, 1), (17, 9, 1, 3, 2, 1), (256, 24, 2, 1, 1, 1), (257, 24, 3, 2, 1, 2), (2049, 64, 1, 1, 1, 1), (2051, 128, 8, 1, 1, 1),
          (2050, 141, 6, 1, 1, 1), (4099, 256, 8, 8, 4, 2), (2100, 300, 5, 1, 1, 1), (2053, 512, 3, 32, 9, 2), (2060, 504, 4, 9, 5, 2),
          (2070, 48, 16, 16, 16, 2), (20001, 32, 2, 4, 2, 1),
          (70001, 9, 2, 1, 1, 1)]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("biased", [0, 1])
@pytest.mark.parametrize("T,E,k,groups,keep,top", SHAPES)
def test_choice_gates_grouping_and_gradient(T, E, k, groups, keep, top, biased, renorm, kind):
    r = Router(E, k, T, kind, groups, keep, top, renorm, 2.5)
    logits, bias, dw = draw(T, E, T * 1000 + E, biased, k)
    dl = cuda(logits)
    r.forward(dl, cuda(bias))
    ids = r.check(logits, bias)
    r.backward(dl, cuda(dw))
    r.check_gradient(logits, ids, dw)


@pytest.mark.parametrize("T", [64512, 64513, 1 << 24])
def test_many_tokens_to_one_expert(T):
    """The most tokens whose counts are bytes and one more; 2^24 tokens, 32,768 a workgroup (counts of 16 bits)."""
    E = 2
    for favour in (9.0, 0.0):
        r = Router(E, 1, T, "sigmoid", renorm=0)
        logits = torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
        logits[32768:65536, 0] = 9.0
        logits[:, 1] += favour * (T < 1 << 20)
        r.forward(logits, None)
        torch.cuda.synchronize()
        ids = (logits[:, 1] > logits[:, 0]).int()
        assert torch.equal(r.ids[:T], ids)
        order = torch.sort(ids, stable=True).indices.int()
        assert torch.equal(r.perm[:T], order)
        assert torch.equal(r.perm[:T][r.inv[:T].long()], torch.arange(T, dtype=torch.int32, device="cuda"))
        n = int((ids == 0).sum())
        assert r.counts[:2].tolist() == [n, T - n] and r.offsets[:3].tolist() == [0, n, T]
    r = Router(E, 1, T, "softmax", renorm=0)
    logits[:, 0], logits[:, 1] = 1.0, -1.0
    r.forward(logits, None)
    torch.cuda.synchronize()
    assert r.counts[:2].tolist() == [T, 0] and bool((r.perm[:T] == torch.arange(T, device="cuda")).all())


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_prefill_chunk(kind):
    r = Router(256, 8, 8192, kind, 8, 4, 2, 1, 2.5)
    logits, bias, dw = draw(8192, 256, 3, True, 8)
    dl = cuda(logits)
    r.forward(dl, cuda(bias))
    ids = r.check(logits, bias)
    r.backward(dl, cuda(dw))
    r.check_gradient(logits, ids, dw)


@pytest.mark.parametrize("T", [2, 40, 300, 2101])
@pytest.mark.parametrize("kind,groups", [("softmax", 1), ("sigmoid", 1), ("sigmoid", 4)])
def test_equal_values_take_the_lower_id(T, kind, groups):
    """All equal; few distinct values; zeros of both signs."""
    E, k = 48, 6
    r = Router(E, k, T, kind, groups, max(1, groups // 2), 2, 1)
    rng = np.random.default_rng(T)
    for logits in (np.zeros((T, E)), rng.integers(0, 3, (T, E)), np.where(rng.random((T, E)) < 0.5, 0.0, -0.0)):
        logits = logits.astype(np.float32)
        for bias in (None, np.zeros(E, np.float32), np.tile(np.float32([0.5, 0.25]), E // 2)):
            r.forward(cuda(logits), cuda(bias))
            r.check(logits, bias)


@pytest.mark.parametrize("T", [6, 70, 2102])
def test_values_that_fp32_does_not_tell_apart(T):
    """Equal logits and biases 2^-25 apart around 1/4: the biased scores differ by less than the upper
    32 bits of a 64-bit number show, some by less than fp32's rounding of 3/4."""
    E, k = 64, 8
    rng = np.random.default_rng(1)
    bias = (0.25 + rng.permutation(E) * 2.0 ** -25).astype(np.float32)
    logits = np.zeros((T, E), np.float32)
    for groups in (1, 4):
        r = Router(E, k, T, "sigmoid", groups, groups, 2)
        r.forward(cuda(logits), cuda(bias))
        r.check(logits, bias)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("biased", [0, 1])
@pytest.mark.parametrize("T", [12, 40, 2103])
def test_masked_experts_and_rows_without_any(T, kind, renorm, biased):
    """Logits of -infinity score 0 and come last; a row of nothing else has gates 0; large logits saturate."""
    E, k = 32, 4
    logits, bias, dw = draw(T, E, 9, biased, k)
    rng = np.random.default_rng(2)
    logits[rng.random((T, E)) < 0.7] = -np.inf
    logits[3] = -np.inf
    logits[4, :2] = 1.0
    logits[4, 2:] = -np.inf
    logits[5] = -3.0e38
    logits[6] = 3.0e38
    logits[7, 1:] = -1000.0
    for groups in (1, 8):
        r = Router(E, k, T, kind, groups, groups, 2, renorm)
        r.forward(cuda(logits), cuda(bias))
        ids = r.check(logits, bias)
        r.backward(cuda(logits), cuda(dw))
        r.check_gradient(logits, ids, dw)


def test_masked_by_the_bias():
    T, E, k = 33, 24, 4
    logits, bias, _ = draw(T, E, 4)
    bias[::3] = -np.inf
    for groups in (1, 6):
        r = Router(E, k, T, "sigmoid", groups, groups, 1)
        r.forward(cuda(logits), cuda(bias))
        r.check(logits, bias)


@pytest.mark.parametrize("T", [6, 50, 600, 2104])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_a_token_with_nans_keeps_to_itself(T, kind):
    E, k = 40, 8
    logits, bias, _ = draw(T, E, 8)
    bad = [1, T - 2]
    logits[bad[0]] = np.nan
    logits[bad[1], ::2] = np.nan
    logits[bad[1], 1] = np.inf
    for b in (None, bias):
        for groups in (1, 4):
            r = Router(E, k, T, kind, groups, 2 if groups > 1 else 1, 2)
            r.forward(cuda(logits), cuda(b))
            ids, w = r.results()
            good = [t for t in range(T) if t not in bad]
            s, ref = S.choose(logits[good], b, k, kind, groups, 2 if groups > 1 else 1, 2)
            assert np.array_equal(ids[good], ref)
            assert np.isfinite(w[good]).all()
            for t in bad:
                assert len(set(ids[t].tolist())) == k and ids[t].min() >= 0 and ids[t].max() < E
            _, offsets, perm, inv = S.group_pairs(ids, E)
            assert np.array_equal(r.perm[:T * k].cpu(), perm) and np.array_equal(r.inv[:T * k].cpu(), inv)


def test_no_tokens():
    r = Router(16, 2, 0, "sigmoid")
    r.forward(None, None)
    r.results()
    assert (r.counts[:16] == 0).all() and (r.offsets[:17] == 0).all()


def test_ids_outside_count_as_none_chosen():
    T, E, k = 5, 20, 3
    logits, _, dw = draw(T, E, 5, False, k)
    ids = np.tile(np.int32([2, 7, 11]), (T, 1))
    for bad in (-1, -5, 20, 1 << 30):
        for kind in KIND:
            for renorm in (0, 1):
                r = Router(E, k, T, kind, renorm=renorm)
                r.ids[:T * k] = torch.from_numpy(ids.ravel()).cuda()
                r.ids[1] = bad
                r.backward(cuda(logits), cuda(dw))
                torch.cuda.synchronize()
                d = r.d[:T * E].cpu().numpy().reshape(T, E)
                two = S.backward(logits[:1], ids[:1, [0, 2]], dw[:1, [0, 2]], kind, renorm, 1.0)
                assert np.abs(d[:1] - two).max() <= 2.0 ** -23 * np.abs(dw).sum()
                assert np.abs(d[1:] - S.backward(logits[1:], ids[1:], dw[1:], kind, renorm, 1.0)).max() <= 2.0 ** -23 * np.abs(dw).sum()


def test_agrees_with_the_softmax_router():
    """Without bias and groups the choice and the grouping are moe_route's, the gates its within fp32."""
    T, E, k = 900, 128, 8
    logits, _, _ = draw(T, E, 12, False)
    dl = cuda(logits)
    for renorm in (0, 1):
        r = Router(E, k, T, "softmax", renorm=renorm)
        r.forward(dl, None)
        ids, w = r.results()
        cfg = B.make_config(64, 32, E, k, renormalize=renorm)
        ctx = B.moe_create(cfg)
        i = [torch.empty_like(t) for t in (r.ids, r.counts, r.offsets, r.perm, r.inv)]
        g = torch.empty_like(r.w)
        B.moe_route(ctx, dl, T, i[0], g, *i[1:], r.ws)
        torch.cuda.synchronize()
        B.moe_destroy(ctx)
        n = T * k
        assert torch.equal(i[0][:n], r.ids[:n]) and torch.equal(i[3][:n], r.perm[:n]) and torch.equal(i[4][:n], r.inv[:n])
        # expf within 2 steps, a sum of up to 128 of them, a division
        assert np.abs(g[:n].cpu().numpy().reshape(T, k) / w - 1).max() < 140 * 2.0 ** -24


@pytest.mark.parametrize("T", [4, 60, 700, 2500])
def test_on_another_stream_and_in_a_graph(T):
    """Replays on new inputs, with eager calls and other work between them."""
    E, k = 96, 4
    r = Router(E, k, T, "sigmoid", 8, 4, 2)
    logits, bias, dw = draw(T, E, 20, True, k)
    dl, db, dd = cuda(logits), cuda(bias), cuda(dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.forward(dl, db, side)
        r.backward(dl, dd, side)
    ids = r.check(logits, bias)
    r.check_gradient(logits, ids, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r.forward(dl, db, side)
        r.backward(dl, dd, side)
    other = Router(E, k, T, "softmax")
    for seed in range(21, 25):
        logits, _, dw = draw(T, E, seed, True, k)
        dl.copy_(cuda(logits))
        dd.copy_(cuda(dw))
        for t in (r.ids, r.perm, r.inv, r.counts, r.offsets):
            t.fill_(POISON)
        r.w.fill_(POISON)
        r.d.fill_(POISON)
        graph.replay()
        ids = r.check(logits, bias)
        r.check_gradient(logits, ids, dw)
        other.forward(dl, None)
        other.check(logits, None)
