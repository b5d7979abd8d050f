"""4-bit weights without a GPU: refusals, sizes, and the 64-bit form against its definition."""
import numpy as np
import pytest

from oracle import i4_oracle as Q

B = pytest.importorskip("expert_cached_moe_amd.binding")

FAKE = 0x1000           # an address that a refused call does not touch; 256-byte aligned


@pytest.fixture
def ctx():
    c = B.moe_create(B.make_config(128, 96, 8, 2, 1))
    yield c
    B.moe_destroy(c)


def refused(status, f, *a):
    with pytest.raises(B.MoeError) as e:
        f(*a)
    assert e.value.status == status, str(e.value)


def quantize(ctx, x=FAKE, x_type=1, ld=64, rows=3, cols=64, group=32, zero=0, q=FAKE, words=FAKE, exps=FAKE):
    B.moe_i4_quantize(ctx, x, x_type, ld, rows, cols, group, zero, q, words, exps)


def matmul(ctx, x=FAKE, x_type=1, ld=64, T=3, w=FAKE, words=FAKE, exps=FAKE, N=5, K=64, group=32, y=FAKE, y_type=1, ld_y=5,
           ws=FAKE):
    B.moe_i4_matmul(ctx, x, x_type, ld, T, w, words, exps, N, K, group, y, y_type, ld_y, ws)


def experts(ctx, x=FAKE, T=3, offsets=FAKE, perm=FAKE, base=FAKE, ids=(0, 5), slots=(0, 1), n=2, shared=FAKE, with_shared=1,
            group=64, o=FAKE, ws=FAKE):
    B.moe_i4_expert_ffn(ctx, x, T, offsets, perm, base, ids, slots, n, shared, with_shared, group, o, ws)


@pytest.mark.parametrize("status,args", [
    (B.MOE_EINVAL, dict(x_type=2)), (B.MOE_EINVAL, dict(group=16)), (B.MOE_EINVAL, dict(group=256)), (B.MOE_EINVAL, dict(zero=2)),
    (B.MOE_EINVAL, dict(rows=-1)), (B.MOE_EINVAL, dict(ld=63)), (B.MOE_EINVAL, dict(x=None)), (B.MOE_EINVAL, dict(q=None)),
    (B.MOE_EINVAL, dict(words=None)), (B.MOE_EINVAL, dict(exps=None)), (B.MOE_EINVAL, dict(x=FAKE + 1)),
    (B.MOE_EINVAL, dict(x=FAKE + 2, x_type=0)), (B.MOE_EINVAL, dict(q=FAKE + 8)), (B.MOE_EINVAL, dict(words=FAKE + 1)),
    (B.MOE_ESHAPE, dict(cols=48)), (B.MOE_ESHAPE, dict(cols=0)), (B.MOE_ESHAPE, dict(cols=(1 << 20) + 32, ld=1 << 21)),
    (B.MOE_ESHAPE, dict(rows=(1 << 23) + 1))])
def test_quantize_refusals(ctx, status, args):
    refused(status, lambda: quantize(ctx, **args))


@pytest.mark.parametrize("status,args", [
    (B.MOE_EINVAL, dict(x_type=2)), (B.MOE_EINVAL, dict(y_type=2)), (B.MOE_EINVAL, dict(group=96)), (B.MOE_EINVAL, dict(T=-1)),
    (B.MOE_EINVAL, dict(ld=63)), (B.MOE_EINVAL, dict(ld_y=4)), (B.MOE_EINVAL, dict(x=None)), (B.MOE_EINVAL, dict(w=None)),
    (B.MOE_EINVAL, dict(words=None)), (B.MOE_EINVAL, dict(exps=None)), (B.MOE_EINVAL, dict(y=None)), (B.MOE_EINVAL, dict(ws=None)),
    (B.MOE_EINVAL, dict(x=FAKE + 1)), (B.MOE_EINVAL, dict(w=FAKE + 8)), (B.MOE_EINVAL, dict(words=FAKE + 1)),
    (B.MOE_EINVAL, dict(y=FAKE + 1)), (B.MOE_EINVAL, dict(y=FAKE + 2, y_type=0)), (B.MOE_EINVAL, dict(ws=FAKE + 16)),
    (B.MOE_ESHAPE, dict(K=40)), (B.MOE_ESHAPE, dict(K=0)), (B.MOE_ESHAPE, dict(K=(1 << 20) + 32)), (B.MOE_ESHAPE, dict(N=0)),
    (B.MOE_ESHAPE, dict(N=(1 << 23) + 1)), (B.MOE_ESHAPE, dict(T=(1 << 23) + 1)),
    (B.MOE_ESHAPE, dict(T=1 << 20, N=(1 << 16) + 1, ld_y=1 << 17))])
def test_matmul_refusals(ctx, status, args):
    refused(status, lambda: matmul(ctx, **args))


@pytest.mark.parametrize("status,args", [
    (B.MOE_EINVAL, dict(T=-1)), (B.MOE_EINVAL, dict(n=-1)), (B.MOE_EINVAL, dict(n=9)), (B.MOE_EINVAL, dict(with_shared=2)),
    (B.MOE_EINVAL, dict(shared=None)), (B.MOE_EINVAL, dict(group=48)), (B.MOE_EINVAL, dict(ids=None)),
    (B.MOE_EINVAL, dict(slots=None)), (B.MOE_EINVAL, dict(ids=(0, 8))), (B.MOE_EINVAL, dict(ids=(-1, 2))),
    (B.MOE_EINVAL, dict(ids=(3, 3))), (B.MOE_EINVAL, dict(slots=(0, -1))), (B.MOE_EINVAL, dict(slots=(0, 1 << 21))),
    (B.MOE_EINVAL, dict(x=None)), (B.MOE_EINVAL, dict(o=None)), (B.MOE_EINVAL, dict(ws=None)), (B.MOE_EINVAL, dict(offsets=None)),
    (B.MOE_EINVAL, dict(perm=None)), (B.MOE_EINVAL, dict(base=None)), (B.MOE_EINVAL, dict(x=FAKE + 8)),
    (B.MOE_EINVAL, dict(o=FAKE + 8)), (B.MOE_EINVAL, dict(ws=FAKE + 16)), (B.MOE_EINVAL, dict(base=FAKE + 16)),
    (B.MOE_EINVAL, dict(shared=FAKE + 16)), (B.MOE_ESHAPE, dict(T=(1 << 23) + 1))])
def test_expert_refusals(ctx, status, args):
    refused(status, lambda: experts(ctx, **args))


def test_calls_that_do_nothing(ctx):
    quantize(ctx, rows=0, x=None, q=None, words=None, exps=None)
    matmul(ctx, T=0, x=None, w=None, words=None, exps=None, y=None, ws=None)
    experts(ctx, T=0, x=None, o=None, ws=None)
    experts(ctx, n=0, with_shared=0, x=None, o=None, ws=None, offsets=None, perm=None, base=None, shared=None)


def test_pack_refusals(ctx):
    for a in ((None, 64, 0, FAKE), (FAKE, 64, 0, None), (FAKE, 65, 0, FAKE), (FAKE, 64, 2, FAKE), (FAKE + 16, 64, 0, FAKE),
              (FAKE, 64, 0, FAKE + 16)):
        refused(B.MOE_EINVAL, B.moe_i4_pack, ctx, *a)


@pytest.mark.parametrize("w", [B.MOE_W_F32, B.MOE_W_MXFP4])
def test_contexts_of_other_weights_are_refused(w):
    cfg = B.make_config(256, 96, 8, 2, 1, w_dtype=w)
    c = B.moe_create(cfg)
    refused(B.MOE_EUNSUPPORTED, B.moe_i4_blob_bytes, cfg, 64)
    refused(B.MOE_EUNSUPPORTED, B.moe_i4_expert_workspace_bytes, cfg, 4)
    refused(B.MOE_EUNSUPPORTED, B.moe_i4_pack, c, FAKE, 64, 0, FAKE)
    refused(B.MOE_EUNSUPPORTED, lambda: experts(c))
    B.moe_destroy(c)


def test_sizes():
    cfg = B.make_config(128, 96, 8, 2, 1)

    def up(n):
        return -(-n // 256) * 256
    for G in (32, 64, 128):
        g, d = -(-128 // G), -(-96 // G)
        assert B.moe_i4_blob_bytes(cfg, G) == sum(map(up, (192 * 64, 192 * g * 2, 192, 128 * 48, 128 * d * 2, 128)))
    refused(B.MOE_EINVAL, B.moe_i4_blob_bytes, cfg, 1)
    refused(B.MOE_ESHAPE, B.moe_i4_blob_bytes, B.make_config((1 << 20) + 64, 32, 1, 1), 32)
    refused(B.MOE_EINVAL, B.moe_i4_expert_workspace_bytes, cfg, -1)
    refused(B.MOE_ESHAPE, B.moe_i4_expert_workspace_bytes, cfg, (1 << 23) + 1)
    sizes = [B.moe_i4_expert_workspace_bytes(cfg, T) for T in (0, 1, 7, 100, 8192)]
    assert sizes == sorted(sizes)
    refused(B.MOE_EINVAL, B.moe_i4_workspace_bytes, -1, 8, 64)
    for a in ((4, 0, 64), (4, 8, 40), (4, 8, 0), (4, (1 << 23) + 1, 64), ((1 << 23) + 1, 8, 64), (4, 8, (1 << 20) + 32)):
        refused(B.MOE_ESHAPE, B.moe_i4_workspace_bytes, *a)
    for N, K in ((5, 64), (100003, 4096), (64, 12288)):
        sizes = [B.moe_i4_workspace_bytes(T, N, K) for T in (0, 1, 16, 17, 100, 256, 8192, 1 << 20)]
        assert sizes == sorted(sizes)


def test_e4m3_table():
    v = Q.E4M3
    assert v[:17].tolist() == [i * 2.0 ** -9 for i in range(16)] + [2.0 ** -5]
    assert v[0x38] == 1 and v[0x7E] == 448 and (np.diff(v) > 0).all()
    assert Q.e4m3_byte([0.0, 1.0, 1.0625, 1.1875, 1.07, 448, 2.0 ** -10, 3 * 2.0 ** -10], False).tolist() == [
        0, 0x38, 0x38, 0x3A, 0x39, 0x7E, 0, 2]
    assert Q.e4m3_byte([0.0, 1.0, 1.0001, 448, 1e-9], True).tolist() == [0, 0x38, 0x39, 0x7E, 1]


@pytest.mark.parametrize("zero", [0, 1])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_weight_is_exact_in_bf16_and_near_what_it_stands_for(group, zero):
    r = np.random.default_rng(group + zero)
    x = (r.normal(size=(40, 416)) * np.exp(r.normal(size=(40, 1)) * 20)).astype(np.float32)
    x[3] = 0
    x[4] = np.abs(x[4])
    x[5, 7] = x[5].max() * 1e4
    c, w, e = Q.quantize(x, group, zero)
    v = Q.weights(c, w, e, group)
    assert (v.astype(np.float32) == v).all()
    assert ((v.astype(np.float32).view(np.uint32) & 0xFFFF) == 0).all()
    s, _ = Q.scales(w, e, group, 416)
    # half a step; at the ends of the range half a step more with zero points (z is rounded), and
    # where s is 0 the group is below half the least step
    assert (np.abs(v - x) <= np.where(s > 0, s * (1.0 if zero else 0.5), np.abs(x)) * (1 + 2.0 ** -40)).all()
    assert (Q.unpack(Q.pack(c)) == c).all()
    assert (Q.unlay_words(Q.lay_words(w), *w.shape) == w).all()


def test_words_lie_by_runs_of_16_rows():
    w = np.arange(37 * 3).reshape(37, 3)
    flat = Q.lay_words(w)
    assert flat[:3].tolist() == [0, 3, 6] and flat[16] == 1 and flat[48] == w[16, 0] and flat[96:101].tolist() == w[32:, 0].tolist()
    assert flat[101] == w[32, 1] and flat[-1] == w[36, 2]
