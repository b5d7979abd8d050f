"""The router by scores without a GPU: refusals, and the 64-bit form against brute force and differences."""
import itertools

import numpy as np
import pytest

from oracle import scored_oracle as S

B = pytest.importorskip("expert_cached_moe_amd.binding")

FAKE = 0x1000           # an address that a refused call does not touch


@pytest.fixture
def ctx():
    c = B.moe_create(B.make_config(64, 32, 24, 4))
    yield c
    B.moe_destroy(c)


def forward(ctx, T=3, rule=None, **at):
    a = dict(logits=FAKE, bias=None, ids=FAKE, w=FAKE, counts=FAKE, offsets=FAKE, perm=FAKE, inv=FAKE, ws=FAKE)
    a.update(at)
    B.moe_route_scored(ctx, a["logits"], a["bias"], T, rule, a["ids"], a["w"], a["counts"], a["offsets"], a["perm"],
                       a["inv"], a["ws"])


def backward(ctx, T=3, rule=None, **at):
    a = dict(logits=FAKE, ids=FAKE, dw=FAKE, dlogits=FAKE)
    a.update(at)
    B.moe_route_scored_backward(ctx, a["logits"], T, rule, a["ids"], a["dw"], a["dlogits"])


BAD_RULES = [None, dict(score=2), dict(score=-1), dict(n_groups=0), dict(n_groups=5), dict(n_groups=65),
             dict(n_groups=4, keep_groups=0), dict(n_groups=4, keep_groups=5), dict(n_groups=12, keep_groups=1),
             dict(group_top=0), dict(group_top=3), dict(renormalize=2), dict(scale=float("nan")),
             dict(scale=float("inf"))]


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("rule", BAD_RULES)
def test_rules_outside_their_bounds_are_refused(ctx, call, rule):
    with pytest.raises(B.MoeError) as e:
        call(ctx, rule=B.make_route_rule(**rule) if rule is not None else None)
    assert e.value.status == B.MOE_EINVAL


@pytest.mark.parametrize("call", [forward, backward])
def test_counts_are_refused(ctx, call):
    r = B.make_route_rule()
    for T, status in ((-1, B.MOE_EINVAL), ((1 << 24) + 1, B.MOE_ESHAPE)):
        with pytest.raises(B.MoeError) as e:
            call(ctx, T=T, rule=r)
        assert e.value.status == status


@pytest.mark.parametrize("call,names", [(forward, ("logits", "ids", "w", "counts", "offsets", "perm", "inv")),
                                        (backward, ("logits", "ids", "dw", "dlogits"))])
def test_null_buffers_are_refused(ctx, call, names):
    for n in names:
        with pytest.raises(B.MoeError) as e:
            call(ctx, rule=B.make_route_rule(), **{n: None})
        assert e.value.status == B.MOE_EINVAL
    if call is forward:
        with pytest.raises(B.MoeError) as e:
            forward(ctx, T=129, rule=B.make_route_rule(), ws=None)
        assert e.value.status == B.MOE_EINVAL


def test_backward_of_no_tokens_does_nothing(ctx):
    backward(ctx, T=0, rule=B.make_route_rule(), logits=None, ids=None, dw=None, dlogits=None)


def test_choice_against_every_subset():
    """Of all subsets of k experts inside the kept groups the choice has the largest values."""
    r = np.random.default_rng(5)
    for kind, biased, groups, keep, top in itertools.product(("softmax", "sigmoid"), (0, 1), (1, 3), (1, 2), (1, 2)):
        if keep > groups:
            continue
        E, k = 9, 3
        logits, bias = r.normal(size=(20, E)), r.normal(size=E) * 0.3 if biased else None
        s, ids = S.choose(logits, bias, k, kind, groups, keep, top)
        c = s if bias is None else s + bias
        for t in range(20):
            best = None
            for kept in itertools.combinations(range(groups), keep):
                worth = sorted((sum(sorted(c[t, 9 // groups * g:9 // groups * (g + 1)])[-top:]) for g in kept))
                if best is None or sum(worth) > best[0]:
                    best = (sum(worth), kept)
            allowed = [e for e in range(E) if groups == 1 or e // (E // groups) in best[1]]
            top_sets = max(itertools.combinations(allowed, k), key=lambda q: sum(c[t, list(q)]))
            assert set(ids[t].tolist()) == set(top_sets)
            assert all(np.diff(c[t, ids[t]]) <= 0)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gradient_against_differences(kind, renorm):
    r = np.random.default_rng(7)
    logits, dw = r.normal(size=(4, 11)) * 2, r.normal(size=(4, 3))
    _, ids = S.choose(logits, None, 3, kind)
    d = S.backward(logits, ids, dw, kind, renorm, 1.7)

    def loss(x):
        return (S.gates(S.scores(x, kind), ids, renorm, 1.7) * dw).sum(1)

    h = 1e-5
    for e in range(11):
        step = np.zeros_like(logits)
        step[:, e] = h
        # central differences of a smooth function of size 1: h^2 and 2^-53 / h
        assert np.abs((loss(logits + step) - loss(logits - step)) / (2 * h) - d[:, e]).max() < 1e-9
