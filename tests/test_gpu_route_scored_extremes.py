"""The router by scores and its gradient where scores leave the ordinary range: sigmoids near the end of
64-bit numbers, chosen logits far below the row's largest, scores that 64 bits do not tell apart."""
import decimal

import numpy as np
import pytest

torch = pytest.importorskip("torch")
B = pytest.importorskip("expert_cached_moe_amd.binding")
from oracle import scored_oracle as S  # noqa: E402
from test_gpu_route_scored import Router, cuda  # noqa: E402

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -1074                     # the least 64-bit number


@pytest.mark.parametrize("T", [6, 40, 2105])
def test_gradient_of_renormalised_sigmoids_near_the_end_of_64_bits(T):
    """Chosen logits between -735 and -700: their scores and the sum are as small as 1e-320, the gradient is not."""
    E, k = 12, 4
    rng = np.random.default_rng(T)
    logits = np.full((T, E), -np.inf, np.float32)
    for t in range(T):
        logits[t, rng.permutation(E)[:k + 2]] = rng.uniform(-735, -700) + rng.uniform(-3, 3, k + 2)
    logits[0, :4], logits[0, 4:] = [-720, -721, -722, -800], -np.inf
    dw = rng.normal(size=(T, k)).astype(np.float32)
    r = Router(E, k, T, "sigmoid", renorm=1, scale=2.5)
    dl = cuda(logits)
    r.forward(dl, None)
    r.backward(dl, cuda(dw))
    ids, w = r.results()
    d = r.d[:T * E].cpu().numpy().reshape(T, E)
    s, ref = S.choose(logits, None, k, "sigmoid")
    assert np.array_equal(ids, ref)
    # a score is off by the least number at most, here and in the oracle, so a share by (k + 1) of them over the sum, and
    # the gradient by that for its own share and for each term of its sum
    total = np.take_along_axis(s, ids, 1).sum(1, keepdims=True)
    off = 2 * (k + 1) * LEAST / total
    gates = S.gates_of(logits, ids, "sigmoid", 1, 2.5)
    assert (np.abs(w - gates) <= np.abs(gates) * 2.0 ** -23 + 2.5 * off).all()
    want = S.backward(logits, ids, dw, "sigmoid", 1, 2.5)
    size = 2.5 * np.abs(dw).sum(1, keepdims=True)
    assert np.isfinite(d).all()
    assert (np.abs(d - want) <= np.abs(want) * 2.0 ** -24 + size * (2.0 ** -46 + 2 * off) + 2.0 ** -149).all()


@pytest.mark.parametrize("T", [6, 40, 2106])
@pytest.mark.parametrize("how", ["bias", "groups"])
def test_chosen_logits_far_below_the_largest(T, how):
    """The largest logit is not chosen, by its bias or by its group, and the chosen ones lie up to 90,000 below it:
    renormalised, they share the gates among themselves, and the gradient is that of these gates."""
    E, k = 24, 4
    rng = np.random.default_rng(T)
    low = -np.exp(rng.uniform(np.log(600), np.log(90000), (T, 1)))
    logits = (low + rng.normal(size=(T, E)) * 2).astype(np.float32)
    logits[0, :5] = [0, -800, -801, -802, -803]
    logits[0, 5:] = -900
    bias = np.zeros(E, np.float32)
    if how == "bias":
        logits[:, 0] = 0
        bias[0] = -np.inf
        groups, keep = 1, 1
    else:
        # (the first group's best is the row's largest; the others win by their bias)
        logits[:, 0] = 0
        logits[:, 1:6] = -np.inf
        bias[6:] = 2.0
        groups, keep = 4, 3
    bias[1:] += rng.permutation(E - 1).astype(np.float32) * np.float32(2.0 ** -10)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    r = Router(E, k, T, "softmax", groups, keep, 1, 1, 2.5)
    dl = cuda(logits)
    r.forward(dl, cuda(bias))
    r.backward(dl, cuda(dw))
    ids, w = r.results()
    _, ref = S.choose(logits, bias, k, "softmax", groups, keep, 1)
    assert np.array_equal(ids, ref) and (ids != 0).all()
    gates = S.gates_of(logits, ids, "softmax", 1, 2.5)
    assert (np.abs(gates.sum(1) - 2.5) < 1e-12).all()
    assert (np.abs(w - gates) <= np.abs(gates) * (2.0 ** -24 + 2.0 ** -46) + 2.0 ** -149).all()
    r.check_gradient(logits, ids, dw)


def sigmoid_exactly(z):
    with decimal.localcontext(decimal.Context(prec=60)):
        return 1 / (1 + (-decimal.Decimal(float(z))).exp())


@pytest.mark.parametrize("T", [6, 40, 2107])
def test_scores_that_64_bits_do_not_tell_apart(T):
    """Sigmoids of 30 to 45: above 53 ln 2 = 36.74 they are 1 (e^-z < 2^-53, half a step of 1 + e^-z, which rounds to 1) and
    the lower id comes first; below, the order is that of the exact scores but where these are as close as the 64-bit
    ones' errors: 2^-53 from 1 + e^-z, 2^-53 from its reciprocal."""
    E, k = 32, 12
    rng = np.random.default_rng(T)
    logits = rng.uniform(30, 45, (T, E)).astype(np.float32)
    logits[T // 2:] = rng.uniform(30, 37.5, (T - T // 2, E)).astype(np.float32)
    r = Router(E, k, T, "sigmoid", renorm=0)
    r.forward(cuda(logits), cuda(np.zeros(E, np.float32)))
    ids, _ = r.results()
    near = decimal.Decimal(2) ** -51
    for t in range(0, T, max(1, T // 40)):
        full = [e for e in range(E) if logits[t, e] > 53 * np.log(2)]
        n = min(len(full), k)
        assert ids[t, :n].tolist() == full[:n]
        assert len(set(ids[t].tolist())) == k
        s = [sigmoid_exactly(z) for z in logits[t]]
        left = set(range(E))
        for j in range(k):
            left.discard(int(ids[t, j]))
            assert all(s[e] <= s[ids[t, j]] + near for e in left)
