"""The 64-bit form of the router's gates and gradient against 60-digit numbers, where scores are near the end of
64-bit numbers or far below the row's largest."""
import decimal

import numpy as np
import pytest

from oracle import scored_oracle as S

D = decimal.Decimal
LEAST = 2.0 ** -1074                     # the least 64-bit number


def exactly(logits, ids, dw, kind, scale):
    """(gates, dlogits) of one row with renormalised gates."""
    with decimal.localcontext(decimal.Context(prec=60)):
        z = [D(float(v)) for v in logits]
        if kind == "sigmoid":
            p = [1 / (1 + (-z[e]).exp()) for e in ids]
        else:
            p = [(z[e] - max(z)).exp() for e in ids]
        a = [v / sum(p) for v in p]
        d = [D(scale) * D(float(v)) for v in dw]
        mean = sum(x * y for x, y in zip(d, a))
        out = np.zeros(len(logits))
        for e, x, y, v in zip(ids, d, a, p):
            out[e] = float((x - mean) * y * (1 - v if kind == "sigmoid" else 1))
        return np.array([float(D(scale) * v) for v in a]), out


ROWS = [[-720, -721, -722, -1000, -1000, -1000], [-733.5, -735, -734.25, -735.5, -736, -900], [-709, -712, -744, -709.5, -800, -745],
        [3, 2.5, -720, 1, 0, -3], [40, 36.5, 33, 30, 1, 0]]
LOW = [[-800, -801, -802, 0, -900, -900], [-2e5, -200000.5, -199999.25, 12, 11, -3e5], [-746, -747, -745.5, 0, 0, 0], [1, 2, 3, 4, 0, -1]]


@pytest.mark.parametrize("kind,rows", [("sigmoid", ROWS), ("softmax", LOW + ROWS)])
def test_gates_and_gradient_against_many_digits(kind, rows):
    k, scale = 3, 2.5
    rng = np.random.default_rng(3)
    for row in rows:
        logits, ids = np.float32([row]), np.arange(k)[None]
        dw = rng.normal(size=(1, k)).astype(np.float32)
        gates, d = exactly(logits[0], ids[0], dw[0], kind, scale)
        total = np.take_along_axis(S.scores(logits, kind), ids, 1).sum()
        # a score is off by the least number at most, a share by (k + 1) of them over the sum; 40 operations of 2^-53
        off = ((k + 1) * LEAST / total if kind == "sigmoid" else 0.0) + 40 * 2.0 ** -53
        assert np.abs(S.gates_of(logits, ids, kind, 1, scale)[0] - gates).max() <= scale * off
        got = S.backward(logits, ids, dw, kind, 1, scale)[0]
        assert np.isfinite(got).all()
        assert np.abs(got - d).max() <= 2 * scale * np.abs(dw).sum() * off


def test_rows_of_scores_that_are_0():
    """Sums of 0 in 64 bits, or nothing but masked logits: gates and gradient are 0."""
    logits = np.float32([[-1000, -1001, -1002, -2000], [-np.inf] * 4])
    ids, dw = np.tile([[0, 1, 2]], (2, 1)), np.ones((2, 3))
    for kind, rows in (("sigmoid", (0, 1)), ("softmax", (1,))):
        for t in rows:
            assert (S.gates_of(logits, ids, kind, 1, 2.0)[t] == 0).all() and (S.backward(logits, ids, dw, kind, 1, 2.0)[t] == 0).all()
