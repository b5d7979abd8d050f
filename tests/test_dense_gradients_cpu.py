"""The comparison of the dense block's gradients with differences accepts the formulas' gradient and
refuses mistakes planted in it."""
import numpy as np
import pytest

from oracle import dense_oracle as D
from test_gpu_dense_gradients import BF16, F32, FORCE, KEYS, NAME, SIZES, check_slope, directions


def _inputs(T, H, I):
    rng = np.random.default_rng(T + I)

    def n(shape, scale):
        return (rng.standard_normal(shape) * scale).astype(np.float32).astype(np.float64)
    s = H ** -0.5
    return rng, n((T, H), 0.1), [n((T, H), 1), n((I, H), 2 * s), n((I, H), s), n((H, I), I ** -0.5)]


def _wrong(dy, x, wg, wu, wd):
    """Gradients with one mistake each, for the arguments they spoil."""
    _, (g, u, a, h) = D.block(x, wg, wu, wd)
    s, dh = D.sigmoid(g), dy @ wd
    right = D.block_backward(dy, x, wg, wu, wd)
    for f in (0.0, 0.5, -1.0, 1.25):
        yield {k: f * right[k] for k in range(4)}
    dg, du = dh * u * s, dh * a                            # silu' without its second term
    yield {0: dg @ wg + du @ wu, 1: dg.T @ x}
    dg = dh * u * (s + g * s)                              # ... without 1 - s
    yield {0: dg @ wg + du @ wu, 1: dg.T @ x}
    dg, du = dh * u * (s + g * s * (1 - s)), dh * g        # du without the sigmoid
    yield {0: dg @ wg + du @ wu, 2: du.T @ x}
    yield {1: right[2], 2: right[1], 3: dy.T @ (g * u)}    # gate and up swapped; h without it
    yield {0: dg @ wg}                                     # up's part of dx left out


@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("w", [F32, BF16])
def test_differences_refuse_mistakes(w, T, H, I):
    rng, dy, args = _inputs(T, H, I)
    bounds = D.block_bounds(dy, *args, NAME[w])
    right, wrong = D.block_backward(dy, *args), list(_wrong(dy, *args))
    for k, d in directions(dy, args, rng):
        check_slope(right[k], dy, args, k, d, bounds, FORCE[w])
        for i, m in enumerate(wrong):
            if k in m:
                with pytest.raises(AssertionError) as e:
                    check_slope(m[k], dy, args, k, d, bounds, FORCE[w])
                assert KEYS[k] in str(e.value), (i, str(e.value))
