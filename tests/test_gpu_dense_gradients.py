"""Gradients of the dense block against differences of the loss sum(y dy), along the gradient itself
on random halves of its entries: there the loss moves so far that the worst case of every rounding
is a few hundredths of the movement, so a wrong gradient cannot pass.  (test_dense_gradients_cpu.py
plants mistakes.)
"""
import numpy as np
import pytest
import torch

from oracle import dense_oracle as D
from test_gpu_dense import BF16, F32, NAME, TORCH, Ctx, _blob, _block_inputs, _views, f64
from test_gpu_dense import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

KEYS = ["dx", "dwg", "dwu", "dwd"]
# y is linear in Wu and Wd; along the others the steps leave a third-order term below the roundings
STEP = {"dx": 2.0 ** -3, "dwg": 2.0 ** -6, "dwu": 2.0 ** -3, "dwd": 2.0 ** -3}
SIZES = [(20, 128, 64), (130, 128, 160)]
FORCE = {F32: 0.05, BF16: 0.1}


def directions(dy, args, rng):
    """(which argument, direction of root mean square near 1): random halves of the gradient."""
    for k, g in enumerate(D.block_backward(dy, *args)):
        for _ in range(2):
            yield k, g / np.sqrt((g ** 2).mean()) * (rng.random(g.shape) < 0.5)


def moved(args, k, step, d):
    """The arguments with the k-th moved along d, as fp32 holds it."""
    out = list(args)
    out[k] = (args[k] + step * d).astype(np.float32).astype(np.float64)
    return out


def formula_slope(dy, args, k, d):
    """(difference quotient of the formulas' loss in 64 bits, its own distance from the derivative)."""
    step = STEP[KEYS[k]]
    up, dn = ((D.block(*moved(args, k, s, d))[0] * dy).sum() for s in (step, -step))
    slope = (up - dn) / (2 * step)
    return slope, abs(slope - (D.block_backward(dy, *args)[k] * d).sum())


def check_slope(grad, dy, args, k, d, bounds, force, slope=None, slope_error=0.0):
    """grad's slope along d against a difference quotient (the formulas' unless given)."""
    formula, third = formula_slope(dy, args, k, d)
    slope = formula if slope is None else slope
    tol = third + (bounds[KEYS[k]] * np.abs(d)).sum() + slope_error
    assert tol <= force * abs(slope), "the test says nothing"
    assert abs((grad * d).sum() - slope) <= tol, (KEYS[k], (grad * d).sum(), slope, tol)


@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("w", [F32, BF16])
def test_block_gradients_follow_the_loss(B, w, T, H, I):
    """Both types against the formulas' loss, fp32 against the library's own as well."""
    rng = np.random.default_rng(T + I)
    x, dy, wg, wu, wd = _block_inputs(rng, T, H, I, w)
    args, dy64 = [f64(t) for t in (x, wg, wu, wd)], f64(dy)
    bounds = D.block_bounds(dy64, *args, NAME[w])
    with Ctx(B, H, I, w) as c:
        work = torch.empty(B.moe_dense_workspace_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
        save = torch.empty(B.moe_dense_save_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
        blob = _blob(B, c, wg, wu, wd)
        y, dx, grad = torch.empty_like(x), torch.empty_like(x), torch.empty_like(blob)
        B.moe_dense_ffn(c.p, x, T, blob, save, y, work)
        B.moe_dense_ffn_backward(c.p, dy, x, T, blob, save, dx, grad, work)
        torch.cuda.synchronize()
        gu, dd = _views(grad, H, I, TORCH[w])
        got = [f64(dx), *D.deinterleave(f64(gu)), f64(dd)]

        def loss(a):
            t = [torch.from_numpy(m.astype(np.float32)).cuda() for m in a]
            B.moe_dense_ffn(c.p, t[0], T, _blob(B, c, *t[1:]), None, y, work)
            torch.cuda.synchronize()
            return (f64(y) * dy64).sum()

        for k, d in directions(dy64, args, rng):
            check_slope(got[k], dy64, args, k, d, bounds, FORCE[w])
            if w == F32:
                step = STEP[KEYS[k]]
                ends = [moved(args, k, s, d) for s in (step, -step)]
                slope = (loss(ends[0]) - loss(ends[1])) / (2 * step)
                noise = sum((D.block_bounds(None, *e, "f32")["y"] * np.abs(dy64)).sum() for e in ends) / (2 * step)
                check_slope(got[k], dy64, args, k, d, bounds, FORCE[w], slope, noise)
