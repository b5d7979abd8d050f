"""Products with 4-bit weights whose results are exact: numbers near the ends of fp32."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
B = pytest.importorskip("expert_cached_moe_amd.binding")
from oracle import i4_oracle as Q  # noqa: E402
from test_gpu_i4 import BF16, F32, TORCH, Weights, ctx, product  # noqa: E402, F401

pytestmark = pytest.mark.gpu


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
