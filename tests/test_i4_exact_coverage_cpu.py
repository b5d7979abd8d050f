"""The exact tests of the products with 4-bit weights run on the kinds of tiles that they are meant for."""
import pytest

import test_gpu_i4_exact as G
from test_i4_coverage_cpu import KINDS, kinds  # noqa: F401


def test_fp32_rows_take_every_kind(kinds):  # noqa: F811
    assert kinds([f"m {T} {N} {K} 3" for T, N, K in G.TILES_F32]) == KINDS


@pytest.mark.parametrize("shape,kind", list(zip(G.FAR, (2, 4, 7, 6))))
def test_far_rows_take_the_tiles_with_32_bit_offsets(kinds, shape, kind):  # noqa: F811
    T, N, K = shape
    assert kinds([f"m {T} {N} {K} 1"]) == {kind}


def test_far_experts_gather_by_32_bit_offsets(kinds):  # noqa: F811
    for H, I, E, k, shared, _, T in G.FAR_EXPERTS:
        assert kinds([f"e {E + shared} {T * (k + shared)} {2 * I} {H}"]) <= KINDS - {8}
        assert 0xFFFF0000 - 2 * 16 * H < T * H * 2 <= 0xFFFF0000
