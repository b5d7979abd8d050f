"""No kernel of the products with 4-bit weights goes untested: the GPU tests' sizes take every kind of tiles that is
compiled, by the library's own rules, and each is what sizes over the range take."""
import os
import random
import re
import shutil
import subprocess

import pytest

import test_gpu_i4 as G

B = pytest.importorskip("expert_cached_moe_amd.binding")

KINDS = set(range(9))


@pytest.fixture(scope="module")
def kinds(tmp_path_factory):
    """Calls to the kinds of tiles that they take, one each."""
    if not shutil.which("g++"):
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("list") / "list_i4_kernels")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "list_i4_kernels.cpp")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", src, "-o", exe], check=True)

    def run(calls):
        out = subprocess.run([exe], input="\n".join(calls) + "\n", capture_output=True, text=True, check=True).stdout.split()
        assert len(out) == len(calls)
        return {int(k) for k in out}
    return run


def experts(shapes):
    """The gate and up, and the down products."""
    gate, down = [], []
    for H, I, E, k, shared, T in shapes:
        rows = T * (k + shared)
        gate.append(f"e {E + shared} {rows} {2 * I} {H}")
        down.append(f"e {E + shared} {rows} {H} {I}")
    return gate, down


def test_every_kind_is_tested(kinds):
    dense = G.SHAPES + G.TILES
    for planes in (1, 3):
        assert kinds([f"m {T} {N} {K} {planes}" for T, N, K in dense]) == KINDS | {-1}
    shapes = [s[:5] + (T,) for s in G.LAYERS for T in G.TOKENS if T > 8] + [s[:5] + s[6:] for s in G.LARGE]
    for calls in experts(shapes):
        assert kinds(calls) == KINDS


def test_every_kind_is_taken_over_the_range(kinds):
    r = random.Random(3)

    def some(lo, hi, step=1):
        return max(step, min(hi // step * step, round(lo * (hi / lo) ** r.random() / step) * step))

    for planes in (1, 3):
        assert kinds([f"m {some(9, 8192)} {some(1, 100003)} {some(32, 12288, 32)} {planes}" for _ in range(20000)]) == KINDS | {-1}
    shapes = [(some(64, 8192, 64), some(32, 8192, 32), some(1, 256), r.randint(1, 8), r.randint(0, 1), some(9, 8192))
              for _ in range(20000)]
    for calls in experts(shapes):
        assert kinds(calls) == KINDS


def test_launches_fit(kinds):
    """The threads of a launch stay within 31 bits up to the largest products (tiles of up to 512 threads)."""
    rows, cols = (32, 64, 128, 64, 128, 32, 64, 128, 256), (32, 32, 32, 64, 64, 128, 128, 128, 256)

    def blocks(k, tiles, N):
        return tiles(rows[k]) * -(-N // cols[k])

    for a in range(13, 24):
        for K in (32, 4096):
            T, N = 1 << a, 1 << min(23, 36 - a)
            (k,) = kinds([f"m {T} {N} {K} 1"])
            assert blocks(k, lambda r: -(-T // r), N) * 512 < 2 ** 31
            (k,) = kinds([f"e 512 {T * 16} {N >> 4} {K}"])
            assert blocks(k, lambda r: T * 16 // r + 512, N >> 4) * 512 < 2 ** 31


def test_compiled_kernels():
    """Nine kinds, the few-row kernel by tokens (dense) and parts of x (dense), for four products."""
    out = subprocess.run(["nm", "-C", B.LIB_PATH], capture_output=True, text=True).stdout
    have = set(re.findall(r"__device_stub__(k_i4_(?:few|mid|wide|turns)<\d+)", out))
    count = len(set(re.findall(r"__device_stub__(k_i4_(?:few|mid|wide|turns)<[^>]*>)", out)))
    assert have == {f"k_i4_{k}<{what}" for k in ("few", "mid", "wide", "turns") for what in range(4)}
    assert count == len(KINDS) * 4 + 2 * 2 * 2 + 2
