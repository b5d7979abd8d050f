"""No kernel of the dense operators goes untested: the kernels that the GPU tests' sizes take, by the
library's own rules, are all that are compiled and all that sizes over the whole range take."""
import random
import re
import shutil
import subprocess

import pytest

import test_gpu_dense as G
import test_gpu_dense_kernels as K

B = pytest.importorskip("expert_cached_moe_amd.binding")

F32, BF16, I8 = 0, 1, 2
SIZE = {F32: 4, BF16: 2, I8: 1}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Lists of calls to the sets of kernels that they take."""
    if not shutil.which("g++"):
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("list") / "list_dense_kernels")
    src = __file__.replace("test_dense_coverage_cpu.py", "list_dense_kernels.cpp")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", src, "-o", exe], check=True)

    def run(calls):
        out = subprocess.run([exe], input="\n".join(calls) + "\n", capture_output=True, text=True, check=True).stdout
        assert out.count("\n") == len(calls)
        return {k for k in out.replace("\n", "").split(";") if k}
    return run


def product(T, N, K, x, y, pad=0, off=0):
    ld = K + pad
    whole = x != I8 and ld * SIZE[x] % 16 == 0 and off * SIZE[x] % 16 == 0
    return f"m {x} {ld} {int(whole)} {T} {N} {K} {y}"


def sizes(test):
    """The sizes a test of the first file is written for."""
    return next(m.args[1] for m in test.pytestmark if m.name == "parametrize" and "," in m.args[0])


def all_tested():
    calls = []
    for s in G.SHAPES:
        calls += [product(*s, BF16, BF16), product(*s, F32, F32, 3), product(*s, I8, F32), product(*s, BF16, F32, 16)]
    for s in K.FEW_PRODUCTS + K.TILE_PRODUCTS:
        calls += [product(*s, x, y) for x, y in ((BF16, BF16), (F32, F32), (I8, BF16), (BF16, F32), (F32, BF16))]
    calls += [product(T, N, k, BF16, y) for T, N, k, y in sizes(G.test_i8_matmul_large)]
    for rows, cols in K.ROWS:
        calls += [f"q {x} {int(off == 0)} {rows} {cols}" for x in (F32, BF16) for off in (0, 1)]
    for w in (F32, BF16):
        calls += [f"{p} {w} {T} {H} {I}" for T, H, I in G.BLOCKS + K.TILE_BLOCKS[w] for p in "fb"]
        calls += [f"f {w} {T} {H} {I}" for T, H, I in K.FEW_BLOCKS[w]]
    calls += [f"{p} {BF16} {T} {H} {I}" for T, H, I in sizes(G.test_block_large) for p in "fb"]
    calls += [f"8 {T} {H} {I}" for T, H, I in sizes(G.test_i8_block) + K.BLOCKS8]
    return calls + ["8 4100 2112 4128"]                    # (test_i8_block_large)


def test_every_compiled_kernel_is_tested(kernels):
    out = subprocess.run(["nm", "-C", B.LIB_PATH], capture_output=True, text=True).stdout
    compiled = set()
    for name in re.findall(r"__device_stub__(k_(?:few|mma|join|quantize)\w*<.*>)\(", out):
        compiled.add(re.sub(r"moe::dense::|\(anonymous namespace\)::", "", name))
    assert len(compiled) > 100
    have = {k.replace(" split", "") for k in kernels(all_tested())}
    assert have == compiled, (sorted(compiled - have), sorted(have - compiled))


def test_every_choice_in_the_range_is_tested(kernels):
    """20,000 calls of each kind, sizes spread over the logarithm; K split and whole apart."""
    r = random.Random(11)

    def some(lo, hi, step=1):
        return max(step, min(hi // step * step, round(lo * (hi / lo) ** r.random() / step) * step))

    calls = []
    for _ in range(20000):
        x = r.choice((F32, BF16, I8))
        calls.append(product(some(1, 8192), some(1, 100003), some(16, 16384, 16), x, r.choice((F32, BF16)),
                             0 if x == I8 else r.choice((0, 3))))
        T, H, I = some(1, 8192), some(64, 32768, 64), some(32, 16384, 32)
        calls += [f"8 {T} {H} {I}"] + [f"{p} {r.choice((F32, BF16))} {T} {H} {I}" for p in "fb"]
        calls.append(f"q {r.choice((F32, BF16))} {r.choice((0, 1))} {some(1, 100000)} {some(16, 65536, 16)}")
    have = kernels(all_tested())
    missing = kernels(calls) - have
    assert not missing, sorted(missing)
