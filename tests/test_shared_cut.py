"""Which blocks hold the partial results of a unit behind a shared prefix: the kernels' own function, compiled for the
host, against the runs that it inverts; and launches in which nothing is shared, where there is no run at all."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from exact_attention_91_gb300 import build as fa_build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    nvcc = fa_build.nvcc_path()
    if not (os.path.exists(nvcc) or shutil.which(nvcc)):
        pytest.skip("nvcc not available")
    out = str(tmp_path_factory.mktemp("cut") / "libcut.so")
    subprocess.run([nvcc, fa_build.ARCH, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-shared",
                    "-I", fa_build.INCLUDE, "-I", fa_build.CSRC, os.path.join(HERE, "helpers", "shared_cut.cu"), "-o", out],
                   check=True)
    lib = ctypes.CDLL(out)
    ll, i, at = ctypes.c_longlong, ctypes.c_int, ctypes.POINTER(ctypes.c_int)
    lib.cut.argtypes, lib.cut.restype = [ll, i, ll, i, at, at], None
    lib.start.argtypes, lib.start.restype = [ll, i, i], ll

    def cut(total, workers, begin, tiles):
        first, last = ctypes.c_int(-9), ctypes.c_int(-9)
        lib.cut(total, workers, begin, tiles, first, last)
        return first.value, last.value

    return lib.start, cut


@pytest.mark.parametrize("workers", [0, 1, 152])
@pytest.mark.parametrize("tiles", [0, 1, 5])
def test_nothing_is_shared(lib, workers, tiles):
    """(x86 raises a signal at a division by zero; nothing may be divided here.)"""
    start, cut = lib
    assert cut(0, workers, 0, tiles) == (0, 0)
    assert cut(0, workers, 1 << 40, tiles) == (0, 0)


@pytest.mark.parametrize("lo,hi", [(1, 2000), (1 << 19, 1 << 21), (1 << 33, 1 << 40)])
def test_the_cut_inverts_the_runs(lib, lo, hi):
    start, cut = lib
    r = random.Random(lo)
    for _ in range(400):
        total, most = r.randint(lo, hi), r.choice([1, 2, 7, 152, 304])
        workers = min(most, (total + 1) // 2)
        begin = r.randrange(total)
        tiles = r.randint(1, min(total - begin, (1 << 24) - 1))
        c0, c1 = cut(total, workers, begin, tiles)
        assert 0 <= c0 <= c1 < workers
        assert start(total, workers, c0) <= begin < start(total, workers, c0 + 1)
        assert start(total, workers, c1) <= begin + tiles - 1 < start(total, workers, c1 + 1)
