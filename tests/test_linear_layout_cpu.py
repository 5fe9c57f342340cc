"""The dense projection's addresses and tiles on the host.

csrc/linear_layout.h holds the arithmetic that places the kernels' loads and chooses their tiles; a small host library
(g++) includes it.  It checks, load by load, that what lies inside a stage's buffer resource is the 16 bytes that belong
at that place of the tile, inside the operand, and that rows and reduction indices that do not exist lie outside; and it
tells which tiles a size runs in, so that the sizes that the GPU tests pick for their tiles keep them.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

from linear_tile_cases import CASES

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host", "linear_layout_check.cpp")
CXX = shutil.which("g++") or shutil.which("clang++")

pytestmark = pytest.mark.skipif(CXX is None, reason="no host C++ compiler")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    out = tmp_path_factory.mktemp("host") / "linear_layout_check.so"
    r = subprocess.run([CXX, "-O2", "-std=c++17", "-shared", "-fPIC", SRC, "-o", str(out)], stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    lib = ctypes.CDLL(str(out))
    i64 = ctypes.c_int64
    lib.forward_wrong.argtypes, lib.forward_wrong.restype = [i64] * 3, i64
    lib.backward_wrong.argtypes, lib.backward_wrong.restype = [i64] * 3 + [ctypes.c_int], i64
    lib.forward_tiles.argtypes = [i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    return lib


EDGES = [1, 17, 63, 64, 65, 130, 255, 256, 300]


@pytest.mark.parametrize("K", [8, 16, 24, 32, 40, 48, 56, 64, 72, 120, 128, 200])
def test_forward_loads_stay_inside_their_operands(host, K):
    for n in EDGES:
        assert host.forward_wrong(n, n, K) == 0, (n, K)


@pytest.mark.parametrize("K", [8, 32, 56, 64, 72, 136, 264])
@pytest.mark.parametrize("mats", [1, 2])
def test_backward_loads_stay_inside_their_operands(host, K, mats):
    for M, N in [(1, 1), (17, 33), (63, 65), (64, 64), (65, 130), (130, 63), (257, 200), (300, 257)]:
        assert host.backward_wrong(M, N, K, mats) == 0, (M, N, K, mats)


@pytest.mark.parametrize("M,N,K,kind,slices,streamed", CASES)
def test_tiles_of_the_sizes_that_the_gpu_tests_run(host, M, N, K, kind, slices, streamed):
    out = (ctypes.c_int * 3)()
    host.forward_tiles(M, N, K, 0, out)
    assert tuple(out) == (kind, slices, streamed)
