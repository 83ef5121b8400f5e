"""The wait for copies in flight that a kernel makes after one of its waits has run out: every item of the ring that was
issued, for any number of them, and no longer than its limit where one never completes."""

import ctypes
import os
import subprocess

import pytest

from nvfp4_block_scaled_mm_b200 import build as B

pytestmark = pytest.mark.gpu

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "native", "ring_drain.cu")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    try:
        nvcc = B._nvcc()
    except RuntimeError:
        pytest.skip("nvcc not found: this test compiles its kernel")
    so = str(tmp_path_factory.mktemp("ring") / "ring_drain.so")
    subprocess.run([nvcc, *B.ARCH_FLAGS, "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", B.CSRC, "-o", so, SRC],
                   check=True)
    lib = ctypes.CDLL(so)
    lib.ring_drain.argtypes = [ctypes.c_uint32] * 3 + [ctypes.c_uint64] * 2 + [ctypes.POINTER(ctypes.c_uint32)]
    return lib


@pytest.mark.parametrize("stages", [1, 6, 8])
@pytest.mark.parametrize("n", [0, 1, 3, 6, 7, 8, 12, 13, 21, 64])
def test_waits_for_every_item_in_flight(lib, stages, n):
    out = (ctypes.c_uint32 * 2)()
    assert lib.ring_drain(stages, n, n, 20_000, 50_000_000, out) == 0
    assert out[0] == min(stages, n)
    assert out[1] < 50_000


@pytest.mark.parametrize("stages,n,missing", [(6, 3, 0), (6, 13, 12), (8, 8, 5), (1, 4, 3)])
def test_gives_up_at_its_limit(lib, stages, n, missing):
    out = (ctypes.c_uint32 * 2)()
    assert lib.ring_drain(stages, n, missing, 1_000, 4_000_000, out) == 0
    assert out[0] == min(stages, n) - 1
    assert 4_000 <= out[1] < 50_000
