"""The workspace of kv_fork and kv_compact (csrc/page_work.cuh), on the CPU: what has
to be zero between two calls is never where another call, with another number of
blocks, leaves numbers."""
import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "speculative_decoding_verification_80_gb300", "csrc")
ZERO = 5  # the first arrays are zero between calls, the others are scratch


@pytest.fixture(scope="module")
def work(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("work") / "work.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-x", "c++", f"-I{CSRC}", f"-I{os.path.join(ROOT, 'include')}",
                    os.path.join(HERE, "cuda", "page_work.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.words_of.restype = ctypes.c_longlong
    lib.words_of.argtypes = [ctypes.c_longlong]
    lib.arrays_of.argtypes = [ctypes.c_void_p, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_void_p]

    def arrays(N, size):
        at = np.zeros((9, 2), dtype=np.int64)
        lib.arrays_of(1 << 40, size, N, at.ctypes.data)
        return at

    return lib.words_of, arrays


SIZES = [1, 2, 31, 32, 33, 100, 200, 4097, 65536, 1 << 20, 1 << 27]


@pytest.mark.parametrize("more", [0, 1, 3, 4, 1000])
@pytest.mark.parametrize("N", SIZES)
def test_arrays_lie_apart_and_inside(work, N, more):
    words, arrays = work
    at = arrays(N, 4 * words(N) + more)
    order = at[np.argsort(at[:, 0])]
    assert order[0, 0] >= 0 and order[-1, 1] <= words(N) + more // 4 and (order[1:, 0] >= order[:-1, 1]).all()
    assert at[0, 0] == 0 and at[:ZERO, 1].max() == at[:ZERO, 1].sum() - at[:ZERO, 0].sum()  # zero ones from the start on


@pytest.mark.parametrize("a,b", list(itertools.permutations(SIZES, 2)))
def test_one_workspace_serves_pools_of_several_sizes(work, a, b):
    words, arrays = work
    for size in (4 * words(max(a, b)), 4 * words(max(a, b)) + 5000):
        scratch, zero = arrays(a, size)[ZERO:], arrays(b, size)[:ZERO]
        assert scratch[:, 0].min() >= zero[:, 1].max()
