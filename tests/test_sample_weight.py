"""spec_sample's weights (csrc/sample_weight.cuh), compiled for the CPU, against
exp in 64 bits."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "speculative_decoding_verification_80_gb300", "csrc")


@pytest.fixture(scope="module")
def weights(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("weight") / "weight.so")
    subprocess.run(["g++", "-O2", "-ffp-contract=off", "-std=c++17", "-shared", "-fPIC", "-x", "c++", f"-I{CSRC}",
                    os.path.join(HERE, "cuda", "sample_weight.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)

    def call(x, top, T):
        x = np.ascontiguousarray(x, dtype=np.float32)
        y = np.zeros(x.size, dtype=np.uint64)
        lib.weights(x.ctypes.data_as(ctypes.c_void_p), x.size, ctypes.c_float(top), ctypes.c_double(np.log2(np.e) / T),
                    y.ctypes.data_as(ctypes.c_void_p))
        return y

    return call


# A weight's own error: t = (x - max) log2(e) / T is below 48 and kept in a pair of floats,
# so it is off by some 2^-47 of itself, 2^-41.4 in all, times ln 2; the series stops at r^5 ln(2)^5 / 120
# < 2^-54, its terms from r^2 on (below 2^-20) are rounded at 2^-24 of themselves, and so are the
# products with the table's pair (below 2^-24 and 2^-20): 2^-43.  Rounding to 2^-44 adds half of that, and
# the float that is rounded, below 2^-22, was itself rounded at 2^-47, an eighth.
REL, ABS = 2.0 ** -40.5, 0.64


@pytest.mark.parametrize("T", [1e-6, 0.013, 0.3, 1.0, 1.7, 40.0])
@pytest.mark.parametrize("top", [-3.7e4, -20.25, -1e-3, 0.0, 2.0 ** -40, 0.71, 13.0, 17.3125, 4097.0])
def test_weights_are_exact_to_2_to_minus_40(weights, T, top):
    rng = np.random.default_rng(int(abs(top) * 10) + int(T * 1000))
    top = np.float32(top)
    x = np.concatenate([top - T * 34.0 * rng.random(20000), top - T * 2.0 ** -rng.integers(0, 40, 4000).astype(float),
                        [top], rng.normal(0, 3, 2000), rng.normal(0, 3, 2000) * 2.0 ** -rng.integers(0, 60, 2000).astype(float)]).astype(np.float32)
    x = x[x <= top]
    d = x.astype(np.longdouble) - np.longdouble(top)
    want = np.exp(d / np.longdouble(T)) * np.longdouble(2) ** 44
    got = weights(x, top, T).astype(np.longdouble)
    assert got[x == top].min() == 2 ** 44
    err = np.abs(got - want)
    # (below e^(-48 / log2 e) of the largest everything is 0, which is nearer than half a unit)
    assert (err <= REL * want + ABS).all(), float((err / (REL * want + ABS)).max())


def test_weights_are_not_biased(weights):
    """Sums of many: errors of both signs, so the mean error is far below one weight's bound."""
    rng = np.random.default_rng(5)
    x = rng.normal(0, 3, 400000).astype(np.float32)
    want = np.exp((x.astype(np.longdouble) - 13) / np.longdouble(1.0)) * np.longdouble(2) ** 44
    x, want = x[x < 13], want[x < 13]
    off = float(abs(weights(x, 13.0, 1.0).astype(np.longdouble).sum() - want.sum()) / want.sum())
    # a rounding to whole numbers has a standard deviation of 0.29; five of those of the sum
    assert off < 5 * 0.3 * x.size ** 0.5 / float(want.sum()) + 2.0 ** -43, off


def test_far_weights_are_zero(weights):
    assert (weights([-1e30, -3.4e38, -40.0], 0.0, 1.0) == 0).all()
    assert (weights([0.0, -1e-5], 1.0, 1e-6) == 0).all()

