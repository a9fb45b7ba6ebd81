"""The references of capped scores (csrc/packed_order.h), on the host: sums of weights stay within float32."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_sparse_score_gb300", "csrc")
SOURCE = """
#include "packed_order.h"
extern "C" void cap_range(double cap, int keys, double* low, double* high, int* fits) {
    const ha::CapRange r = ha::CapRange::of(cap, keys);
    *low = r.low, *high = r.high, *fits = r.fits();
}
"""


@pytest.fixture(scope="module")
def cap_range(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("range")
    src, so = d / "range.cpp", d / "librange.so"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def of(cap, keys):
        low, high, fits = ctypes.c_double(), ctypes.c_double(), ctypes.c_int()
        lib.cap_range(ctypes.c_double(cap), keys, ctypes.byref(low), ctypes.byref(high), ctypes.byref(fits))
        return low.value, high.value, bool(fits.value)

    return of


@pytest.mark.parametrize("keys", [1, 2, 1000, 1 << 14, 1 << 24, (1 << 24) + 1, (1 << 28) - 1, 1 << 28, (1 << 28) + 1, 1 << 30])
def test_sums_of_weights_stay_within_float32(cap_range, keys):
    """A row whose first keys give the lowest reference, and all others weigh 2^(cap - low), beside values of 2^20; and
    the smallest weight, 2^(-cap - high), beside values of 2^-40: 24 bits above 2^-149."""
    fitting = 0
    for cap in [2.0 ** -60, 1e-3, 1.0, *range(5, 130), 1e3, 2.0 ** 60]:
        low, high, fits = cap_range(cap, keys)
        assert fits == (low <= high)
        if fits:
            fitting += 1
            assert math.log2(keys) + (cap - low) + 20 <= 125
            assert -cap - high - 40 - 24 >= -149 - 1e-9
    assert fitting > 75  # caps of 50 e-folds (72 powers of 2) among them
    assert cap_range(50 / math.log(2), keys)[2]
